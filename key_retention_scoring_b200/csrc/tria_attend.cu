// Attention of many query rows at once on the sm_100a tensor cores: whole
// prompts, causal, packed (tria_prompt_attention), and drafted tokens over the
// cached rows of a layer (tria_tree_attention).
//
// Query row (token i, query head qh of KV head h = qh / G) of sequence s sees
// the keys j < ctx + T for which
//   j < ctx, or j - ctx <= i (a chain), or bit j - ctx of its mask is set
// (prompts: ctx = 0, T = the sequence's length):
//   out_i = sum_j softmax(scale q_i.k_j)_j v_j,  lse_i = log sum_j exp(scale q_i.k_j).
//
// Rows of a KV head's G query heads share its keys, so a tile of 128 rows is
// 128 / G tokens x G heads (one TMA box), and two tiles are in flight:
//   DUALQ: two tiles of rows against the same key blocks (prompts; more than
//          128 rows of drafted tokens);
//   DUALK: one tile of rows, its even and odd key blocks (at most 128 rows:
//          both halves of the SM stay busy although there is one tile).
// Roles (one CTA per SM, persistent):
//   warps 0-3, 4-7  softmax of tile (or key half) 0 and 1, one thread per row:
//                   S from tensor memory, running maximum and sum in fp32,
//                   P as bf16 back over S, the output at the end;
//   warps 8, 10     issue tcgen05.mma for half 0 and 1 (one elected lane):
//                   S = Q K^T (both in shared memory), O += P V (P in tensor
//                   memory, V as it lies, MN-major);
//   warp 9          items of work, and TMA loads of Q and the K tiles;
//   warp 11         TMA loads of the V tiles.
// A step is 64 keys, and each half has two buffers of S, so the product of the
// next step is ready while the softmax of this one runs: with one 128-key
// buffer the chain product, softmax, product set the pace (8448-token prompt,
// 32 query and 8 KV heads: 597 us against 540 when both were built, single
// launches).  In repetition, as the layers of a prefill follow one another, that
// prompt takes 590 us (990 TFLOP/s, SM clock 1.67 GHz under the power cap), 16384
// tokens of 64 query heads 4.25 ms (1035 TFLOP/s, 1.61 GHz; single launches at
// 1.965 GHz 3.79 ms).  What bounds it, single launches: the products alone take 449 us
// (Q K^T in steps of 64 keys reads more shared memory than the tensor core can
// hide), the exponentials, conversions and maxima alone 433 us, and the two
// share the warps' issue slots.
// P is rounded to bf16: the second product needs 16-bit operands, the output
// is rounded to bf16 anyway, and l sums the unrounded weights.
//
// What no row may see.  Masked logits become -inf, so masked weights are 0;
// but 0 x inf and 0 x NaN are NaN, and V rows in a masked place may hold
// anything (later tokens, other sequences, unused slots).  In steps that hold
// masked places the softmax warps therefore look V over in shared memory
// before the product reads it, replace what is not finite by 0 and note it;
// the epilogue then adds those values to the rows that do see them.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "tria_tc.cuh"

namespace tria {
namespace {

using namespace dev;
using namespace tc;

// Waits of the pipeline: the threads sleep in the barrier unit (polling took
// shared-memory cycles from the products: 1.25 times the time); the clock and
// the abort flag are looked at after a sleep that ran out.  The limit counts
// SM cycles at 2 GHz, which is never short and does not step back (time_over).
__device__ __forceinline__ bool poll_on(uint32_t bar, uint32_t parity, const WaitCtl &w) {
  const long long t0 = clock64();
  for (;;) {
    if (mbar_try_sleep(bar, parity, w.hint_ns)) return true;
    if (*w.abort_flag) return false;
    if ((uint64_t)(clock64() - t0) / 2 > w.limit_ns) {
      flag_expiry(w);
      return false;
    }
  }
}

__device__ __forceinline__ bool poll(uint64_t *bar, uint32_t parity, const WaitCtl &w) {
  const uint32_t a = smem_u32(bar);
  return mbar_try_sleep(a, parity, w.hint_ns) || poll_on(a, parity, w);
}

// The same for a whole warp, which leaves together.
__device__ __forceinline__ bool warp_poll(uint64_t *bar, uint32_t parity, const WaitCtl &w) {
  const uint32_t a = smem_u32(bar);
  if (__all_sync(kFull, mbar_try_sleep(a, parity, w.hint_ns))) return true;
  return __all_sync(kFull, poll_on(a, parity, w));
}

constexpr int kBN = 128;                       // keys per block (a ring stage of K or V)
constexpr int kHN = 64;                        // keys per step (a product and its softmax)
constexpr int kNB = kBN / kHN;                 // steps per block, and buffers of S in tensor memory
static_assert(kNB == 2, "mma_role's order of releases");
constexpr int kTile = 2 * kHalfBlock;          // bytes of 128 rows x 128 bf16
constexpr int kSoftWarps = 8;
constexpr int kIssueWarp = 8, kLoadWarp = 9;   // issue: 8 and 10; loads: 9 (items, Q, K) and 11 (V)
constexpr int kAtThreads = 384;                 // the third warpgroup holds the four single-warp roles
// Registers a thread: the kernel is launched with 168 (65536 / 384, rounded
// down to 8); the softmax groups hold a row of S and raise theirs, the third
// group gives up what they take (2 x 208 + 88 = 3 x 168).
constexpr int kLaunchRegs = 168, kSoftRegs = 208, kRoleRegs = 88;
static_assert(2 * kSoftRegs + kRoleRegs == 3 * kLaunchRegs, "register split");
constexpr int kPacked = 2;                     // LAYOUT of prompts, next to the cache layouts
constexpr uint32_t kColS = 0, kColO = 256;     // tensor-memory columns: S (and P) of half t at 128 t, O after them
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum of a row (base 2) moves only when a step exceeds it by
// more than this, so most steps leave O in tensor memory alone; weights stay
// below 2^8, well inside fp32 and bf16.
constexpr float kSlack = 8.f;
// Range of the running maximum.  It is rounded, by up to 64 at 2^30, and all weights
// of the row are off by that factor, which fp32 holds; further out they would
// overflow or vanish.  So it begins at -2^30, logits below have no weight (-inf of
// masked places among them), and one above 2^30 makes its row NaN.
constexpr float kLowest = -1073741824.f;
// Of every 8 pairs of exponentials this many run on the FMA pipe, the rest on the
// special-function unit (16384-token prompt, 64 query heads: 0, 1, 2, 3 of 8 took
// 3779, 3719, 3870, 3800 us).
constexpr int kFmaOf8 = 1;

// A unit (sequence, KV head, tile of rows) whose key blocks several CTAs share,
// written down by the CTA that has its first block: its rows, the slot of the
// first partial, and those of the others.  Every CTA of a call writes one, first
// of all without rows: a CTA that leaves early must not leave combine_kernel what
// an earlier call of the workspace wrote there.
struct Shared {
  int64_t row0;          // first token's row in the output
  int h, rows;           // rows: 0 when no unit begins in this CTA and goes on in the next
  int first, next, step, count;  // slots: first, then next, next + step, ... (count of them)
};

struct AttendParams {
  CUtensorMap qmap, kmap, vmap;
  const uint16_t *v;
  int64_t v_tok, v_head;                       // packed rows
  RowsView view;                               // cached rows
  int layer, n_seq, hq, hkv, g, g_log2;
  int64_t n_tokens;
  const int32_t *starts;
  int max_draft;
  const uint32_t *mask;
  int mask_words;
  float qscale;                                // scale log2(e): base-2 logits
  uint16_t *out;
  float *lse;
  float *part_o, *part_ml;                     // partials (part_at), and their m and l [2 grid][rows][2]
  Shared *shared;                              // [grid]
  int32_t *status;
  uint64_t wait_ns;                            // bound of every wait (0: 2 s)
};

// One piece of work: rows of tokens [tok0, ..) of (s, h) against key blocks [kb0, kb1).
struct Item {
  int s, h, tok0, T, ctx, kb0, kb1, slot;      // slot: -1 writes the output, else a partial
  int steps;                                   // steps with keys that some row sees
  int64_t row0;                                // first row of the sequence in q and out
};

// The ring of K and V tiles.  DUALQ: both halves of the CTA use every tile.
// DUALK: each half has a ring of its own for its key blocks, so that it waits
// for loads in the order in which it used the stages before (the phase of a
// stage that the other half still waits for could not be told apart).
template <bool DUALK>
struct AtCfg {
  static constexpr int QT = DUALK ? 1 : 2;           // tiles of rows
  static constexpr int ROWS = 128 * QT;
  static constexpr int ST = DUALK ? 3 : 5;           // stages of a ring
  static constexpr int RINGS = DUALK ? 2 : 1;
  static __device__ __forceinline__ int stage(int t, int i) { return (DUALK ? ST * t : 0) + i % ST; }
  static __device__ __forceinline__ uint32_t phase(int i) { return (uint32_t)((i / ST) & 1); }
};

template <bool DUALK>
struct AtSmem {
  alignas(1024) uint8_t q[AtCfg<DUALK>::QT][kTile];
  alignas(1024) uint8_t kv[AtCfg<DUALK>::RINGS * AtCfg<DUALK>::ST][kTile];
  alignas(8) uint64_t kv_full[AtCfg<DUALK>::RINGS * AtCfg<DUALK>::ST], kv_empty[AtCfg<DUALK>::RINGS * AtCfg<DUALK>::ST];
  uint64_t q_full, q_empty, s_full[2][2], p_full[2][2], o_done[2], o_full[2], it_full[2], it_empty[2], ml_full, o_read, drain[2];
  Item item[2];
  float ml[DUALK ? 2 : 1][2][DUALK ? 128 : 1];
  volatile int poison[4];  // by item: one half may be two items ahead of the other
  int last_load[2][AtCfg<DUALK>::RINGS], q_loads;  // what the K and the V warp loaded, as they leave
  uint32_t tmem_base;
  volatile int abort_flag;
};

// ---------------------------------------------------------------------------
// what a sequence holds, and the order of the work
// ---------------------------------------------------------------------------
// T, ctx and first row of sequence s; T = 0 for one that is empty or bad (*bad;
// a cached length outside its range is bad with or without drafted tokens).
template <int LAYOUT>
__device__ __forceinline__ void seq_of(const AttendParams &p, int s, int &T, int &ctx, int64_t &row0, bool &bad) {
  const int64_t a = p.starts[s], b = p.starts[s + 1];
  const int n = LAYOUT != kPacked ? view_len(p.view, s, p.layer) : 0;  // read at the same time
  row0 = a;
  bad = a < 0 || b < a || b > p.n_tokens;
  if (LAYOUT != kPacked && !bad)
    bad = n < 0 || b - a > p.max_draft || b - a > p.view.max_seq_len - n;
  T = bad ? 0 : (int)(b - a);
  ctx = T > 0 ? n : 0;
}

// key blocks that tokens [.., tok_end) of a sequence see
__device__ __forceinline__ int key_blocks(const AttendParams &p, int ctx, int T, int tok_end) {
  const int n = ctx + (p.mask != nullptr ? T : min(T, tok_end));
  return (n + kBN - 1) / kBN;
}

// steps of a piece [kb0, kb1) that hold a key some row sees
__device__ __forceinline__ int item_steps(const AttendParams &p, const Item &x, int tok_end) {
  const int keys = x.ctx + (p.mask != nullptr ? x.T : min(x.T, tok_end));
  return min(kNB * (x.kb1 - x.kb0), (keys - x.kb0 * kBN + kHN - 1) / kHN);
}

// Steps of a piece of n blocks that half t of the CTA works on, and its blocks.
// Its ring holds K of its block b in load 2 b and V in load 2 b + 1, counted
// from the item's first load.
template <bool DUALK>
__device__ __forceinline__ int blocks_of(int n, int t) {
  return DUALK ? (n - t + 1) / 2 : n;
}
template <bool DUALK>
__device__ __forceinline__ int steps_of(int n, int steps, int t) {
  if (!DUALK) return steps;
  return kNB * blocks_of<DUALK>(n, t) - (((n - 1) & 1) == t ? kNB * n - steps : 0);
}

// key blocks of a KV head's units (tiles of ROWS rows) of a sequence
template <int ROWS>
__device__ __forceinline__ int64_t seq_blocks(const AttendParams &p, int ctx, int T) {
  const int tpi = ROWS >> p.g_log2, tiles = (T + tpi - 1) / tpi;
  int64_t n = 0;
  if (p.mask != nullptr) {
    n = (int64_t)tiles * key_blocks(p, ctx, T, T);
  } else {
    for (int t = 0; t < T; t += tpi) n += key_blocks(p, ctx, T, t + tpi);
  }
  return n;
}

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

// Prompts: tiles of all sequences, those with the most keys first (tile t of a
// sequence sees t + 1 tiles of keys), all KV heads of a tile side by side; the
// CTAs take them in turn, forth and back, which evens the sums out.
template <bool DUALK>
struct PromptCursor {
  int64_t n_items;
  int tmax, round, mine;  // mine: tiles of sequence `lane` (the first 32 sequences stay in registers)

  static __device__ __forceinline__ int tpi(const AttendParams &p) { return AtCfg<DUALK>::ROWS >> p.g_log2; }

  static __device__ __forceinline__ int tiles(const AttendParams &p, int s, bool &bad) {
    int T, ctx;
    int64_t row0;
    seq_of<kPacked>(p, s, T, ctx, row0, bad);
    return (T + tpi(p) - 1) / tpi(p);
  }

  // tiles with index >= t, over all sequences (their number fits 31 bits, as the tokens' does)
  __device__ __forceinline__ int from(const AttendParams &p, int t, int lane) const {
    int n = max(0, mine - t);
    for (int s = 32 + lane; s < p.n_seq; s += 32) {
      bool bad;
      n += max(0, tiles(p, s, bad) - t);
    }
    return __reduce_add_sync(kFull, n);
  }

  __device__ void init(const AttendParams &p, int lane) {
    bool any_bad = false;
    mine = lane < p.n_seq ? tiles(p, lane, any_bad) : 0;
    int most = mine;
    for (int s = 32 + lane; s < p.n_seq; s += 32) {
      bool bad;
      most = max(most, tiles(p, s, bad));
      any_bad = any_bad || bad;
    }
    if (any_bad && blockIdx.x == 0) atomicOr(p.status, 1);
    tmax = __reduce_max_sync(kFull, most);
    n_items = (int64_t)from(p, 0, lane) * p.hkv;
    round = 0;
  }

  __device__ bool next(const AttendParams &p, int lane, Item &x) {
    const int64_t grid = gridDim.x, b = blockIdx.x;
    const int64_t k = round * grid + ((round & 1) ? grid - 1 - b : b);
    ++round;
    if (k >= n_items) return false;  // later rounds begin behind k
    const int pos = (int)(k / p.hkv);
    x.h = (int)(k % p.hkv);
    int lo = 0, hi = tmax - 1;  // the largest t with from(t) > pos
    if (p.n_seq == 1) {
      lo = tmax - 1 - pos;
    } else {
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (from(p, mid, lane) > pos) lo = mid; else hi = mid - 1;
      }
    }
    int rem = p.n_seq == 1 ? 0 : pos - from(p, lo + 1, lane);
    x.s = 0;
    for (int s0 = 0; s0 < p.n_seq; s0 += 32) {
      int t = mine;
      if (s0 > 0) {
        bool bad;
        t = s0 + lane < p.n_seq ? tiles(p, s0 + lane, bad) : 0;
      }
      const uint32_t has = __ballot_sync(kFull, t > lo);
      const int cnt = __popc(has);
      if (rem < cnt) {
        x.s = s0 + __fns(has, 0, rem + 1);
        break;
      }
      rem -= cnt;
    }
    bool bad;
    seq_of<kPacked>(p, x.s, x.T, x.ctx, x.row0, bad);
    x.tok0 = lo * tpi(p);
    x.kb0 = 0;
    x.kb1 = key_blocks(p, 0, x.T, x.tok0 + tpi(p));
    x.steps = item_steps(p, x, x.tok0 + tpi(p));
    x.slot = -1;
    return true;
  }

  __device__ void finish(const AttendParams &p) const {}
};

// Drafted tokens: the key blocks of all units (sequence, KV head, tile of rows)
// in one line, cut into one piece of equal length per CTA.  A unit that lies in
// several pieces is put together from partials by combine_kernel.
// Paged caches whose rows lie head by head inside a page: one line for each KV
// head, cut into grid / hkv pieces, and neighbouring CTAs take the same piece
// for all heads, so that the pages are read whole at about the same time (64
// sequences of 2048 rows, 8 KV heads, 16-row pages: 147 us in one line, 141 in
// eight).  Where the CTAs are fewer than the heads, one line serves.
struct Lines {
  int heads, cuts, step;  // KV heads in a line, pieces of a line, CTAs between two pieces
};

template <int LAYOUT>
__host__ __device__ __forceinline__ Lines lines_of(int hkv, int grid) {
  if (LAYOUT == TRIA_LAYOUT_PAGED && hkv > 1 && grid >= hkv) return {1, grid / hkv, hkv};
  return {hkv, grid, 1};
}

template <bool DUALK, int LAYOUT>
struct TreeCursor {
  int64_t pos, end, ub;  // blocks of this CTA still to do; where the unit begins
  int s, h, tok0, T, ctx, pieces, heads;
  int64_t row0, w;       // w: blocks of a piece
  Shared goes_on;        // the unit that begins here and goes on in the next CTA

  static __device__ __forceinline__ int tpi(const AttendParams &p) { return AtCfg<DUALK>::ROWS >> p.g_log2; }

  // blocks of sequence s in one head's line
  static __device__ __forceinline__ int64_t blocks(const AttendParams &p, int s, bool &bad) {
    int T, ctx;
    int64_t row0;
    seq_of<LAYOUT>(p, s, T, ctx, row0, bad);
    return seq_blocks<AtCfg<DUALK>::ROWS>(p, ctx, T);
  }

  __device__ void init(const AttendParams &p, int lane) {
    const Lines li = lines_of<LAYOUT>(p.hkv, gridDim.x);
    heads = li.heads;
    // the first 32 sequences stay in registers
    bool any_bad = false;
    const int64_t c0 = lane < p.n_seq ? blocks(p, lane, any_bad) * heads : 0;
    int64_t all = c0;
    for (int i = 32 + lane; i < p.n_seq; i += 32) {
      bool bad;
      all += blocks(p, i, bad) * heads;
      any_bad = any_bad || bad;
    }
    all = warp_sum(all);
    if (any_bad && blockIdx.x == 0) atomicOr(p.status, 1);
    w = (all + li.cuts - 1) / li.cuts;
    goes_on.rows = 0;
    const int cut = blockIdx.x / li.step;
    pos = cut * w;
    end = cut < li.cuts ? min(all, pos + w) : 0;
    pieces = 0;
    if (pos >= end) return;
    // the sequence that holds block `pos`
    int64_t before = 0;
    for (int s0 = 0;; s0 += 32) {
      int64_t c = c0;
      if (s0 > 0) {
        bool bad;
        c = s0 + lane < p.n_seq ? blocks(p, s0 + lane, bad) * heads : 0;
      }
      int64_t incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t past = __ballot_sync(kFull, before + incl > pos);
      if (past) {
        const int at = __ffs(past) - 1;
        s = s0 + at;
        ub = before + __shfl_sync(kFull, incl - c, at);
        break;
      }
      before += __shfl_sync(kFull, incl, 31);
    }
    h = heads > 1 ? 0 : blockIdx.x % li.step;
    load(p);
    while (ub + unit(p) <= pos) step(p);
  }

  __device__ void load(const AttendParams &p) {
    bool bad;
    seq_of<LAYOUT>(p, s, T, ctx, row0, bad);
    if (heads > 1) h = 0;
    tok0 = 0;
  }
  __device__ int unit(const AttendParams &p) const { return key_blocks(p, ctx, T, tok0 + tpi(p)); }
  __device__ void step(const AttendParams &p) {
    ub += unit(p);
    tok0 += tpi(p);
    if (tok0 < T) return;
    tok0 = 0;
    if (heads > 1 && ++h < heads) return;
    do {
      ++s;
      load(p);
    } while (T == 0);  // a block at or behind ub exists, so a later sequence has one
  }

  __device__ bool next(const AttendParams &p, int lane, Item &x) {
    if (pos >= end) return false;
    const int nb = unit(p);
    x.s = s;
    x.h = h;
    x.tok0 = tok0;
    x.T = T;
    x.ctx = ctx;
    x.row0 = row0;
    x.kb0 = (int)(pos - ub);
    x.kb1 = (int)(min(end, ub + nb) - ub);
    x.steps = item_steps(p, x, tok0 + tpi(p));
    x.slot = x.kb1 - x.kb0 == nb ? -1 : 2 * (int)blockIdx.x + (pieces > 0 ? 1 : 0);
    if (x.kb0 == 0 && x.kb1 < nb) {
      const int step = lines_of<LAYOUT>(p.hkv, gridDim.x).step;
      goes_on.row0 = row0 + tok0;
      goes_on.h = h;
      goes_on.rows = min(T - tok0, tpi(p)) << p.g_log2;
      goes_on.first = x.slot;
      goes_on.next = 2 * ((int)blockIdx.x + step);  // the next CTA's first piece
      goes_on.step = 2 * step;
      goes_on.count = (int)((nb - x.kb1 + w - 1) / w);
    }
    pos = ub + x.kb1;
    ++pieces;
    if (pos < end) step(p);
    return true;
  }

  __device__ void finish(const AttendParams &p) const { p.shared[blockIdx.x] = goes_on; }
};

// ---------------------------------------------------------------------------
// loads
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// The K or the V tiles of the items, by one warp each: a tile of a paged cache
// with small pages is up to 32 boxes, and one warp for both fell behind (64
// paged sequences of 2048 rows: 141 us against 116).  A stage passes between
// the two warps; its phases stay apart because the stages of a ring come free in
// the order of the loads (mma_role), so when load i - 2 found its stage free,
// every phase before the one load i waits for is over.
template <bool DUALK, int LAYOUT, bool IS_V>
struct TileLoads {
  using Cfg = AtCfg<DUALK>;
  uint64_t pol;
  int base[Cfg::RINGS];  // loads of each ring before the item
  int done[Cfg::RINGS];  // this warp's last load of each ring, or -1

  __device__ TileLoads() {
    // drafted rows read the cache once; prompts read their keys again for later tiles
    pol = LAYOUT != kPacked && DUALK ? evict_first_policy() : normal_policy();
    for (int t = 0; t < Cfg::RINGS; ++t) {
      base[t] = 0;
      done[t] = -1;
    }
  }

  // all tiles of an item; false when a wait ran out
  __device__ bool item(const AttendParams &p, AtSmem<DUALK> &sm, const Item &x, int lane, const WaitCtl &wc) {
    const CUtensorMap *map = IS_V ? &p.vmap : &p.kmap;
    const int n = x.kb1 - x.kb0, bs = p.view.block_size, at = lane >> 1, half = lane & 1;
    auto page = [&](int j) {  // this lane's block id of key block j
      const int t = (x.kb0 + j) * kBN + at * bs;
      return LAYOUT == TRIA_LAYOUT_PAGED && j < n && at < kBN / bs && t < x.ctx + x.T
                 ? __ldg(p.view.block_table + (int64_t)x.s * p.view.max_blocks + (t >> p.view.block_log2))
                 : 0;
    };
    int blk = page(0);
    for (int j = 0; j < n; ++j) {
      const int t = DUALK ? j & 1 : 0, i = base[t] + 2 * (DUALK ? j >> 1 : j) + (IS_V ? 1 : 0);
      const int stage = Cfg::stage(t, i), slot0 = (x.kb0 + j) * kBN;
      if (i >= Cfg::ST) {
        bool free = true;
        if (lane == 0) free = poll(&sm.kv_empty[stage], Cfg::phase(i - Cfg::ST), wc);
        if (!__shfl_sync(kFull, free ? 1 : 0, 0)) return false;
      }
      const uint32_t dst = smem_u32(&sm.kv[stage][0]);
      if (LAYOUT != TRIA_LAYOUT_PAGED) {
        if (lane == 0) mbar_arrive_expect_tx(&sm.kv_full[stage], kTile);
        __syncwarp();
        if (lane < 2) {
          if (LAYOUT == kPacked)
            tma_load_4d(dst + lane * kHalfBlock, map, lane * 64, (int)x.row0 + slot0, x.h, 0, &sm.kv_full[stage], pol);
          else
            tma_load_4d(dst + lane * kHalfBlock, map, lane * 64, slot0, x.h, x.s, &sm.kv_full[stage], pol);
        }
      } else {
        // one box per page and 64-dim half; pages behind the last row stay unread
        // (what the stage holds there is masked)
        const bool valid = at < kBN / bs && slot0 + at * bs < x.ctx + x.T;
        const int boxes = __popc(__ballot_sync(kFull, valid)), now = blk;
        blk = page(j + 1);
        if (lane == 0) mbar_arrive_expect_tx(&sm.kv_full[stage], (uint32_t)(boxes * bs * 128));
        __syncwarp();
        if (valid)
          tma_load_4d(dst + half * kHalfBlock + at * bs * 128, map, half * 64, x.h, 0, now, &sm.kv_full[stage], pol);
      }
      done[t] = i;
    }
    for (int t = 0; t < Cfg::RINGS; ++t) base[t] += 2 * blocks_of<DUALK>(n, t);
    return true;
  }

  // as the warp leaves: what drain_loads may have to wait for
  __device__ void leave(AtSmem<DUALK> &sm) const {
    for (int t = 0; t < Cfg::RINGS; ++t) sm.last_load[IS_V ? 1 : 0][t] = done[t];
  }
};

// After a wait ran out, when every role has left (one thread): loads still in
// flight must land before the block exits, those of a load warp that had come to
// the end of its work included.  A stage passes from one load warp to the other,
// so the last load into it, of either, is the one to wait for: it was issued when
// those before it had landed.
template <bool DUALK>
__device__ void drain_loads(AtSmem<DUALK> &sm, int32_t *status) {
  using Cfg = AtCfg<DUALK>;
  for (int t = 0; t < Cfg::RINGS; ++t) {
    for (int s = 0; s < Cfg::ST; ++s) {
      int last = -1;  // of the K warp's even loads and the V warp's odd ones
      for (int w = 0; w < 2; ++w)
        for (int i = sm.last_load[w][t]; i >= w && i > last; i -= 2)
          if (i % Cfg::ST == s) last = i;
      if (last >= 0) mbar_drain(&sm.kv_full[Cfg::stage(t, last)], Cfg::phase(last), status);
    }
  }
  if (sm.q_loads > 0) mbar_drain(&sm.q_full, (uint32_t)((sm.q_loads - 1) & 1), status);
}

// Items of work for everyone, Q and K.
template <bool DUALK, int LAYOUT, class Cursor>
__device__ void load_role(const AttendParams &p, AtSmem<DUALK> &sm, int lane, const WaitCtl wc) {
  using Cfg = AtCfg<DUALK>;
  const uint64_t qpol = normal_policy();
  TileLoads<DUALK, LAYOUT, false> keys;
  Cursor cur;
  cur.init(p, lane);
  int it = 0, q_loads = 0;
  Item x{};
  auto wait = [&](uint64_t *bar, int phase) {
    bool good = true;
    if (lane == 0) good = poll(bar, (uint32_t)(phase & 1), wc);
    return __shfl_sync(kFull, good ? 1 : 0, 0) != 0;
  };
  for (;;) {
    const bool more = cur.next(p, lane, x);
    const int slot = it & 1;
    if (it >= 2 && !wait(&sm.it_empty[slot], (it >> 1) - 1)) break;
    if (lane == 0) {
      if (!more) x.kb1 = -1;
      sm.item[slot] = x;
      mbar_arrive(&sm.it_full[slot]);
    }
    ++it;
    if (!more) {
      if (lane == 0) cur.finish(p);
      break;
    }
    if (it > 1 && !wait(&sm.q_empty, it - 2)) break;
    if (lane == 0) mbar_arrive_expect_tx(&sm.q_full, Cfg::QT * kTile);
    __syncwarp();
    if (lane < 2 * Cfg::QT) {
      const int t = lane >> 1, half = lane & 1;
      tma_load_4d(smem_u32(&sm.q[t][half * kHalfBlock]), &p.qmap, half * 64, x.h << p.g_log2,
                  (int)x.row0 + x.tok0 + t * (kRows >> p.g_log2), 0, &sm.q_full, qpol);
    }
    ++q_loads;
    if (!keys.item(p, sm, x, lane, wc)) break;
  }
  if (lane == 0) {
    keys.leave(sm);
    sm.q_loads = q_loads;
  }
  __syncwarp();
}

template <bool DUALK, int LAYOUT>
__device__ void value_role(const AttendParams &p, AtSmem<DUALK> &sm, int lane, const WaitCtl wc) {
  TileLoads<DUALK, LAYOUT, true> values;
  bool ok = true;
  for (int it = 0; ok; ++it) {
    if (!(ok = warp_poll(&sm.it_full[it & 1], (uint32_t)((it >> 1) & 1), wc))) break;
    const Item x = sm.item[it & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.it_empty[it & 1]);
    if (x.kb1 < 0) break;
    ok = values.item(p, sm, x, lane, wc);
  }
  if (lane == 0) values.leave(sm);
  __syncwarp();
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
// V tile as the B operand of O += P V: N = dims, which lie contiguous (MN-
// major): 128-byte swizzle, the two 64-dim halves kHalfBlock bytes apart
// (leading offset), 8-key groups 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(kHalfBlock >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

constexpr uint32_t kIdescS = idesc_bf16_m128_n(kHN);
constexpr uint32_t kIdescO = idesc_bf16_m128_n(kHeadDim) | (1u << 16);  // B is MN-major

// The products are issued by one elected lane of a warp that stays together,
// several to one asm block: an issue from a diverged lane took 64 cycles
// whatever the product's size (the operands went through the vector registers
// one by one), one of these takes 20, and a step of 16 keys takes 64.
#define TRIA_MMA_QK(step) \
  "add.s64 x, %1, " step ";\n add.s64 y, %2, " step ";\n" \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n"
// S = Q K^T: 8 steps of 16 dims; a step is 32 bytes on in the swizzled rows,
// four steps on is the other 64-dim half.
__device__ __forceinline__ void mma_qk(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  static_assert(kHalfBlock >> 4 == 1024, "descriptor offset of the second half");
  asm volatile(
      "{\n .reg .pred q, t, f;\n .reg .b64 x, y;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 t, 1, 0;\n"
      " setp.ne.b32 f, 0, 0;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n"
      TRIA_MMA_QK("2") TRIA_MMA_QK("4") TRIA_MMA_QK("6") TRIA_MMA_QK("1024") TRIA_MMA_QK("1026")
      TRIA_MMA_QK("1028") TRIA_MMA_QK("1030") "}" ::"r"(d), "l"(a), "l"(b), "r"(idesc)
      : "memory");
}
#undef TRIA_MMA_QK

#define TRIA_MMA_PV(col, row) \
  "add.s32 z, %1, " col ";\n add.s64 y, %2, " row ";\n" \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [z], y, %3, t;\n"
// O += P V: 4 steps of 16 keys, 8 columns of P and 16 rows of V each.
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred q, t, f;\n .reg .b64 y;\n .reg .b32 z;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 t, 1, 0;\n"
      " setp.ne.b32 f, %4, 0;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n"
      TRIA_MMA_PV("8", "128") TRIA_MMA_PV("16", "256") TRIA_MMA_PV("24", "384")
      "}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
#undef TRIA_MMA_PV

__device__ __forceinline__ void elect_commit(uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar))
      : "memory");
}

// One warp for each half t of the CTA: the tensor core takes their products in
// turn, and neither waits where the other waits for its softmax.
template <bool DUALK>
__device__ void mma_role(const AttendParams &p, AtSmem<DUALK> &sm, uint32_t tmem, int t, int lane, const WaitCtl wc) {
  using Cfg = AtCfg<DUALK>;
  constexpr uint32_t kHalfRows = (kHN * 128) >> 4;  // 64 rows on in a tile, as a descriptor offset
  const uint32_t s_col = tmem + kColS + 128u * t, o_col = tmem + kColO + 128u * t;
  const uint64_t q_at = sw128_desc(smem_u32(&sm.q[DUALK ? 0 : t][0]));
  const uint64_t k_at = sw128_desc(smem_u32(&sm.kv[0][0])), v_at = v_desc(smem_u32(&sm.kv[0][0]));
  int base = 0;
  uint32_t pp = 0;  // phases of p_full, bit b
  bool ok = true, issued = false;
  for (int it = 0; ok; ++it) {
    if (!(ok = warp_poll(&sm.it_full[it & 1], (uint32_t)((it >> 1) & 1), wc))) break;
    const int n = sm.item[it & 1].kb1 - sm.item[it & 1].kb0, steps = sm.item[it & 1].steps;
    const bool end = sm.item[it & 1].kb1 < 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.it_empty[it & 1]);
    if (end) break;
    if (!(ok = warp_poll(&sm.q_full, (uint32_t)(it & 1), wc))) break;
    const int mine = steps_of<DUALK>(n, steps, t);
    if (mine == 0 && lane == 0) mbar_arrive(&sm.q_empty);
    auto kv_wait = [&](int i) { return warp_poll(&sm.kv_full[Cfg::stage(t, i)], Cfg::phase(i), wc); };
    // S of step g into its buffer.  K is released behind its last step, but never
    // before V of the block before it (the loads count on stages coming free in
    // the order of their use): a block with one step leaves that to the product
    // of the step before it.
    auto qk = [&](int g) {
      const int i = base + 2 * (g / kNB), b = g % kNB;
      if (b == 0 && !kv_wait(i)) return false;
      mma_qk(s_col + 64u * b, q_at, k_at + (uint32_t)(Cfg::stage(t, i) * (kTile >> 4)) + b * kHalfRows, kIdescS);
      elect_commit(&sm.s_full[t][b]);
      if (b == kNB - 1 || mine == 1) elect_commit(&sm.kv_empty[Cfg::stage(t, i)]);
      if (g + 1 == mine) elect_commit(&sm.q_empty);
      issued = true;
      return true;
    };
    for (int g = 0; ok && g < kNB && g < mine; ++g) ok = qk(g);
    for (int g = 0; ok && g < mine; ++g) {
      const int b = g % kNB, i = base + 2 * (g / kNB) + 1;
      if (b == 0 && !(ok = kv_wait(i))) break;
      if (!(ok = warp_poll(&sm.p_full[t][b], (pp >> b) & 1u, wc))) break;
      pp ^= 1u << b;
      tc_fence_after();
      mma_pv(o_col, s_col + 64u * b, v_at + (uint32_t)(Cfg::stage(t, i) * (kTile >> 4)) + b * kHalfRows, kIdescO, g > 0 ? 1u : 0u);
      elect_commit(&sm.o_done[t]);
      if (b == kNB - 1 || g + 1 == mine) elect_commit(&sm.kv_empty[Cfg::stage(t, i)]);
      if (b == kNB - 1 && g + 2 == mine) elect_commit(&sm.kv_empty[Cfg::stage(t, i + 1)]);
      if (g + 1 == mine) elect_commit(&sm.o_full[t]);
      if (g + kNB < mine) ok = qk(g + kNB);
    }
    base += 2 * blocks_of<DUALK>(n, t);
  }
  // the products already issued must land before the tensor memory is freed
  if (issued) {
    elect_commit(&sm.drain[t]);
    if (lane == 0) mbar_drain(&sm.drain[t], 0, wc.status);
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// softmax and output
// ---------------------------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 in a register pair: the packed multiply-add and add take one issue
// slot for both, and pairs that stay pairs need no moves.
using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 2^x of both on the FMA pipe (far below -126 gives about 2^-126): 2^x = 2^n 2^f
// with n the nearest integer (the low bits of x + 1.5 2^23) and f in [-1/2,
// 1/2], 2^f by a polynomial of degree 4 fitted to the smallest maximal relative
// error (2.7e-6), n added to the exponent bits.
__device__ __forceinline__ f32x2 exp2_fma(f32x2 v) {
  float2 x = both(v);
  v = pair(fmaxf(x.x, -126.f), fmaxf(x.y, -126.f));
  auto c2 = [](float c) { return pair(c, c); };
  const f32x2 t = add2(v, c2(12582912.f));
  const f32x2 f = fma2(add2(t, c2(-12582912.f)), c2(-1.f), v);
  f32x2 q = fma2(c2(0.009570101276040077f), f, c2(0.05591786280274391f));
  q = fma2(q, f, c2(0.240247443318367f));
  q = fma2(q, f, c2(0.6931217908859253f));
  q = fma2(q, f, c2(0.9999992847442627f));
  const float2 n = both(t), y = both(q);
  return pair(__int_as_float(__float_as_int(y.x) + (__float_as_int(n.x) << 23)),
              __int_as_float(__float_as_int(y.y) + (__float_as_int(n.y) << 23)));
}

__device__ __forceinline__ uint32_t pack_bf16(float x0, float x1) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ bool bf16_not_finite(uint32_t half) { return (half & 0x7f80u) == 0x7f80u; }

// Replaces what is not finite in half a V tile (64 keys) by 0 (the 128 threads
// of a softmax group); true where this thread found something.  x * 0 + acc
// keeps a NaN, so one bf16x2 multiply-add per two values tells whether to look
// closer.
__device__ __forceinline__ bool clean_v(uint8_t *half, int tid, volatile int *poison, int mark) {
  constexpr int kPasses = kHN * 8 / 128;  // of 128 x 16 bytes over the keys of one 64-dim half
  auto at = [&](int i) { return half + (i / kPasses) * kHalfBlock + ((i % kPasses) * 128 + tid) * 16; };
  uint32_t acc = 0;
#pragma unroll
  for (int i = 0; i < 2 * kPasses; ++i) {
    const uint4 w = lds128(at(i));
    for (uint32_t x : {w.x, w.y, w.z, w.w})
      asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
  }
  if ((acc & 0x7fff7fffu) == 0) return false;
  *poison = mark;
  __threadfence_block();
  for (int i = 0; i < 2 * kPasses; ++i) {
    uint32_t *w = reinterpret_cast<uint32_t *>(at(i));
    for (int e = 0; e < 4; ++e) {
      const uint32_t x = w[e];
      const uint32_t y = (bf16_not_finite(x) ? 0u : x & 0xffffu) | (bf16_not_finite(x >> 16) ? 0u : x & 0xffff0000u);
      if (y != x) w[e] = y;
    }
  }
  return true;
}

// Bit c: this row may see key k0 + c (c < 32).
__device__ __forceinline__ uint32_t sees(const AttendParams &p, const Item &x, int tok, int k0) {
  if (tok >= x.T) return 0u;
  const int rel = k0 - x.ctx;  // drafted row of the first key
  int n;                       // keys [k0, k0 + n) exist (and a chain's row sees them all)
  if (p.mask == nullptr) {
    n = tok + 1 - rel;
  } else {
    n = x.T - rel;
  }
  if (n <= 0) return 0u;
  uint32_t bits = n >= 32 ? ~0u : (1u << n) - 1u;
  if (p.mask != nullptr && rel > -32) {
    const uint32_t *m = p.mask + (x.row0 + tok) * p.mask_words;
    if (rel < 0) {
      bits &= (m[0] << -rel) | ((1u << -rel) - 1u);
    } else {
      const int w = rel >> 5;
      const uint32_t lo = w < p.mask_words ? m[w] : 0u, hi = w + 1 < p.mask_words ? m[w + 1] : 0u;
      bits &= __funnelshift_r(lo, hi, rel & 31);
    }
  }
  return bits;
}

// Whether the step of keys from k0 on holds masked places.
__device__ __forceinline__ bool step_masked(const AttendParams &p, const Item &x, int k0) {
  return p.mask != nullptr ? k0 + kHN > x.ctx : k0 + kHN - 1 > x.ctx + x.tok0;
}

// Whether this row may see any key at all (asked where no logit had weight).
__device__ __noinline__ bool sees_any(const AttendParams &p, const Item &x, int tok) {
  if (tok >= x.T) return false;
  if (x.ctx > 0 || p.mask == nullptr) return true;
  uint32_t any = 0;
  for (int k0 = 0; k0 < x.T; k0 += 32) any |= sees(p, x, tok, k0);
  return any != 0;
}

// v_j that are not finite, of the masked steps' keys that this row sees, added to o (dims d0 .. d0 + 31).
template <int LAYOUT>
__device__ __noinline__ void add_not_finite(const AttendParams &p, const Item &x, int tok, int d0, float (&o)[32]) {
  if (tok >= x.T) return;
  for (int h0 = x.kb0 * kBN; h0 < x.kb0 * kBN + x.steps * kHN; h0 += kHN) {
    if (!step_masked(p, x, h0)) continue;
    for (int k0 = h0; k0 < h0 + kHN; k0 += 32) {
      uint32_t bits = sees(p, x, tok, k0);
      while (bits) {
        const int j = k0 + __ffs(bits) - 1;
        bits &= bits - 1u;
        const uint16_t *v = p.v;
        if (LAYOUT == kPacked) {
          v += (x.row0 + j) * p.v_tok + (int64_t)x.h * p.v_head;
        } else {
          int64_t off;
          if (!view_row(p.view, x.s, x.h, j, &off)) continue;
          v += off;
        }
#pragma unroll
        for (int d = 0; d < 32; ++d) {
          const uint32_t y = v[d0 + d];
          if (bf16_not_finite(y)) o[d] += __uint_as_float(y << 16);
        }
      }
    }
  }
}

// O *= a for the rows of this warp.  Seldom: kept out of the softmax loop.
__device__ __noinline__ bool rescale(uint32_t o_col, float a, uint64_t *done, uint32_t parity, const WaitCtl &wc) {
  // The product before this step's must have been added to O.  The one before
  // that has (S of this step was issued behind it and its barrier came after),
  // so the phase waited for is this one or the one after it.
  if (!warp_poll(done, parity, wc)) return false;
  tc_fence_after();
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t o[32];
    tmem_ld_nowait<32>(o_col + 32u * c, o);
    tmem_wait_ld();
    uint32_t o0[16], o1[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      o0[e] = __float_as_uint(__uint_as_float(o[e]) * a);
      o1[e] = __float_as_uint(__uint_as_float(o[16 + e]) * a);
    }
    tmem_st<16>(o_col + 32u * c, o0);
    tmem_st<16>(o_col + 32u * c + 16u, o1);
  }
  tmem_wait_st();
  return true;
}

// Four dims (d4) of a row of a partial, in float4: the rows lie side by side, so
// that warps whose lanes are rows write and read whole lines (row by row, the
// writes alone took 3 us of a 32K-token call).
template <int ROWS>
__device__ __forceinline__ int64_t part_at(int slot, int row, int d4) {
  return ((int64_t)slot * 32 + d4) * ROWS + row;
}

// A row's l where it sees keys, none with weight: such a row has no softmax (0 / 0).
// 0 is a row that sees no key.
constexpr float kNoWeight = -1.f;

// l of a row at the end: what its weights summed to at kLowest is the FMA pipe's
// floor (a NaN stays).
__device__ __forceinline__ float weight_sum(float m, float l) { return m == kLowest && l == l ? 0.f : l; }

__device__ __forceinline__ float inverse(float l) { return l > 0.f ? 1.f / l : l == 0.f ? 0.f : NAN; }
__device__ __forceinline__ float log_sum(float m, float l) { return l <= 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }

// One step of transposing 4 x 4 pieces of 4 words over 4 lanes: lanes MASK apart
// swap the pieces that lie WORDS apart.
template <int MASK, int WORDS>
__device__ __forceinline__ void exchange4(uint32_t (&w)[16], int lane) {
  const bool upper = (lane & MASK) != 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    if (e & WORDS) continue;
    const uint32_t got = __shfl_xor_sync(kFull, upper ? w[e] : w[e + WORDS], MASK);
    if (upper) w[e] = got; else w[e + WORDS] = got;
  }
}

template <bool DUALK, int LAYOUT>
__device__ void soft_role(const AttendParams &p, AtSmem<DUALK> &sm, uint32_t tmem, int warp, int lane,
                          const WaitCtl wc) {
  using Cfg = AtCfg<DUALK>;
  const int t = warp >> 2, w = warp & 3, r = w * 32 + lane;
  const uint32_t lanes = (uint32_t)(32 * w) << 16;
  const uint32_t ts = tmem + lanes + kColS + 128u * t, to = tmem + lanes + kColO + 128u * t;
  const float qs = p.qscale;
  uint32_t sp = 0;           // phases of s_full, bit b
  uint32_t of = 0;           // phases of o_full, bit i
  int od[2] = {0, 0};        // products of each half before the item
  int base = 0;              // loads of this half's ring before the item
  for (int it = 0;; ++it) {
    if (!warp_poll(&sm.it_full[it & 1], (uint32_t)((it >> 1) & 1), wc)) return;
    const Item x = sm.item[it & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.it_empty[it & 1]);
    if (x.kb1 < 0) return;
    const int n = x.kb1 - x.kb0, mine = steps_of<DUALK>(n, x.steps, t);
    const int first_tok = x.tok0 + (DUALK ? 0 : t * (kRows >> p.g_log2));
    const int tok = first_tok + (r >> p.g_log2);
    const bool idle = first_tok + ((w * 32) >> p.g_log2) >= x.T;  // no row of this warp is one of the sequence
    float m = kLowest, l = 0.f;
    // The softmax of step g.  Steps with masked places come last and have code of
    // their own: one loop for both took 1.25 times as long, masked or not.
    auto step = [&](auto is_masked, int g) -> bool {
      constexpr bool MASKED = decltype(is_masked)::value;
      const int b = g % kNB, j = DUALK ? 2 * (g / kNB) + t : g / kNB, k0 = (x.kb0 + j) * kBN + b * kHN;
      if constexpr (MASKED) {
        const int i = base + 2 * (g / kNB) + 1;
        if (!warp_poll(&sm.kv_full[Cfg::stage(t, i)], Cfg::phase(i), wc)) return false;
        const bool found = clean_v(sm.kv[Cfg::stage(t, i)] + b * (kHN * 128), r, &sm.poison[it & 3], it + 1);
        // DUALQ: what this thread found clean the other half's may have replaced
        if (found || !DUALK)
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      if (!warp_poll(&sm.s_full[t][b], (sp >> b) & 1u, wc)) return false;
      sp ^= 1u << b;
      tc_fence_after();
      if (!idle) {
        const uint32_t tsb = ts + 64u * b;
        f32x2 s[kHN / 2];
        {
          uint32_t u[kHN / 32][32];
#pragma unroll
          for (int c = 0; c < kHN / 32; ++c) tmem_ld_nowait<32>(tsb + 32u * c, u[c]);
          tmem_wait_ld();
          if constexpr (MASKED) {
#pragma unroll
            for (int c = 0; c < kHN / 32; ++c) {
              const uint32_t bits = sees(p, x, tok, k0 + 32 * c);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((bits >> e) & 1u)) u[c][e] = 0xff800000u;  // -inf
            }
          }
#pragma unroll
          for (int c = 0; c < kHN / 2; ++c)
            s[c] = pair(__uint_as_float(u[c >> 4][2 * c & 31]), __uint_as_float(u[c >> 4][(2 * c + 1) & 31]));
        }
        float2 mx[4] = {both(s[0]), both(s[1]), both(s[2]), both(s[3])};
#pragma unroll
        for (int c = 4; c < kHN / 2 - 4; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = both(s[c + e]), z = both(s[c + 4 + e]);
            mx[e].x = max3_nan(mx[e].x, y.x, z.x);
            mx[e].y = max3_nan(mx[e].y, y.y, z.y);
          }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 y = both(s[kHN / 2 - 4 + e]);
          mx[e].x = max_nan(mx[e].x, y.x);
          mx[e].y = max_nan(mx[e].y, y.y);
        }
        const float top = max3_nan(max3_nan(mx[0].x, mx[0].y, mx[1].x), max3_nan(mx[1].y, mx[2].x, mx[2].y),
                                   max_nan(mx[3].x, mx[3].y)) * qs;
        const bool up = top > m + kSlack;
        if (__any_sync(kFull, up)) {
          const float mn = up ? top : m;
          const float a = up ? ex2(m - mn) : 1.f;
          m = mn;
          l *= a;
          if (g > 0 && !rescale(to, a, &sm.o_done[t], (uint32_t)((od[t] + g - 1) & 1), wc)) return false;
        }
        // a NaN, +inf or too large logit makes the row NaN, whichever way its exponential is taken
        if (!(top <= -kLowest)) l = NAN;
        const f32x2 mu2 = pair(-m, -m), qs2 = pair(qs, qs);
        // of every 8 pairs of weights, the first `fma` go to the FMA pipe
        auto weights = [&](int fma) {
#pragma unroll
          for (int c = 0; c < kHN / 32; ++c) {
            uint32_t pw[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              f32x2 &v = s[16 * c + e];
              v = fma2(v, qs2, mu2);
              if (e % 8 < fma) {
                v = exp2_fma(v);
              } else {
                const float2 y = both(v);
                v = pair(ex2(y.x), ex2(y.y));
              }
              const float2 y = both(v);
              pw[e] = pack_bf16(y.x, y.y);
            }
            tmem_st<16>(tsb + 16u * c, pw);
          }
        };
        weights(MASKED ? 0 : kFmaOf8);  // masked logits need exact zeros
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[t][b]);
        // the sum is not on the way to the next product
        f32x2 sum[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < kHN / 2; c += 4)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], s[c + e]);
        const float2 all = both(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
        l += all.x + all.y;
      } else {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[t][b]);
      }
      return true;
    };
    int clear = 0;  // steps without masked places
    {
      const int keys = p.mask != nullptr ? x.ctx : x.ctx + x.tok0 + 1;  // seen by every row
      const int whole = keys / kHN - x.kb0 * kNB;                         // steps of the item below them
      const int blocks = whole > 0 ? whole / kNB : 0, rest = whole > 0 ? whole % kNB : 0;
      clear = DUALK ? kNB * (max(0, blocks - t + 1) / 2) + ((blocks & 1) == t ? rest : 0) : whole;
      clear = max(0, min(mine, clear));
    }
    int g = 0;
    for (; g < clear; ++g)
      if (!step(std::false_type{}, g)) return;
    for (; g < mine; ++g)
      if (!step(std::true_type{}, g)) return;
    base += 2 * blocks_of<DUALK>(n, t);

    // output: O / l, or O, m and l as a partial
    float f0 = 1.f, f1 = 0.f;  // DUALK: factors of the two halves' O
    if (DUALK) {
      sm.ml[t][0][r] = m;
      sm.ml[t][1][r] = weight_sum(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ml_full);
      if (!warp_poll(&sm.ml_full, (uint32_t)(it & 1), wc)) return;
      const float m0 = sm.ml[0][0][r], m1 = sm.ml[1][0][r];
      m = fmaxf(m0, m1);
      f0 = ex2(m0 - m);
      f1 = ex2(m1 - m);
      l = sm.ml[0][1][r] * f0 + sm.ml[1][1][r] * f1;
    }
    // the last product of this half (DUALK: of both) must have been added to O
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int hi = steps_of<DUALK>(n, x.steps, i);
      od[i] += hi;
      if (hi == 0) continue;
      if ((DUALK || i == t) && !warp_poll(&sm.o_full[i], (of >> i) & 1u, wc)) return;
      of ^= 1u << i;
    }
    tc_fence_after();
    if (!idle) {
      const bool poisoned = sm.poison[it & 3] == it + 1;
      const bool mine_row = tok < x.T;
      l = weight_sum(m, l);
      if (l == 0.f) {
        const Item z = x;
        if (sees_any(p, z, tok)) l = kNoWeight;
      }
      __syncwarp();  // the reads of O below are the whole warp's
      const float inv = x.slot >= 0 ? 1.f : inverse(l);
      const int row = (DUALK ? 0 : 128 * t) + r;
      const int64_t orow = (x.row0 + tok) * p.hq + ((int64_t)x.h << p.g_log2) + (r & (p.g - 1));
      constexpr int kChunks = DUALK ? 2 : 4;  // DUALK: each group takes 64 of the dims
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int d0 = (DUALK ? 64 * t : 0) + 32 * c;
        const uint32_t col = tmem + lanes + kColO + (DUALK ? 0u : 128u * t) + (uint32_t)d0;
        float o[32];
        {
          uint32_t u[32];
          tmem_ld_nowait<32>(col, u);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(u[e]) * (DUALK ? f0 : 1.f);
          if (DUALK && n > 1) {
            tmem_ld_nowait<32>(col + 128u, u);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(u[e]), f1, o[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= inv;
        if (poisoned) {
          float y[32];  // a copy, so that o itself stays in registers
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = o[e];
          const Item z = x;
          add_not_finite<LAYOUT>(p, z, tok, d0, y);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = y[e];
        }
        if (x.slot >= 0) {
          float4 *dst = reinterpret_cast<float4 *>(p.part_o) + part_at<Cfg::ROWS>(x.slot, row, d0 / 4);
          if (mine_row)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e * Cfg::ROWS] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else {
          // Four lanes exchange 16-byte pieces so that they write 64 bytes of one
          // row at a time (each lane its own row: four times the line accesses).
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) pw[e] = pack_bf16(o[2 * e], o[2 * e + 1]);
          exchange4<1, 4>(pw, lane);
          exchange4<2, 8>(pw, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t to = __shfl_sync(kFull, mine_row ? orow : -1, (lane & ~3) + i);
            if (to >= 0)
              *reinterpret_cast<uint4 *>(p.out + to * 128 + d0 + 8 * (lane & 3)) =
                  make_uint4(pw[4 * i], pw[4 * i + 1], pw[4 * i + 2], pw[4 * i + 3]);
          }
        }
      }
      if (mine_row && (!DUALK || t == 0)) {
        if (x.slot >= 0)
          *reinterpret_cast<float2 *>(p.part_ml + ((int64_t)x.slot * Cfg::ROWS + row) * 2) = make_float2(m, l);
        else if (p.lse != nullptr)
          p.lse[orow] = log_sum(m, l);
      }
    }
    tc_fence_before();
    if (DUALK) {
      // the next item's products may overwrite O once both groups have read it
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_read);
      if (!warp_poll(&sm.o_read, (uint32_t)(it & 1), wc)) return;
    }
  }
}

template <bool DUALK, int LAYOUT>
__global__ void __launch_bounds__(kAtThreads, 1) attend_kernel(const __grid_constant__ AttendParams p) {
  using Cfg = AtCfg<DUALK>;
  extern __shared__ __align__(1024) uint8_t smem_dyn[];
  AtSmem<DUALK> &sm = *reinterpret_cast<AtSmem<DUALK> *>(smem_dyn);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // by the thread that writes the CTA's record at the end
  auto no_record = [&] {
    if (LAYOUT != kPacked && tid == 32 * kLoadWarp) p.shared[blockIdx.x].rows = 0;
  };
  // the block's memory is full, with no room to move the tiles to a boundary
  if (smem_u32(smem_dyn) & 1023u) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    no_record();
    if (tid == 0) atomicOr(p.status, 2);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < Cfg::RINGS * Cfg::ST; ++i) {
      mbar_init(&sm.kv_full[i], 1);
      mbar_init(&sm.kv_empty[i], DUALK ? 1 : 2);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 2);
    for (int i = 0; i < 2; ++i) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sm.s_full[i][b], 1);
        mbar_init(&sm.p_full[i][b], 4);
      }
      mbar_init(&sm.o_done[i], 1);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.drain[i], 1);
      mbar_init(&sm.it_full[i], 1);
      mbar_init(&sm.it_empty[i], kSoftWarps + 3);
    }
    for (int i = 0; i < 4; ++i) sm.poison[i] = 0;
    mbar_init(&sm.ml_full, kSoftWarps);
    mbar_init(&sm.o_read, kSoftWarps);
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == kLoadWarp && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &p.qmap : lane == 1 ? &p.kmap : &p.vmap) : "memory");
  if (warp == kIssueWarp) tmem_alloc(&sm.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  // The block may have started beside the kernel before it in the stream: no global
  // memory is touched before this, and no role's limit on its waits runs before it
  // (that kernel may take longer than the limit).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  no_record();
  const WaitCtl wc = wait_ctl(&sm.abort_flag, p.status, p.wait_ns);
  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    soft_role<DUALK, LAYOUT>(p, sm, tmem, warp, lane, wc);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
    if (warp == kLoadWarp) {
      if constexpr (LAYOUT == kPacked)
        load_role<DUALK, LAYOUT, PromptCursor<DUALK>>(p, sm, lane, wc);
      else
        load_role<DUALK, LAYOUT, TreeCursor<DUALK, LAYOUT>>(p, sm, lane, wc);
    } else if (warp == kLoadWarp + 2) {
      value_role<DUALK, LAYOUT>(p, sm, lane, wc);
    } else {
      mma_role<DUALK>(p, sm, tmem, (warp - kIssueWarp) >> 1, lane, wc);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && sm.abort_flag) drain_loads<DUALK>(sm, p.status);
}

// ---------------------------------------------------------------------------
// Partials of a unit that several CTAs worked on, put together: out = sum_c
// 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c.  A lane has one row and four dims,
// as the partials lie.  Latency bounds it: the unit's record, then its partials
// (8 units of 128 rows in 19 parts each, 10 MB: 7 us of a call of 41).
// ---------------------------------------------------------------------------
constexpr int kCombineWarps = 8;
constexpr int kBatch = 6;  // partials in flight

template <int ROWS>
__global__ void __launch_bounds__(32 * kCombineWarps, 4) combine_kernel(const __grid_constant__ AttendParams p, int grid) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // started beside the end of attend_kernel
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the blockIdx.x-th of the CTAs in which a shared unit begins
  int cta = -1;
  for (int c0 = 0, before = 0; c0 < grid && cta < 0; c0 += 32 * 5) {
    int rows[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int c = c0 + 32 * i + lane;
      rows[i] = c < grid ? __ldcg(&p.shared[c].rows) : 0;
    }
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const uint32_t has = __ballot_sync(kFull, rows[i] > 0);
      const int nth = (int)blockIdx.x - before;
      if (cta < 0 && nth < __popc(has)) cta = c0 + 32 * i + __fns(has, 0, nth + 1);
      before += __popc(has);
    }
  }
  if (cta < 0) return;
  const Shared u = p.shared[cta];
  const int tasks = 32 * ((u.rows + 31) / 32);
  for (int w = blockIdx.y * kCombineWarps + warp; w < tasks; w += gridDim.y * kCombineWarps) {
    const int d4 = w & 31, r = (w >> 5) * 32 + lane;
    if (r >= u.rows) continue;
    // partial c: 0 is the first CTA's
    auto slot = [&](int c) { return c == 0 ? u.first : u.next + (c - 1) * u.step; };
    float M = kLowest, L = 0.f;
    bool none = false;  // a part says that the row sees keys (the L of such a part has no weight)
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = 0; b <= u.count; b += kBatch) {
      const int n = min(kBatch, u.count + 1 - b);
      float4 o[kBatch];
      float2 ml[kBatch];
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        ml[c] = make_float2(kLowest, 0.f);
        o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < n) {
          o[c] = __ldcg(reinterpret_cast<const float4 *>(p.part_o) + part_at<ROWS>(slot(b + c), r, d4));
          ml[c] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml) + (int64_t)slot(b + c) * ROWS + r);
        }
      }
      float top = M;
#pragma unroll
      for (int c = 0; c < kBatch; ++c) top = fmaxf(top, ml[c].x);
      const float back = ex2(M - top);
      M = top;
      L *= back;
      acc.x *= back;
      acc.y *= back;
      acc.z *= back;
      acc.w *= back;
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        const float f = ex2(ml[c].x - M);
        const bool empty = ml[c].y == kNoWeight;
        none = none || empty;
        L = fmaf(f, empty ? 0.f : ml[c].y, L);
        acc.x = fmaf(f, o[c].x, acc.x);
        acc.y = fmaf(f, o[c].y, acc.y);
        acc.z = fmaf(f, o[c].z, acc.z);
        acc.w = fmaf(f, o[c].w, acc.w);
      }
    }
    if (L == 0.f && none) L = kNoWeight;
    const float inv = inverse(L);
    const int64_t orow = (u.row0 + (r >> p.g_log2)) * p.hq + ((int64_t)u.h << p.g_log2) + (r & (p.g - 1));
    *reinterpret_cast<uint2 *>(p.out + orow * 128 + 4 * d4) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (p.lse != nullptr && d4 == 0) p.lse[orow] = log_sum(M, L);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
thread_local int64_t g_wait_ns = 0;  // tria_set_attention_wait_limit

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool strides_ok(int64_t tok, int64_t head) { return tok > 0 && head > 0 && tok % 8 == 0 && head % 8 == 0; }

tria_status check_desc(const tria_model_desc &d) {
  if (d.n_kv_heads < 1 || d.n_q_heads < 1 || d.n_q_heads % d.n_kv_heads != 0) return TRIA_ERR_INVALID_ARG;
  if (d.n_q_heads > 65535) return TRIA_ERR_UNSUPPORTED;
  if (d.head_dim != TRIA_HEAD_DIM) return TRIA_ERR_UNSUPPORTED;
  const int g = d.n_q_heads / d.n_kv_heads;
  if (g != 1 && g != 2 && g != 4 && g != 8 && g != 16) return TRIA_ERR_UNSUPPORTED;
  return TRIA_OK;
}

float base2(float scale) { return (float)((double)scale * 1.4426950408889634); }

// What both operators ask of the queries and the outputs.
tria_status check_rows(const void *q, int64_t q_tok, int64_t q_head, int64_t n_tokens,
                       const int32_t *starts, float scale, const void *out, const float *lse) {
  if (n_tokens < 0 || n_tokens > INT32_MAX - 1024 || !(scale > 0.f) || !std::isfinite(base2(scale))) return TRIA_ERR_INVALID_ARG;
  if (!strides_ok(q_tok, q_head) || starts == nullptr || !aligned(starts, 4)) return TRIA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (q == nullptr || out == nullptr)) return TRIA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return TRIA_ERR_INVALID_ARG;
  return TRIA_OK;
}

void fill_rows(AttendParams &p, const tria_model_desc &d, int n_seq, int64_t n_tokens, const int32_t *starts,
               float scale, void *out, float *lse, void *ws) {
  p.n_seq = n_seq;
  p.hq = d.n_q_heads;
  p.hkv = d.n_kv_heads;
  p.g = p.hq / p.hkv;
  for (p.g_log2 = 0; (1 << p.g_log2) < p.g; ++p.g_log2) {}
  p.n_tokens = n_tokens;
  p.starts = starts;
  p.qscale = base2(scale);
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.status = reinterpret_cast<int32_t *>(static_cast<unsigned char *>(ws) + 4);
  p.wait_ns = (uint64_t)g_wait_ns;
}

// q as tiles of 128 rows: 128 / G tokens x the G heads of a KV head x 64 dims
bool query_map(CUtensorMap *map, const void *q, int64_t tok, int64_t head, int hq, int g, int64_t n_tokens) {
  const uint64_t dims[4] = {128, (uint64_t)hq, (uint64_t)n_tokens, 1};
  const int64_t strides[3] = {head, tok, 0};
  const uint32_t box[4] = {64, (uint32_t)g, (uint32_t)(kRows / g), 1};
  return encode_rows_map(map, q, dims, strides, box);
}

bool cache_map(CUtensorMap *map, const void *base, const RowsView &v) {
  if (v.layout == TRIA_LAYOUT_CONTIGUOUS) {
    const uint64_t dims[4] = {128, (uint64_t)v.max_seq_len, (uint64_t)v.hkv, (uint64_t)v.n_seq};
    const int64_t strides[3] = {v.s_tok, v.s_head, v.s_seq};
    const uint32_t box[4] = {64, (uint32_t)kBN, 1, 1};
    return encode_rows_map(map, base, dims, strides, box);
  }
  const uint64_t dims[4] = {128, (uint64_t)v.hkv, (uint64_t)v.block_size, (uint64_t)v.num_blocks};
  const int64_t strides[3] = {v.s_head, v.s_tok, v.s_blk};
  const uint32_t box[4] = {64, 1, (uint32_t)v.block_size, 1};
  return encode_rows_map(map, base, dims, strides, box);
}

bool packed_map(CUtensorMap *map, const void *base, int64_t tok, int64_t head, int hkv, int64_t n_tokens) {
  const uint64_t dims[4] = {128, (uint64_t)n_tokens, (uint64_t)hkv, 1};
  const int64_t strides[3] = {tok, head, 0};
  const uint32_t box[4] = {64, (uint32_t)kBN, 1, 1};
  return encode_rows_map(map, base, dims, strides, box);
}

cudaError_t sm_count(int *sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// A launch whose blocks may start while the kernel before it in the stream ends;
// the kernels wait for that one (griddepcontrol.wait) before they touch memory.
template <class Kernel, class... Args>
cudaError_t launch_early(Kernel kernel, dim3 grid, int threads, int smem, cudaStream_t st, const Args &...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool DUALK, int LAYOUT>
cudaError_t launch_attend(const AttendParams &p, int grid, cudaStream_t st) {
  const int smem = (int)sizeof(AtSmem<DUALK>);
  static_assert(sizeof(AtSmem<DUALK>) <= kMaxDynSmem, "shared memory of the attention kernel");
  // the shared-memory opt-in once per device (it is a property of the kernel)
  static thread_local int attr_dev = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (attr_dev != dev) {
    e = cudaFuncSetAttribute(attend_kernel<DUALK, LAYOUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // The register split draws on what the block is launched with: where a compiler
    // gave the kernel another count, a group would wait for registers for good.
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, attend_kernel<DUALK, LAYOUT>)) != cudaSuccess) return e;
    if (fa.numRegs != kLaunchRegs) return cudaErrorNotSupported;
    attr_dev = dev;
  }
  return launch_early(attend_kernel<DUALK, LAYOUT>, dim3((unsigned)grid), kAtThreads, smem, st, p);
}

tria_status launch_status(cudaError_t e) {
  return e == cudaSuccess ? TRIA_OK : e == cudaErrorNotSupported ? TRIA_ERR_UNSUPPORTED : TRIA_ERR_CUDA;
}

// Tiles of rows per (sequence, KV head) at most, and rows of a partial.
struct TreeShape {
  bool dualk;
  int rows, tiles, grid, sms;
};

tria_status tree_shape(const tria_model_desc &d, const tria_cache_view *c, int max_draft, TreeShape *sh) {
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess) return TRIA_ERR_CUDA;
  const int g = d.n_q_heads / d.n_kv_heads;
  // Up to 128 rows fit one tile: its two key halves side by side, against two
  // tiles of which one is empty, took 41 us against 52 (16 tokens over 32768 rows,
  // 8 query heads per KV head) and 112 against 144 (64 paged sequences).
  sh->dualk = (int64_t)max_draft * g <= kRows;
  sh->rows = sh->dualk ? AtCfg<true>::ROWS : AtCfg<false>::ROWS;
  sh->tiles = (int)(((int64_t)max_draft * g + sh->rows - 1) / sh->rows);
  const int64_t blocks = (int64_t)c->n_seq * d.n_kv_heads * sh->tiles * ((c->max_seq_len + (int64_t)kBN - 1) / kBN);
  sh->grid = blocks < sms ? (int)blocks : sms;
  sh->sms = sms;
  return TRIA_OK;
}

size_t tree_ws_bytes(const TreeShape &sh) {
  return kHeaderBytes + (size_t)2 * sh.grid * sh.rows * (128 + 2) * sizeof(float) + (size_t)sh.grid * sizeof(Shared);
}

template <bool DUALK, int LAYOUT>
cudaError_t launch_tree(const AttendParams &p, const TreeShape &sh, cudaStream_t st) {
  const cudaError_t e = launch_attend<DUALK, LAYOUT>(p, sh.grid, st);
  if (e != cudaSuccess || sh.grid == 1) return e;
  const int64_t rows = (int64_t)p.max_draft * p.g < sh.rows ? (int64_t)p.max_draft * p.g : sh.rows;
  // a warp for 32 rows and 4 dims, as far as the blocks (four to an SM) are resident at once
  const int64_t all = (int64_t)p.n_seq * p.hkv * sh.tiles;
  const int64_t units = all < sh.grid ? all : sh.grid;  // no more shared ones than CTAs
  int64_t y = 32 * ((rows + 31) / 32) / kCombineWarps;
  const int64_t resident = 4 * (int64_t)sh.sms / units;
  if (y > resident) y = resident > 0 ? resident : 1;
  const dim3 grid((unsigned)units, (unsigned)y);
  return launch_early(combine_kernel<AtCfg<DUALK>::ROWS>, grid, 32 * kCombineWarps, 0, st, p, sh.grid);
}

}  // namespace
}  // namespace tria

using namespace tria;

extern "C" {

tria_status tria_set_attention_wait_limit(int64_t ns) {
  if (ns < 0) return TRIA_ERR_INVALID_ARG;
  g_wait_ns = ns;
  return TRIA_OK;
}

tria_status tria_prompt_workspace_size(const tria_model_desc *desc, int n_seq, size_t *bytes) {
  if (desc == nullptr || bytes == nullptr || n_seq < 1 || n_seq > TRIA_MAX_SEQS) return TRIA_ERR_INVALID_ARG;
  const tria_status st = check_desc(*desc);
  if (st != TRIA_OK) return st;
  *bytes = kHeaderBytes;
  return TRIA_OK;
}

tria_status tria_prompt_attention(const tria_model_desc *desc, const void *q, int64_t q_tok, int64_t q_head,
                                  const void *k, int64_t k_tok, int64_t k_head, const void *v, int64_t v_tok,
                                  int64_t v_head, int64_t n_tokens, const int32_t *starts, int n_seq, float scale,
                                  void *out, float *lse, void *ws, size_t ws_bytes, tria_stream_t stream) {
  if (desc == nullptr || n_seq < 1 || n_seq > TRIA_MAX_SEQS) return TRIA_ERR_INVALID_ARG;
  tria_status st = check_desc(*desc);
  if (st != TRIA_OK) return st;
  if ((st = check_rows(q, q_tok, q_head, n_tokens, starts, scale, out, lse)) != TRIA_OK) return st;
  if (!strides_ok(k_tok, k_head) || !strides_ok(v_tok, v_head) || !aligned(k, 16) || !aligned(v, 16) ||
      (n_tokens > 0 && (k == nullptr || v == nullptr)))
    return TRIA_ERR_INVALID_ARG;
  if ((st = check_header_workspace(ws, ws_bytes, kHeaderBytes)) != TRIA_OK) return st;
  if (n_tokens == 0) return TRIA_OK;
  AttendParams p{};
  fill_rows(p, *desc, n_seq, n_tokens, starts, scale, out, lse, ws);
  p.v = static_cast<const uint16_t *>(v);
  p.v_tok = v_tok;
  p.v_head = v_head;
  if (!query_map(&p.qmap, q, q_tok, q_head, p.hq, p.g, n_tokens) ||
      !packed_map(&p.kmap, k, k_tok, k_head, p.hkv, n_tokens) ||
      !packed_map(&p.vmap, v, v_tok, v_head, p.hkv, n_tokens))
    return TRIA_ERR_UNSUPPORTED;
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess) return TRIA_ERR_CUDA;
  // at most one item per tile of rows and KV head, the sequences' last tiles part full
  const int64_t tiles = (n_tokens * p.g + AtCfg<false>::ROWS - 1) / AtCfg<false>::ROWS + n_seq;
  const int grid = (int)(tiles * p.hkv < sms ? tiles * p.hkv : sms);
  return launch_status(launch_attend<false, kPacked>(p, grid, reinterpret_cast<cudaStream_t>(stream)));
}

tria_status tria_tree_workspace_size(const tria_stats *stats, const tria_cache_view *cache, int max_draft,
                                     size_t *bytes) {
  if (stats == nullptr || cache == nullptr || bytes == nullptr) return TRIA_ERR_INVALID_ARG;
  if (cache->n_seq < 1 || cache->n_seq > TRIA_MAX_SEQS || max_draft < 1 || max_draft > cache->max_seq_len)
    return TRIA_ERR_INVALID_ARG;
  tria_model_desc d;
  tria_status st = tria_stats_desc(stats, &d);
  if (st != TRIA_OK || (st = check_desc(d)) != TRIA_OK) return st;
  TreeShape sh;
  if ((st = tree_shape(d, cache, max_draft, &sh)) != TRIA_OK) return st;
  *bytes = tree_ws_bytes(sh);
  return TRIA_OK;
}

tria_status tria_tree_attention(const tria_stats *stats, const tria_cache_view *cache, int layer, const void *q,
                                int64_t q_tok, int64_t q_head, int64_t n_tokens, const int32_t *starts,
                                int max_draft, const uint32_t *mask, int mask_words, float scale, void *out,
                                float *lse, void *ws, size_t ws_bytes, tria_stream_t stream) {
  tria_model_desc d;
  AttendParams p{};
  if (layer < 0) return TRIA_ERR_INVALID_ARG;
  tria_status st = make_rows_view(stats, cache, layer, layer + 1, &d, &p.view);
  if (st != TRIA_OK) return st;
  if ((st = check_desc(d)) != TRIA_OK) return st;
  if ((st = check_rows(q, q_tok, q_head, n_tokens, starts, scale, out, lse)) != TRIA_OK) return st;
  if (max_draft < 1 || max_draft > cache->max_seq_len) return TRIA_ERR_INVALID_ARG;
  if (cache->max_seq_len > INT32_MAX - 1024) return TRIA_ERR_UNSUPPORTED;  // key indices of a block past the end
  if (mask != nullptr && (!aligned(mask, 4) || mask_words < (max_draft + 31) / 32)) return TRIA_ERR_INVALID_ARG;
  TreeShape sh;
  if ((st = tree_shape(d, cache, max_draft, &sh)) != TRIA_OK) return st;
  if ((st = check_header_workspace(ws, ws_bytes, tree_ws_bytes(sh))) != TRIA_OK) return st;
  if (n_tokens == 0) return TRIA_OK;
  fill_rows(p, d, cache->n_seq, n_tokens, starts, scale, out, lse, ws);
  p.v = static_cast<const uint16_t *>(cache->v_layers[layer]);
  p.layer = layer;
  p.max_draft = max_draft;
  p.mask = mask;
  p.mask_words = mask_words;
  p.part_o = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + kHeaderBytes);
  p.part_ml = p.part_o + (size_t)2 * sh.grid * sh.rows * 128;
  p.shared = reinterpret_cast<Shared *>(p.part_ml + (size_t)2 * sh.grid * sh.rows * 2);
  if (!query_map(&p.qmap, q, q_tok, q_head, p.hq, p.g, n_tokens) ||
      !cache_map(&p.kmap, cache->k_layers[layer], p.view) || !cache_map(&p.vmap, cache->v_layers[layer], p.view))
    return TRIA_ERR_UNSUPPORTED;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (p.view.layout == TRIA_LAYOUT_PAGED)
    e = sh.dualk ? launch_tree<true, TRIA_LAYOUT_PAGED>(p, sh, cs) : launch_tree<false, TRIA_LAYOUT_PAGED>(p, sh, cs);
  else
    e = sh.dualk ? launch_tree<true, TRIA_LAYOUT_CONTIGUOUS>(p, sh, cs)
                 : launch_tree<false, TRIA_LAYOUT_CONTIGUOUS>(p, sh, cs);
  return launch_status(e);
}

}  // extern "C"
