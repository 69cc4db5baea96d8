// Moving cached rows: the accepted path of drafted tokens (tria_tree_commit)
// and copies of whole sequences (tria_fork_sequences).  Both move K and V rows
// of 256 bytes (and int32 positions) byte for byte, so what bounds them is HBM
// (or, for a few rows, the latency of the chain length -> path -> block table
// -> row -> store).
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "tria_device.cuh"

namespace tria {

tria_status make_rows_view(const tria_stats *stats, const tria_cache_view *c, int layer0, int layer1,
                           tria_model_desc *desc, RowsView *view) {
  if (stats == nullptr || c == nullptr) return TRIA_ERR_INVALID_ARG;
  const tria_status st = tria_stats_desc(stats, desc);
  if (st != TRIA_OK) return st;
  if (layer0 < 0 || layer1 <= layer0 || layer1 > desc->n_layers) return TRIA_ERR_INVALID_ARG;
  if (c->n_seq < 1 || c->n_seq > TRIA_MAX_SEQS || c->max_seq_len < 1) return TRIA_ERR_INVALID_ARG;
  if (c->layout != TRIA_LAYOUT_CONTIGUOUS && c->layout != TRIA_LAYOUT_PAGED) return TRIA_ERR_INVALID_ARG;
  if (c->k_layers == nullptr || c->v_layers == nullptr) return TRIA_ERR_INVALID_ARG;
  if (c->layer_seq_lens == nullptr && c->seq_lens == nullptr) return TRIA_ERR_INVALID_ARG;
  for (int l = layer0; l < layer1; ++l)
    for (const void *p : {c->k_layers[l], c->v_layers[l]})
      if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u)) return TRIA_ERR_INVALID_ARG;
  if (c->stride_head < 0 || c->stride_token <= 0 || c->stride_seq < 0 || c->stride_block < 0 ||
      (c->stride_head % 8) || (c->stride_token % 8) || (c->stride_seq % 8) || (c->stride_block % 8))
    return TRIA_ERR_INVALID_ARG;
  if (c->positions != nullptr && (reinterpret_cast<uintptr_t>(c->positions) & 3u)) return TRIA_ERR_INVALID_ARG;
  const bool paged = c->layout == TRIA_LAYOUT_PAGED;
  if (paged) {
    const int bs = c->block_size;
    if (c->block_table == nullptr || c->max_blocks_per_seq < 1 || c->num_blocks < 1 ||
        !(bs == 8 || bs == 16 || bs == 32 || bs == 64 || bs == 128) ||
        (int64_t)c->max_blocks_per_seq * bs < c->max_seq_len)
      return TRIA_ERR_INVALID_ARG;
  }
  RowsView v{};
  v.layout = c->layout;
  v.block_size = paged ? c->block_size : 1;
  while ((1 << v.block_log2) < v.block_size) ++v.block_log2;  // a power of two
  v.max_blocks = paged ? c->max_blocks_per_seq : 0;
  v.n_seq = c->n_seq;
  v.n_layers = desc->n_layers;
  v.hkv = desc->n_kv_heads;
  v.max_seq_len = c->max_seq_len;
  v.s_seq = c->stride_seq;
  v.s_head = c->stride_head;
  v.s_tok = c->stride_token;
  v.s_blk = c->stride_block;
  v.num_blocks = paged ? c->num_blocks : 0;
  v.block_table = c->block_table;
  const bool per_layer = c->layer_seq_lens != nullptr;
  v.lens = per_layer ? c->layer_seq_lens : c->seq_lens;
  v.lens_s = per_layer ? desc->n_layers : 1;
  v.lens_l = per_layer ? 1 : 0;
  v.positions = c->positions;
  *view = v;
  return TRIA_OK;
}

tria_status check_header_workspace(void *ws, size_t have, size_t need) {
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) % 256) != 0 || have < need) return TRIA_ERR_WORKSPACE;
  return TRIA_OK;
}

namespace {

using namespace dev;

constexpr int kMoveThreads = 256;
constexpr int kPieces = kHeadDim * 2 / 16;  // 16-byte pieces of a row

struct LayerPtrs {
  uint16_t *k[TRIA_MAX_LAYERS];
  uint16_t *v[TRIA_MAX_LAYERS];
};

// ---------------------------------------------------------------------------
// Accepted path: row N + accepted[j] -> row N + j, j ascending.  One block
// moves the K and V rows of one (sequence, layer), all KV heads, in chunks of
// kMoveU x 256 pieces of each: a chunk is read into registers, a barrier, written.
// In place this is safe: accepted[j] >= j, so a later chunk's sources lie
// above every destination already written, and within a chunk every read
// comes before the barrier.  The path is checked by the threads while the
// first chunk's rows are on their way (a source out of range is not read), and
// one barrier serves both.  A position moves with its row, behind the row's page
// check.  Up to 12 rows of 64 paged sequences x 32 layers x 8 KV heads (102 MB):
// 34.7 us a call in all, 27 on the GPU, bound by the chain length -> path -> page
// -> row; chunks of 32 rows and six blocks to an SM took 39 us in all against 43
// with larger ones.  4 rows of one sequence x 36 layers: 6 us.
// ---------------------------------------------------------------------------
constexpr int kMoveU = 2;
constexpr int kMoveRows = kMoveU * kMoveThreads / kPieces;  // rows of a chunk: 32
constexpr int kRowStep = kMoveThreads / kPieces;            // rows of one pass of the block: 16

struct CommitParams {
  RowsView view;
  LayerPtrs at;        // layers layer0 ..
  int layer0, nl;
  const int32_t *accepted, *n_accepted;
  int max_accept;
  int grow;            // lengths are updated by this call
  uint32_t *arrived;   // [n_seq] blocks done; the last one updates the lengths and resets it
  int32_t *status;
};

__global__ void __launch_bounds__(kMoveThreads, 6) commit_kernel(const __grid_constant__ CommitParams p) {
  const RowsView &v = p.view;
  const int s = blockIdx.x / p.nl, l = blockIdx.x % p.nl;
  const int tid = threadIdx.x, layer = p.layer0 + l, hkv = v.hkv;
  const int N = view_len(v, s, layer);
  const int n = p.n_accepted[s];
  const int32_t *acc = p.accepted + (int64_t)s * p.max_accept;
  const bool count_ok = n >= 0 && n <= p.max_accept;
  const int room = N >= 0 ? v.max_seq_len - N : 0;  // drafted slots behind the committed rows
  uint16_t *kp = p.at.k[l] + (tid % kPieces) * 8, *vp = p.at.v[l] + (tid % kPieces) * 8;
  int32_t *pos = (v.positions == nullptr || tid % kPieces != 0)
                     ? nullptr
                     : v.positions + ((int64_t)s * v.n_layers + layer) * hkv * v.max_seq_len + max(N, 0);
  const int rows = count_ok && N >= 0 ? n * hkv : 0;  // at most INT32_MAX - kMoveRows (host)
  const int step_j = kRowStep / hkv, step_h = kRowStep % hkv;
  bool path_ok = count_ok, ok = count_ok && N >= 0, bad = false;
  int last = -1;
  for (int r0 = 0; r0 == 0 || (ok && r0 < rows); r0 += kMoveRows) {
    uint4 xk[kMoveU], xv[kMoveU];
    int64_t to[kMoveU];
    int32_t xp[kMoveU];
    uint32_t moves = 0;
    const int first = r0 + tid / kPieces;
    int j = first / hkv, h = first % hkv;
#pragma unroll
    for (int u = 0; u < kMoveU; ++u) {
      if (first + u * kRowStep < rows) {
        const int a = acc[j];
        if (a > j && a < room) {  // a = j stays; anything else is no path
          int64_t from;
          if (view_row(v, s, h, N + a, &from) && view_row(v, s, h, N + j, &to[u])) {
            xk[u] = *reinterpret_cast<const uint4 *>(kp + from);
            xv[u] = *reinterpret_cast<const uint4 *>(vp + from);
            if (pos != nullptr) xp[u] = pos[(int64_t)h * v.max_seq_len + a];
            moves |= 1u << u;
          } else {
            bad = true;  // neither the rows nor the position move
          }
        }
      }
      j += step_j;
      h += step_h;
      if (h >= hkv) {
        h -= hkv;
        ++j;
      }
    }
    if (r0 == 0) {
      bool asc = count_ok;
      if (count_ok) {
        for (int i = tid; i < n; i += kMoveThreads) asc = asc && acc[i] > (i > 0 ? acc[i - 1] : -1);
        if (n > 0) last = acc[n - 1];
      }
      path_ok = __syncthreads_and(asc) != 0;
      ok = path_ok && N >= 0 && last < room;
    } else {
      __syncthreads();
    }
    if (ok) {
      j = first / hkv;
      h = first % hkv;
#pragma unroll
      for (int u = 0; u < kMoveU; ++u) {
        if ((moves >> u) & 1u) {
          *reinterpret_cast<uint4 *>(kp + to[u]) = xk[u];
          *reinterpret_cast<uint4 *>(vp + to[u]) = xv[u];
          if (pos != nullptr) pos[(int64_t)h * v.max_seq_len + j] = xp[u];
        }
        j += step_j;
        h += step_h;
        if (h >= hkv) {
          h -= hkv;
          ++j;
        }
      }
    }
  }
  if (ok ? bad : tid == 0) atomicOr(p.status, 1);
  if (!p.grow || tid >= 32) return;
  // every thread has read the length before the barrier, so this block may arrive
  int is_last = 0;
  if (tid == 0) is_last = atom_add_acq_rel(p.arrived + s, 1u) == (uint32_t)(p.nl - 1) ? 1 : 0;
  if (!__shfl_sync(kFull, is_last, 0)) return;
  if (tid == 0) p.arrived[s] = 0u;
  if (!path_ok) return;
  if (v.lens_l == 0) {
    if (tid == 0 && ok) v.lens[s] = N + n;
  } else {
    for (int i = tid; i < p.nl; i += 32) {
      const int len = view_len(v, s, p.layer0 + i);
      if (len >= 0 && last < v.max_seq_len - len) v.lens[(int64_t)s * v.lens_s + p.layer0 + i] = len + n;
    }
  }
}

// ---------------------------------------------------------------------------
// Forks.  The destinations of one source form a group, so a source row is read
// once and written to (up to kForkDst at a time) destinations.  One block
// copies kForkRows slots of the K or V rows of one (group, layer), all KV
// heads; slots whose block a destination shares are skipped for it.  Two private
// copies of each of two sequences, 32 layers (2.02 GB): 330 us, 6.1 TB/s (HBM);
// three children that share all but the last block (12 MB): 14 us (latency).
// ---------------------------------------------------------------------------
constexpr int kForkRows = 64;
constexpr int kForkDst = 4;
constexpr int kForkU = 8;                   // 16-byte loads in flight per thread
constexpr int kForkBlocks = kForkRows / 8;  // paged blocks of a chunk, at most

struct ForkParams {
  RowsView view;
  LayerPtrs at;
  int layer0, nl;
  int write_len;
  int32_t *status;
  uint16_t src[TRIA_MAX_SEQS];        // source of each group
  uint16_t first[TRIA_MAX_SEQS + 1];  // the group's destinations: dst[first[g] .. first[g + 1])
  uint16_t dst[TRIA_MAX_SEQS];
};

__global__ void __launch_bounds__(kMoveThreads) fork_kernel(const __grid_constant__ ForkParams p) {
  const RowsView &v = p.view;
  const int g = blockIdx.z, l = blockIdx.y >> 1, is_v = blockIdx.y & 1, tid = threadIdx.x;
  const int layer = p.layer0 + l, s = p.src[g];
  const int d0 = p.first[g], d1 = p.first[g + 1];
  const int N = view_len(v, s, layer);
  if (N < 0) {
    if (tid == 0) atomicOr(p.status, 1);
    return;
  }
  if (blockIdx.x == 0 && !is_v && p.write_len && (v.lens_l != 0 || l == 0))
    for (int d = d0 + tid; d < d1; d += kMoveThreads)
      v.lens[(int64_t)p.dst[d] * v.lens_s + (int64_t)layer * v.lens_l] = N;
  const int t0 = blockIdx.x * kForkRows;
  if (t0 >= N) return;
  const int nt = min(kForkRows, N - t0);
  uint16_t *base = is_v ? p.at.v[l] : p.at.k[l];
  const bool paged = v.layout == TRIA_LAYOUT_PAGED;
  const int bs = v.block_size, bs_log2 = v.block_log2;
  const int b0 = paged ? t0 >> bs_log2 : 0, nb = paged ? ((t0 + nt - 1) >> bs_log2) - b0 + 1 : 1;
  __shared__ int64_t s_from[kForkBlocks], s_to[kForkDst][kForkBlocks];
  __shared__ uint32_t s_need[kForkBlocks], s_has[kForkBlocks];
  for (int d = d0; d < d1; d += kForkDst) {
    const int nd = min(kForkDst, d1 - d);
    __syncthreads();
    if (tid < nb) {
      // where block b0 + tid of the source and of each destination begins,
      // which destinations need a copy of it, and which have the rows afterwards
      uint32_t need = 0, has = 0;
      if (!paged) {
        s_from[0] = (int64_t)s * v.s_seq;
        for (int i = 0; i < nd; ++i) s_to[i][0] = (int64_t)p.dst[d + i] * v.s_seq;
        need = has = (1u << nd) - 1u;
      } else {
        const int sb = v.block_table[(int64_t)s * v.max_blocks + b0 + tid];
        const bool s_ok = sb >= 0 && sb < v.num_blocks;
        bool bad = !s_ok;
        s_from[tid] = (int64_t)sb * v.s_blk;
        for (int i = 0; i < nd; ++i) {
          const int db = v.block_table[(int64_t)p.dst[d + i] * v.max_blocks + b0 + tid];
          const bool d_ok = db >= 0 && db < v.num_blocks;
          s_to[i][tid] = (int64_t)db * v.s_blk;
          bad = bad || !d_ok;
          if (s_ok && d_ok) has |= 1u << i;
          if (s_ok && d_ok && db != sb) need |= 1u << i;
        }
        if (bad) atomicOr(p.status, 1);
      }
      s_need[tid] = need;
      s_has[tid] = has;
    }
    // nothing to copy where every destination shares the chunk's blocks
    const bool any = __syncthreads_or(tid < nb && s_need[tid] != 0) != 0;
    const int t = tid % kForkRows;
    if (!is_v && v.positions != nullptr && t < nt) {
      // a position goes with its row, that of a shared block included
      const uint32_t to = s_has[paged ? ((t0 + t) >> bs_log2) - b0 : 0];
      const int64_t unit = (int64_t)v.hkv * v.max_seq_len;
      int32_t *pos = v.positions + (int64_t)layer * unit + t0 + t;
      for (int h = tid / kForkRows; h < v.hkv; h += kMoveThreads / kForkRows) {
        int32_t *at = pos + (int64_t)h * v.max_seq_len;
        const int32_t x = at[(int64_t)s * v.n_layers * unit];
        for (int k = 0; k < nd; ++k)
          if ((to >> k) & 1u) at[(int64_t)p.dst[d + k] * v.n_layers * unit] = x;
      }
    }
    if (!any) continue;
    const int pieces = nt * v.hkv * kPieces;  // at most 64 x hkv x 16, 32 bits (host)
    for (int i0 = tid; i0 < pieces; i0 += kForkU * kMoveThreads) {
      uint4 x[kForkU];
      int64_t off[kForkU];
      uint32_t meta[kForkU];  // block of the chunk, and the destinations
#pragma unroll
      for (int u = 0; u < kForkU; ++u) {
        const int i = i0 + u * kMoveThreads;
        meta[u] = 0;
        if (i < pieces) {
          const int row = i / kPieces, t = row / v.hkv, h = row - t * v.hkv;
          const int b = paged ? ((t0 + t) >> bs_log2) - b0 : 0;
          const int in = paged ? (t0 + t) & (bs - 1) : t0 + t;
          const uint32_t need = s_need[b];
          off[u] = (int64_t)h * v.s_head + (int64_t)in * v.s_tok + (i % kPieces) * 8;
          meta[u] = need | ((uint32_t)b << 8);
          if (need) x[u] = __ldcs(reinterpret_cast<const uint4 *>(base + s_from[b] + off[u]));
        }
      }
#pragma unroll
      for (int u = 0; u < kForkU; ++u)
#pragma unroll
        for (int k = 0; k < kForkDst; ++k)
          if ((meta[u] >> k) & 1u)
            *reinterpret_cast<uint4 *>(base + s_to[k][meta[u] >> 8] + off[u]) = x[u];
    }
  }
}

void layer_ptrs(const tria_cache_view *c, int layer0, int layer1, LayerPtrs *at) {
  for (int l = layer0; l < layer1; ++l) {
    at->k[l - layer0] = static_cast<uint16_t *>(c->k_layers[l]);
    at->v[l - layer0] = static_cast<uint16_t *>(c->v_layers[l]);
  }
}

size_t commit_ws_bytes(const tria_cache_view *c) {
  return kHeaderBytes + ((size_t)c->n_seq * 4 + 255) / 256 * 256;
}

int32_t *status_of(void *ws) { return reinterpret_cast<int32_t *>(static_cast<unsigned char *>(ws) + 4); }

// lengths move with the call over the last layer, or with their own layer
bool moves_lens(const RowsView &v, int layer1) { return v.lens_l != 0 || layer1 == v.n_layers; }

}  // namespace
}  // namespace tria

using namespace tria;

extern "C" {

tria_status tria_commit_workspace_size(const tria_stats *stats, const tria_cache_view *cache, size_t *bytes) {
  if (stats == nullptr || cache == nullptr || bytes == nullptr) return TRIA_ERR_INVALID_ARG;
  if (cache->n_seq < 1 || cache->n_seq > TRIA_MAX_SEQS) return TRIA_ERR_INVALID_ARG;
  *bytes = commit_ws_bytes(cache);
  return TRIA_OK;
}

tria_status tria_tree_commit(const tria_stats *stats, const tria_cache_view *cache,
                             const int32_t *accepted, const int32_t *n_accepted, int max_accept,
                             int layer0, int layer1, void *ws, size_t ws_bytes, tria_stream_t stream) {
  tria_model_desc d;
  CommitParams p{};
  const tria_status st = make_rows_view(stats, cache, layer0, layer1, &d, &p.view);
  if (st != TRIA_OK) return st;
  if (accepted == nullptr || n_accepted == nullptr || max_accept < 1 ||
      (reinterpret_cast<uintptr_t>(accepted) & 3u) || (reinterpret_cast<uintptr_t>(n_accepted) & 3u))
    return TRIA_ERR_INVALID_ARG;
  // the kernel counts rows of 32 bits
  if ((int64_t)max_accept * d.n_kv_heads > INT32_MAX - kMoveRows) return TRIA_ERR_UNSUPPORTED;
  const tria_status sw = check_header_workspace(ws, ws_bytes, commit_ws_bytes(cache));
  if (sw != TRIA_OK) return sw;
  layer_ptrs(cache, layer0, layer1, &p.at);
  p.layer0 = layer0;
  p.nl = layer1 - layer0;
  p.accepted = accepted;
  p.n_accepted = n_accepted;
  p.max_accept = max_accept;
  p.grow = moves_lens(p.view, layer1) ? 1 : 0;
  p.arrived = reinterpret_cast<uint32_t *>(static_cast<unsigned char *>(ws) + kHeaderBytes);
  p.status = status_of(ws);
  const unsigned blocks = (unsigned)cache->n_seq * (unsigned)p.nl;
  commit_kernel<<<blocks, kMoveThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? TRIA_OK : TRIA_ERR_CUDA;
}

tria_status tria_fork_workspace_size(const tria_stats *stats, const tria_cache_view *cache, size_t *bytes) {
  if (stats == nullptr || cache == nullptr || bytes == nullptr) return TRIA_ERR_INVALID_ARG;
  *bytes = kHeaderBytes;
  return TRIA_OK;
}

tria_status tria_fork_sequences(const tria_stats *stats, const tria_cache_view *cache, const int32_t *src,
                                const int32_t *dst, int n_fork, int layer0, int layer1, void *ws,
                                size_t ws_bytes, tria_stream_t stream) {
  tria_model_desc d;
  ForkParams p;
  std::memset(&p, 0, sizeof(p));
  const tria_status st = make_rows_view(stats, cache, layer0, layer1, &d, &p.view);
  if (st != TRIA_OK) return st;
  // the kernel counts pieces of 32 bits
  if (d.n_kv_heads > (INT32_MAX - kForkU * kMoveThreads) / (kForkRows * kPieces)) return TRIA_ERR_UNSUPPORTED;
  if (n_fork < 0 || n_fork > TRIA_MAX_SEQS || (n_fork > 0 && (src == nullptr || dst == nullptr)))
    return TRIA_ERR_INVALID_ARG;
  uint16_t count[TRIA_MAX_SEQS] = {};  // destinations of each source
  bool is_dst[TRIA_MAX_SEQS] = {};
  for (int i = 0; i < n_fork; ++i) {
    if (src[i] < 0 || src[i] >= cache->n_seq || dst[i] < 0 || dst[i] >= cache->n_seq || is_dst[dst[i]])
      return TRIA_ERR_INVALID_ARG;
    is_dst[dst[i]] = true;
    ++count[src[i]];
  }
  int groups = 0, filled = 0;
  uint16_t at[TRIA_MAX_SEQS];  // next free place of each source's group
  for (int s = 0; s < cache->n_seq; ++s) {
    if (count[s] == 0) continue;
    if (is_dst[s]) return TRIA_ERR_INVALID_ARG;
    p.src[groups] = (uint16_t)s;
    p.first[groups++] = at[s] = (uint16_t)filled;
    filled += count[s];
  }
  p.first[groups] = (uint16_t)filled;
  for (int i = 0; i < n_fork; ++i) p.dst[at[src[i]]++] = (uint16_t)dst[i];
  const tria_status sw = check_header_workspace(ws, ws_bytes, kHeaderBytes);
  if (sw != TRIA_OK) return sw;
  if (n_fork == 0) return TRIA_OK;
  layer_ptrs(cache, layer0, layer1, &p.at);
  p.layer0 = layer0;
  p.nl = layer1 - layer0;
  p.write_len = moves_lens(p.view, layer1) ? 1 : 0;
  p.status = status_of(ws);
  const dim3 grid((unsigned)((cache->max_seq_len + (int64_t)kForkRows - 1) / kForkRows), 2u * p.nl,
                  (unsigned)groups);
  fork_kernel<<<grid, kMoveThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? TRIA_OK : TRIA_ERR_CUDA;
}

}  // extern "C"
