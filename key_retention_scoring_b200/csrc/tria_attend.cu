// Attention of many query rows at once: whole prompts, causal, packed
// (tria_prompt_attention), and drafted tokens over the cached rows of a layer
// (tria_tree_attention).
//
// Query row i (token i of sequence s, query head qh, KV head h = qh / G) sees
// the keys j < ctx + T of its sequence for which
//   j < ctx, or j - ctx <= i (a chain), or bit j - ctx of its mask is set
// (prompts: ctx = 0, T = the sequence's length):
//   out_i = sum_j softmax(scale q_i.k_j)_j v_j,  lse_i = log sum_j exp(scale q_i.k_j).
//
// One warp per (token, query head), a key after the other with a running
// maximum and sum; each lane holds 4 of the 128 dims.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "tria_device.cuh"

namespace tria {
namespace {

using namespace dev;

constexpr int kWarps = 8;

struct AttendParams {
  const uint16_t *q, *k, *v;
  int64_t q_tok, q_head;
  int64_t k_tok, k_head, v_tok, v_head;  // packed rows
  RowsView view;                         // cached rows
  int layer;
  int cached;
  const int32_t *starts;
  int n_seq, hq, hkv, g;
  int64_t n_tokens;
  int max_draft;
  const uint32_t *mask;
  int mask_words;
  float scale;
  uint16_t *out;
  float *lse;
  int32_t *status;
};

__device__ __forceinline__ float4 row4(const uint16_t *p, int lane) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p + 4 * lane);
  return make_float4(bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y));
}

__global__ void __launch_bounds__(32 * kWarps) attend_kernel(const __grid_constant__ AttendParams p) {
  const int s = blockIdx.y, qh = blockIdx.z, h = qh / p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t a = p.starts[s], b = p.starts[s + 1];
  bool ok = a >= 0 && b >= a && b <= p.n_tokens;
  int ctx = 0;
  if (ok && b > a && p.cached) {
    ctx = view_len(p.view, s, p.layer);
    ok = ctx >= 0 && b - a <= p.max_draft && b - a <= p.view.max_seq_len - ctx;
  }
  if (!ok) {
    if (threadIdx.x == 0) atomicOr(p.status, 1);
    return;
  }
  const int T = (int)(b - a);
  for (int i = blockIdx.x * kWarps + warp; i < T; i += gridDim.x * kWarps) {
    const float4 q = row4(p.q + (a + i) * p.q_tok + (int64_t)qh * p.q_head, lane);
    const uint32_t *bits = p.mask ? p.mask + (a + i) * p.mask_words : nullptr;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const int n = ctx + (bits ? T : i + 1);
    for (int j = 0; j < n; ++j) {
      if (bits && j >= ctx && !((bits[(j - ctx) >> 5] >> ((j - ctx) & 31)) & 1u)) continue;
      float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
      if (p.cached) {
        int64_t off;
        if (view_row(p.view, s, h, j, &off)) {
          k = row4(p.k + off, lane);
          v = row4(p.v + off, lane);
        }
      } else {
        k = row4(p.k + (a + j) * p.k_tok + (int64_t)h * p.k_head, lane);
        v = row4(p.v + (a + j) * p.v_tok + (int64_t)h * p.v_head, lane);
      }
      float z = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, q.w * k.w)));
#pragma unroll
      for (int x = 16; x >= 1; x >>= 1) z += __shfl_xor_sync(kFull, z, x);
      z *= p.scale;
      const float mn = fmaxf(m, z), f = expf(m - mn), e = expf(z - mn);
      l = fmaf(l, f, e);
      o.x = fmaf(o.x, f, e * v.x);
      o.y = fmaf(o.y, f, e * v.y);
      o.z = fmaf(o.z, f, e * v.z);
      o.w = fmaf(o.w, f, e * v.w);
      m = mn;
    }
    const float inv = n > 0 && l != 0.f ? 1.f / l : 0.f;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t *>(&lo);
    w.y = *reinterpret_cast<const uint32_t *>(&hi);
    *reinterpret_cast<uint2 *>(p.out + ((a + i) * p.hq + qh) * 128 + 4 * lane) = w;
    if (p.lse != nullptr && lane == 0) p.lse[(a + i) * p.hq + qh] = m + logf(l);
  }
}

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

// What both operators ask of the queries and the outputs.
tria_status check_rows(const void *q, int64_t q_tok, int64_t q_head, int64_t n_tokens,
                       const int32_t *starts, float scale, const void *out, const float *lse) {
  if (n_tokens < 0 || n_tokens > INT32_MAX || !std::isfinite(scale) || !(scale > 0.f)) return TRIA_ERR_INVALID_ARG;
  if (!strides_ok(q_tok, q_head) || starts == nullptr || !aligned(starts, 4)) return TRIA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (q == nullptr || out == nullptr)) return TRIA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return TRIA_ERR_INVALID_ARG;
  return TRIA_OK;
}

tria_status launch_attend(const AttendParams &p, int64_t max_tokens, cudaStream_t st) {
  int64_t x = (max_tokens + kWarps - 1) / kWarps;
  if (x > 2048) x = 2048;
  attend_kernel<<<dim3((unsigned)x, (unsigned)p.n_seq, (unsigned)p.hq), 32 * kWarps, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? TRIA_OK : TRIA_ERR_CUDA;
}

}  // namespace
}  // namespace tria

using namespace tria;

extern "C" {

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
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.q_tok = q_tok;
  p.q_head = q_head;
  p.k_tok = k_tok;
  p.k_head = k_head;
  p.v_tok = v_tok;
  p.v_head = v_head;
  p.starts = starts;
  p.n_seq = n_seq;
  p.hq = desc->n_q_heads;
  p.hkv = desc->n_kv_heads;
  p.g = p.hq / p.hkv;
  p.n_tokens = n_tokens;
  p.scale = scale;
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.status = reinterpret_cast<int32_t *>(static_cast<unsigned char *>(ws) + 4);
  return launch_attend(p, n_tokens, reinterpret_cast<cudaStream_t>(stream));
}

tria_status tria_tree_workspace_size(const tria_stats *stats, const tria_cache_view *cache, int max_draft,
                                     size_t *bytes) {
  if (stats == nullptr || cache == nullptr || bytes == nullptr) return TRIA_ERR_INVALID_ARG;
  if (cache->n_seq < 1 || cache->n_seq > TRIA_MAX_SEQS || max_draft < 1 || max_draft > cache->max_seq_len)
    return TRIA_ERR_INVALID_ARG;
  *bytes = kHeaderBytes;
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
  if (mask != nullptr && (!aligned(mask, 4) || mask_words < (max_draft + 31) / 32)) return TRIA_ERR_INVALID_ARG;
  if ((st = check_header_workspace(ws, ws_bytes, kHeaderBytes)) != TRIA_OK) return st;
  if (n_tokens == 0) return TRIA_OK;
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(cache->k_layers[layer]);
  p.v = static_cast<const uint16_t *>(cache->v_layers[layer]);
  p.q_tok = q_tok;
  p.q_head = q_head;
  p.layer = layer;
  p.cached = 1;
  p.starts = starts;
  p.n_seq = cache->n_seq;
  p.hq = d.n_q_heads;
  p.hkv = d.n_kv_heads;
  p.g = p.hq / p.hkv;
  p.n_tokens = n_tokens;
  p.max_draft = max_draft;
  p.mask = mask;
  p.mask_words = mask_words;
  p.scale = scale;
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.status = reinterpret_cast<int32_t *>(static_cast<unsigned char *>(ws) + 4);
  return launch_attend(p, max_draft, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
