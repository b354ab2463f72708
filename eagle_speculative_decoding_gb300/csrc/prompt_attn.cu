// Causal attention of the packed rows of many requests over the paged cache.
//
// Source: "M7.5 - EAGLE Feature Drafting: Uncertainty, Dynamic Trees, HASS, and
// EAGLE-3", section 0x03C (the drafter's committed prefix), 0x05D (rows go to
// the cache by position).
//
// One warp per (row, query head), the lanes sharing the channels: one pass
// over the keys with a running maximum and sum.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kv4.cuh"

namespace eagle {
namespace {

struct AttnParams {
  const void* q;
  long long q_stride;
  const void *kc, *vc;     // 4-bit: the codes
  const uint8_t *ks, *vs;  // 4-bit: the scales
  float k_scale, v_scale;
  int num_pages, max_pages, B, T, Hq, Hkv;
  const int32_t *table, *cu, *ctx;
  void* out;
  float* lse;
  float scale;
  int32_t* status;
};

enum Source { kF32, kBf16, kKv4 };

template <int D, Source S>
__device__ __forceinline__ void load_row(const void* base, const uint8_t* scales, int page, int slot, int h, int Hkv,
                                         float* f) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  if (S == kKv4) {
    const size_t row = ((size_t)page * Hkv + h) * 16 + slot;
    const uint8_t* c = static_cast<const uint8_t*>(base) + row * (D / 2);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = lane + 32 * e;
      f[e] = kv4_code_value((c[ch >> 1] >> (4 * (ch & 1))) & 15u) * kv4_scale_value(scales[row * (D / 16) + ch / 16]);
    }
  } else {
    const size_t at = (((size_t)page * 16 + slot) * Hkv + h) * D + lane;
#pragma unroll
    for (int e = 0; e < E; ++e)
      f[e] = S == kF32 ? static_cast<const float*>(base)[at + 32 * e]
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at + 32 * e]);
  }
}

template <int D, Source S>
__global__ void __launch_bounds__(128) prompt_attn_kernel(const AttnParams p) {
  constexpr int E = D / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, t = blockIdx.x, h = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (h >= p.Hq) return;
  const int b = warp_find_request(p.cu, p.B, t);
  const int c0 = p.cu[b], c1 = p.cu[b + 1], ctx = p.ctx[b];
  if (t < c0 || t >= c1 || ctx < 0) {
    set_status(p.status, EAGLE_ERR_INVALID_ARG);
    return;
  }
  const int hk = h / (p.Hq / p.Hkv);
  const long long n = (long long)ctx + (t - c0) + 1;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const size_t at = (size_t)t * p.q_stride + (size_t)h * D + lane + 32 * e;
    q[e] = S == kF32 ? static_cast<const float*>(p.q)[at]
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[at]);
    o[e] = 0.f;
  }
  const float scale = p.scale * p.k_scale;
  for (long long j = 0; j < n; ++j) {
    const long long pi = j / 16;
    const int page = pi < p.max_pages ? p.table[(size_t)b * p.max_pages + pi] : -1;
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) k[e] = v[e] = 0.f;
    if (page >= 0 && page < p.num_pages) {
      load_row<D, S>(p.kc, p.ks, page, (int)(j & 15), hk, p.Hkv, k);
      load_row<D, S>(p.vc, p.vs, page, (int)(j & 15), hk, p.Hkv, v);
    } else {
      set_status(p.status, EAGLE_ERR_BAD_KV);
    }
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) z = fmaf(q[e], k[e], z);
#pragma unroll
    for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    z *= scale;
    const float mn = fmaxf(m, z), a = m == -INFINITY ? 0.f : expf(m - mn), w = z == -INFINITY ? 0.f : expf(z - mn);
    l = fmaf(l, a, w);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], a, w * v[e]);
    m = mn;
  }
  const float inv = p.v_scale / l;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const size_t at = ((size_t)t * p.Hq + h) * D + lane + 32 * e;
    if (S == kF32)
      static_cast<float*>(p.out)[at] = o[e] * inv;
    else
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(o[e] * inv);
  }
  if (p.lse && lane == 0) p.lse[(size_t)t * p.Hq + h] = m + logf(l);
}

int attn_check(const AttnParams& p, int D, int page_size, size_t es) {
  if (p.B <= 0 || p.T < 0 || p.Hq <= 0 || p.Hkv <= 0 || p.num_pages <= 0 || p.max_pages <= 0 || p.Hq % p.Hkv)
    return EAGLE_ERR_INVALID_ARG;
  if (!p.q || !p.kc || !p.vc || !p.table || !p.cu || !p.ctx || !p.out) return EAGLE_ERR_INVALID_ARG;
  if (!(p.scale > 0.f) || !isfinite(p.scale) || !(p.k_scale > 0.f) || !(p.v_scale > 0.f) || !isfinite(p.k_scale) ||
      !isfinite(p.v_scale))
    return EAGLE_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || page_size != 16 || p.Hq / p.Hkv > 64 || p.B > 65535 || p.num_pages > (1 << 26))
    return EAGLE_ERR_UNSUPPORTED;
  if (p.q_stride < (long long)p.Hq * D || p.q_stride % (long long)(16 / es)) return EAGLE_ERR_INVALID_ARG;
  if (!aligned16(p.q) || !aligned16(p.kc) || !aligned16(p.vc) || !aligned16(p.out)) return EAGLE_ERR_INVALID_ARG;
  return EAGLE_OK;
}

template <Source S>
int attn_launch(const AttnParams& p, int D, void* ws, size_t ws_bytes, void* stream) {
  if (p.T == 0) return EAGLE_OK;
  if (!ws || ws_bytes < eagle_prompt_attn_workspace_size(p.B, p.T, p.Hq, p.Hkv, D)) return EAGLE_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(p.T, (p.Hq + 3) / 4);
  if (D == 128)
    launch(prompt_attn_kernel<128, S>, grid, 128, 0, s, p);
  else
    launch(prompt_attn_kernel<64, S>, grid, 128, 0, s, p);
  note_launch();
  return last_launch_status();
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" size_t eagle_prompt_attn_workspace_size(int B, int T, int Hq, int Hkv, int D) {
  if (B <= 0 || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || (D != 64 && D != 128)) return 0;
  return 256;
}

extern "C" int eagle_prompt_attn(const void* q, long long q_stride, const void* k_cache, const void* v_cache,
                                 int num_pages, const int32_t* block_table, int max_pages, const int32_t* cu_seqlens,
                                 const int32_t* ctx_lens, void* out, float* lse, int B, int T, int Hq, int Hkv, int D,
                                 int page_size, float scale, int dtype, void* ws, size_t ws_bytes,
                                 int32_t* dev_status, void* stream) {
  if (dtype != EAGLE_BF16 && dtype != EAGLE_FP32) return EAGLE_ERR_INVALID_ARG;
  const AttnParams p = {q, q_stride, k_cache, v_cache, nullptr, nullptr, 1.f, 1.f, num_pages, max_pages, B, T, Hq, Hkv,
                        block_table, cu_seqlens, ctx_lens, out, lse, scale, dev_status};
  const int rc = attn_check(p, D, page_size, dtype == EAGLE_BF16 ? 2 : 4);
  if (rc != EAGLE_OK) return rc;
  return dtype == EAGLE_BF16 ? attn_launch<kBf16>(p, D, ws, ws_bytes, stream) : attn_launch<kF32>(p, D, ws, ws_bytes, stream);
}

extern "C" int eagle_prompt_attn_kv4(const void* q, long long q_stride, const uint8_t* k_codes,
                                     const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
                                     float k_scale, float v_scale, int num_pages, const int32_t* block_table,
                                     int max_pages, const int32_t* cu_seqlens, const int32_t* ctx_lens, void* out,
                                     float* lse, int B, int T, int Hq, int Hkv, int D, int page_size, float scale,
                                     void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  const AttnParams p = {q, q_stride, k_codes, v_codes, k_scales, v_scales, k_scale, v_scale, num_pages, max_pages, B, T,
                        Hq, Hkv, block_table, cu_seqlens, ctx_lens, out, lse, scale, dev_status};
  if (!k_scales || !v_scales) return EAGLE_ERR_INVALID_ARG;
  const int rc = attn_check(p, D, page_size, 2);
  if (rc != EAGLE_OK) return rc;
  return attn_launch<kKv4>(p, D, ws, ws_bytes, stream);
}
