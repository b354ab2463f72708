// Appending the packed rows of many requests to the paged cache, rotated to
// their positions on the way, into 16- or 32-bit pages or into 4-bit pages.
//
// Source: "M7.5 - EAGLE Feature Drafting: Uncertainty, Dynamic Trees, HASS, and
// EAGLE-3", section 0x03C (the drafter keeps its own K/V of the committed
// prefix) and section 0x05D "Feature And KV Commit" (rows go to the cache by
// position; the new frontier token needs a later target append).
//
// The work is a copy: each q, k and v element is read once and written once,
// beside D fp32 of the rotation table per row (which the row's heads share
// through L1).  An item is a 16-byte vector of the first half of a head and
// its partner vector of the second half, so that a thread holds both
// channels of every pair it turns; v items are moved the same way, unturned.
// A CTA takes `tpc` whole rows (one for ordinary head counts, more for few
// heads, so that no thread idles).  Its loads of q, k and v do not depend on
// the row's request, so they are in flight while a warp looks up the request,
// the position and the page.
// Bound by HBM for many rows: 9061 rows of 32 + 2 x 8 heads, D 128, bf16: 40 us,
// 5.6 TB/s; 8125 rows into 4-bit pages, whose elements take a division and a
// conversion as well: 45 us in the kernel (bound by its latencies: with a plain
// multiplication for the division it takes as long).  One row of each of 64 requests is
// bound by the launch: 3.6 us in a graph.  Reading 4-bit pages back
// (eagle_kv4_read): 8.2 us for one cache of these rows.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kv4.cuh"

namespace eagle {
namespace {

constexpr int kThreads = 128;
// items a thread has in flight: 3 hold fewer registers than 4 (9061 rows of 32 +
// 2 x 8 heads: 40 us, 44 us; of 64 + 2 x 8: 63, 70; of 16 + 2 x 2: 19, 19), with 2
// the rows take another round of loads (43, 63, 23)
constexpr int kUnroll = 3;
constexpr int kMaxRows = 64;  // rows per CTA

struct AppendParams {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements from row to row
  const float* rope;                       // [max_pos, 2, D/2] or null
  int max_pos;
  const int32_t *cu, *ctx, *table;
  int B, T, Hq, Hkv, num_pages, max_pages, tpc;
  void *q_out, *kc, *vc;  // 4-bit: kc, vc are the codes
  uint8_t *ks, *vs;       // 4-bit: the scales
  float k_inv, v_inv;     // 4-bit: 1 / k_scale, 1 / v_scale
  int32_t* status;
};

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
};
__device__ __forceinline__ void unpack(const uint4& u, float* f, const __nv_bfloat16*) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& u, float* f, const float*) {
  f[0] = __uint_as_float(u.x);
  f[1] = __uint_as_float(u.y);
  f[2] = __uint_as_float(u.z);
  f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 pack(const float* f, const __nv_bfloat16*) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float* f, const float*) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// 4-bit rows: 8 channels per vector, 16 channels (this lane's vector and its
// neighbour's) share a scale.  Every lane of the warp calls this.
__device__ __forceinline__ void store4(const float* x, float inv, bool live, uint8_t* codes, uint8_t* scales, int vec) {
  float y[8], a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = __fmul_rn(x[i], inv);
    a = fmax_nan(a, fabsf(y[i]));
  }
  a = fmax_nan(a, __shfl_xor_sync(0xffffffffu, a, 1));
  const uint8_t sb = kv4_scale(a);
  const uint32_t w = kv4_codes(y, kv4_scale_value(sb));
  if (!live) return;
  *reinterpret_cast<uint32_t*>(codes + vec * 4) = w;
  if ((vec & 1) == 0) scales[vec >> 1] = sb;
}

template <typename T, int D, bool KV4>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p) {
  constexpr int kV = Vec<T>::N, kHalf = D / 2, kVph = kHalf / kV;  // vectors per half head
  __shared__ int s_pos[kMaxRows], s_dst[kMaxRows];  // position (-1: skip), cache row (-1: none)
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * p.tpc, rows = min(p.tpc, p.T - t0);
  const int per_row = (p.Hq + 2 * p.Hkv) * kVph, items = rows * per_row;
  const int lane = threadIdx.x & 31;
  const T* tag = nullptr;

  uint4 a[kUnroll], b[kUnroll];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int it = base + u * kThreads + threadIdx.x;
      a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
      if (it >= items) continue;
      const int r = it / per_row, h = (it % per_row) / kVph, i0 = (it % kVph) * kV;
      const size_t t = (size_t)(t0 + r);
      const T* src;
      if (h < p.Hq)
        src = static_cast<const T*>(p.q) + t * p.q_stride + (size_t)h * D;
      else if (h < p.Hq + p.Hkv)
        src = static_cast<const T*>(p.k) + t * p.k_stride + (size_t)(h - p.Hq) * D;
      else
        src = static_cast<const T*>(p.v) + t * p.v_stride + (size_t)(h - p.Hq - p.Hkv) * D;
      a[u] = *reinterpret_cast<const uint4*>(src + i0);
      b[u] = *reinterpret_cast<const uint4*>(src + i0 + kHalf);
    }
  };
  load(0);

  for (int r = threadIdx.x >> 5; r < rows; r += kThreads / 32) {
    const int t = t0 + r;
    const int bq = warp_find_request(p.cu, p.B, t);
    if (lane == 0) {
      const int c0 = p.cu[bq], c1 = p.cu[bq + 1], ctx = p.ctx[bq];
      const long long pos = (long long)ctx + (t - c0);
      int dst = -1, at = -1;
      if (t < c0 || t >= c1 || ctx < 0 || pos > 0x7fffffff || (p.rope && pos >= p.max_pos)) {
        set_status(p.status, EAGLE_ERR_INVALID_ARG);
      } else {
        at = (int)pos;
        const int page = at / 16 < p.max_pages ? p.table[(size_t)bq * p.max_pages + at / 16] : -1;
        if (page < 0 || page >= p.num_pages)
          set_status(p.status, EAGLE_ERR_BAD_KV);
        else
          dst = page * 16 + at % 16;
      }
      s_pos[r] = at;
      s_dst[r] = dst;
    }
  }
  __syncthreads();

  for (int base = 0; base < items; base += kUnroll * kThreads) {
    if (base) load(base);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int it = base + u * kThreads + threadIdx.x;
      const bool in = it < items;
      const int r = in ? it / per_row : 0, rem = it % per_row;
      const int h = rem / kVph, vec = rem % kVph, i0 = vec * kV;
      const int pos = s_pos[r], dst = s_dst[r];
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
      float x1[kV], x2[kV];
      unpack(a[u], x1, tag);
      unpack(b[u], x2, tag);
      if (!is_v && p.rope && in && pos >= 0) {
        const float4* cs = reinterpret_cast<const float4*>(p.rope + (size_t)pos * D + i0);
        const float4* sn = reinterpret_cast<const float4*>(p.rope + (size_t)pos * D + kHalf + i0);
#pragma unroll
        for (int j = 0; j < kV / 4; ++j) {
          const float4 c4 = cs[j], s4 = sn[j];
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // rounded one by one: the 4-bit codes are then those of the
            // same three operations anywhere
            const float y1 = x1[4 * j + e], y2 = x2[4 * j + e];
            x1[4 * j + e] = __fsub_rn(__fmul_rn(y1, c[e]), __fmul_rn(y2, s[e]));
            x2[4 * j + e] = __fadd_rn(__fmul_rn(y2, c[e]), __fmul_rn(y1, s[e]));
          }
        }
      }
      if (is_q && in && pos >= 0) {
        T* o = static_cast<T*>(p.q_out) + ((size_t)(t0 + r) * p.Hq + h) * D + i0;
        *reinterpret_cast<uint4*>(o) = pack(x1, tag);
        *reinterpret_cast<uint4*>(o + kHalf) = pack(x2, tag);
      }
      const int hk = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
      if constexpr (KV4) {
        // whole warps take part in the neighbours' exchange
        const bool live = in && !is_q && dst >= 0;
        const size_t row = live ? ((size_t)(dst >> 4) * p.Hkv + hk) * 16 + (dst & 15) : 0;
        uint8_t* codes = static_cast<uint8_t*>(is_v ? p.vc : p.kc) + row * (D / 2);
        uint8_t* scales = (is_v ? p.vs : p.ks) + row * (D / 16);
        const float inv = is_v ? p.v_inv : p.k_inv;
        if (__any_sync(0xffffffffu, live)) {
          store4(x1, inv, live, codes, scales, vec);
          store4(x2, inv, live, codes, scales, vec + kVph);
        }
      } else if (in && !is_q && dst >= 0) {
        T* o = static_cast<T*>(is_v ? p.vc : p.kc) + ((size_t)dst * p.Hkv + hk) * D + i0;
        *reinterpret_cast<uint4*>(o) = pack(x1, tag);
        *reinterpret_cast<uint4*>(o + kHalf) = pack(x2, tag);
      }
    }
  }
}

// cos and sin of pos * theta^(-2i/D): the angle in fp64 (the far positions of
// the fast pairs would lose their fraction in fp32), its sine and cosine too.
__global__ void __launch_bounds__(256) rope_table_kernel(int max_pos, int half, double theta, float* table) {
  pdl_wait();
  pdl_trigger();
  const long long n = (long long)max_pos * half;
  for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < n; t += (long long)gridDim.x * 256) {
    const int i = (int)(t % half);
    const long long pos = t / half;
    double s, c;
    sincos((double)pos * pow(theta, -(double)i / (double)half), &s, &c);
    table[pos * 2 * half + i] = (float)c;
    table[pos * 2 * half + half + i] = (float)s;
  }
}

// 16 channels (8 code bytes, one scale byte) per thread; a warp reads 256
// contiguous code bytes and writes whole rows of the token-major layout.  A CTA
// takes `ppc` whole pages, so that the places are 32-bit divisions within them
// (with 64-bit quotients per thread 9.4 us, now 8.2 us, for the
// 566 pages of 8 heads, D 128, of 8125 rows).
template <typename T>
__global__ void __launch_bounds__(256)
    kv4_read_kernel(const uint2* __restrict__ codes, const uint8_t* __restrict__ scales, float scale, int Hkv, int D,
                    int num_pages, int ppc, T* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int gpr = D / 16, per_page = Hkv * 16 * gpr;  // groups per row and page
  const T* tag = nullptr;
  for (int p0 = blockIdx.x * ppc; p0 < num_pages; p0 += gridDim.x * ppc) {
    const int n = min(ppc, num_pages - p0) * per_page;
    const size_t g0 = (size_t)p0 * per_page;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += 256) {
      const uint2 c = codes[g0 + i];
      const float s = kv4_scale_value(scales[g0 + i]);
      const int row = i / gpr, slot = row & 15, ph = row >> 4, page = ph / Hkv, h = ph - page * Hkv;
      T* o = out + (((size_t)(p0 + page) * 16 + slot) * Hkv + h) * D + (i - row * gpr) * 16;
      float f[16];
      kv4_values(c.x, f);
      kv4_values(c.y, f + 8);
#pragma unroll
      for (int x = 0; x < 16; ++x) f[x] = __fmul_rn(__fmul_rn(f[x], s), scale);
      constexpr int kV = Vec<T>::N;
#pragma unroll
      for (int x = 0; x < 16; x += kV) *reinterpret_cast<uint4*>(o + x) = pack(f + x, tag);
    }
  }
}

int append_check(const AppendParams& p, int D, size_t es) {
  if (p.B <= 0 || p.T < 0 || p.Hq < 0 || p.Hkv <= 0 || p.num_pages <= 0 || p.max_pages <= 0)
    return EAGLE_ERR_INVALID_ARG;
  if (!p.kc || !p.vc || !p.cu || !p.ctx || !p.table) return EAGLE_ERR_INVALID_ARG;
  // (arrays of no rows may have no address)
  if (p.T > 0 && (!p.k || !p.v || (p.Hq > 0) != (p.q != nullptr) || (p.Hq > 0) != (p.q_out != nullptr)))
    return EAGLE_ERR_INVALID_ARG;
  if (p.rope && p.max_pos <= 0) return EAGLE_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || (long long)p.Hq + 2ll * p.Hkv > 1024 || p.num_pages > (1 << 26))
    return EAGLE_ERR_UNSUPPORTED;
  const long long ev = (long long)(16 / es);
  if (p.k_stride < (long long)p.Hkv * D || p.v_stride < (long long)p.Hkv * D || p.k_stride % ev || p.v_stride % ev ||
      (p.Hq > 0 && (p.q_stride < (long long)p.Hq * D || p.q_stride % ev)))
    return EAGLE_ERR_INVALID_ARG;
  // a row of q_out is written by the CTA that read the same row of q
  if (p.q && p.q == p.q_out && p.q_stride != (long long)p.Hq * D) return EAGLE_ERR_INVALID_ARG;
  if (!aligned16(p.q) || !aligned16(p.k) || !aligned16(p.v) || !aligned16(p.rope) || !aligned16(p.q_out) ||
      !aligned16(p.kc) || !aligned16(p.vc))
    return EAGLE_ERR_INVALID_ARG;
  return EAGLE_OK;
}

template <typename T, bool KV4>
int append_launch(AppendParams p, int D, void* stream) {
  if (p.T == 0) return EAGLE_OK;
  const int per_row = (p.Hq + 2 * p.Hkv) * (D / 2 / Vec<T>::N);
  // whole rows per CTA: one when its items fill the threads, else as many as
  // give every thread its unrolled share
  p.tpc = std::max(1, std::min(kMaxRows, kThreads * kUnroll / per_row));
  const int grid = (p.T + p.tpc - 1) / p.tpc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (D == 128)
    launch(kv_append_kernel<T, 128, KV4>, grid, kThreads, 0, s, p);
  else
    launch(kv_append_kernel<T, 64, KV4>, grid, kThreads, 0, s, p);
  note_launch();
  return last_launch_status();
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" int eagle_rope_table(int max_pos, int D, double theta, float* table, void* stream) {
  if (max_pos <= 0 || !table || !(theta > 0.0) || !isfinite(theta) || !aligned16(table)) return EAGLE_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return EAGLE_ERR_UNSUPPORTED;
  const long long n = (long long)max_pos * (D / 2);
  const int grid = (int)std::min<long long>((n + 255) / 256, 8ll * std::max(1, sm_count()));
  launch(rope_table_kernel, grid, 256, 0, static_cast<cudaStream_t>(stream), max_pos, D / 2, theta, table);
  note_launch();
  return last_launch_status();
}

extern "C" int eagle_kv_append(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                               long long v_stride, const float* rope, int max_pos, const int32_t* cu_seqlens,
                               const int32_t* ctx_lens, int B, int T, int Hq, int Hkv, int D, int dtype, void* q_out,
                               void* k_cache, void* v_cache, int num_pages, const int32_t* block_table, int max_pages,
                               int32_t* dev_status, void* stream) {
  if (dtype != EAGLE_BF16 && dtype != EAGLE_FP32) return EAGLE_ERR_INVALID_ARG;
  const AppendParams p = {q,  k,   v,         q_stride,  k_stride, v_stride, rope,    max_pos, cu_seqlens, ctx_lens, block_table,
                          B,  T,   Hq,        Hkv,       num_pages, max_pages, 1,     q_out,   k_cache,    v_cache,  nullptr,
                          nullptr, 1.f, 1.f, dev_status};
  const int rc = append_check(p, D, dtype == EAGLE_BF16 ? 2 : 4);
  if (rc != EAGLE_OK) return rc;
  return dtype == EAGLE_BF16 ? append_launch<__nv_bfloat16, false>(p, D, stream) : append_launch<float, false>(p, D, stream);
}

extern "C" int eagle_kv_append_kv4(const void* q, const void* k, const void* v, long long q_stride,
                                   long long k_stride, long long v_stride, const float* rope, int max_pos,
                                   const int32_t* cu_seqlens, const int32_t* ctx_lens, int B, int T, int Hq, int Hkv,
                                   int D, void* q_out, uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes,
                                   uint8_t* v_scales, float k_scale, float v_scale, int num_pages,
                                   const int32_t* block_table, int max_pages, int32_t* dev_status, void* stream) {
  if (!k_scales || !v_scales || !kv4_scale_ok(k_scale) || !kv4_scale_ok(v_scale)) return EAGLE_ERR_INVALID_ARG;
  const AppendParams p = {q,  k,   v,         q_stride,  k_stride, v_stride, rope,    max_pos, cu_seqlens, ctx_lens, block_table,
                          B,  T,   Hq,        Hkv,       num_pages, max_pages, 1,     q_out,   k_codes,    v_codes,  k_scales,
                          v_scales, 1.f / k_scale, 1.f / v_scale, dev_status};
  const int rc = append_check(p, D, 2);
  if (rc != EAGLE_OK) return rc;
  return append_launch<__nv_bfloat16, true>(p, D, stream);
}

extern "C" int eagle_kv4_read(const uint8_t* codes, const uint8_t* scales, float scale, int num_pages, int Hkv, int D,
                              int dtype, void* out, void* stream) {
  if (!codes || !scales || !out || num_pages <= 0 || Hkv <= 0 || !(scale > 0.f) || !isfinite(scale))
    return EAGLE_ERR_INVALID_ARG;
  if (dtype != EAGLE_BF16 && dtype != EAGLE_FP32) return EAGLE_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || Hkv > 1024 || num_pages > (1 << 26)) return EAGLE_ERR_UNSUPPORTED;
  if (!aligned16(codes) || !aligned16(out)) return EAGLE_ERR_INVALID_ARG;
  const int ppc = std::max(1, 1024 / (Hkv * D));  // four groups per thread
  const int grid = (int)std::min<long long>((num_pages + ppc - 1) / ppc, 16ll * std::max(1, sm_count()));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == EAGLE_BF16)
    launch(kv4_read_kernel<__nv_bfloat16>, grid, 256, 0, s, (const uint2*)codes, scales, scale, Hkv, D, num_pages, ppc,
           (__nv_bfloat16*)out);
  else
    launch(kv4_read_kernel<float>, grid, 256, 0, s, (const uint2*)codes, scales, scale, Hkv, D, num_pages, ppc, (float*)out);
  note_launch();
  return last_launch_status();
}
