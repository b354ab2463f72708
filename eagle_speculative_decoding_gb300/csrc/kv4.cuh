// 4-bit cache rows and the lookup of a packed row's request, shared by the
// append and attention kernels of the prompt path.
//
// A group of 16 channels shares one e4m3 scale; a channel's code is a sign
// and one of the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "common.cuh"

namespace eagle {

// A cache's k_scale or v_scale that rows can be divided by: finite, positive, and
// of a finite reciprocal (an infinite one would make NaN of zeros).
inline bool kv4_scale_ok(float s) { return s > 0.f && isfinite(s) && isfinite(1.f / s); }

// e4m3 scale byte of a group whose largest magnitude is `amax`: amax / 6 to
// nearest even, at most 448; NaN stays NaN.
__device__ __forceinline__ uint8_t kv4_scale(float amax) {
  return (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.f), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float kv4_scale_value(uint8_t s) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3)));
}
// Codes of eight values under the scale s, the first in the low bits: the
// magnitude nearest to |x| / s, a tie to the even code (0 if s is 0 or NaN).
// The rounded quotient decides as the exact one would: a midpoint times s has at
// most seven significant bits, so an x that is not on it is off by 2^-24 of
// itself or more, and the quotient then rounds to the same side of the midpoint.
// (Comparisons with s times the seven midpoints instead: 54 us against 51 us for
// 8125 rows of 32 + 2 x 8 heads, when four items were in flight.)
__device__ __forceinline__ uint32_t kv4_codes(const float* x, float s) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = s > 0.f ? __fdiv_rn(x[i], s) : copysignf(0.f, x[i]);
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}
// The values of eight codes.
__device__ __forceinline__ void kv4_values(uint32_t w, float* f) {
  uint32_t v[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

// The last request b of [0, B) with cu[b] <= t, by 32-way search (one load
// per level: B <= 32 takes one, B <= 1024 two).  Whole warps call it with the
// same t; reads only cu[0 .. B-1], whatever they hold.
__device__ __forceinline__ int warp_find_request(const int32_t* __restrict__ cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const bool le = i < hi && cu[i] <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    const int at = lo + max(n - 1, 0) * step;
    hi = min(hi, at + step);
    lo = at;
  }
  return lo;
}

}  // namespace eagle
