// 4-bit cache rows and the lookup of a packed row's request, shared by the
// append and attention kernels of the prompt path.
//
// A group of 16 channels shares one e4m3 scale; a channel's code is a sign
// and one of the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace eagle {

// e4m3 scale byte of a group whose largest magnitude is `amax`: amax / 6 to
// nearest even, at most 448; NaN stays NaN.
__device__ __forceinline__ uint8_t kv4_scale(float amax) {
  return (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.f), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float kv4_scale_value(uint8_t s) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3)));
}
// Code of x under the scale s: the magnitude nearest to |x| / s.  The
// comparisons with s times the midpoints are exact (a midpoint has three
// significant bits, s four), so no division decides a code; a tie goes to the
// even code.
__device__ __forceinline__ uint32_t kv4_code(float x, float s) {
  const float a = fabsf(x);
  uint32_t c = 0;
  if (s > 0.f)
    c = (a > 0.25f * s) + (a >= 0.75f * s) + (a > 1.25f * s) + (a >= 1.75f * s) + (a > 2.5f * s) + (a >= 3.5f * s) +
        (a > 5.f * s);
  return c | (__float_as_uint(x) >> 31 << 3);
}
__device__ __forceinline__ float kv4_code_value(uint32_t c) {
  // magnitudes 0, 0.5 (no leading one), then 2^(e-1) (1 + m/2), e = c >> 1
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float f = e ? __uint_as_float(((126u + e) << 23) | (m << 22)) : 0.5f * (float)m;
  return (c & 8u) ? -f : f;
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
