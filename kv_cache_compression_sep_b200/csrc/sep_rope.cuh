// Rotation angles and 16-bit / fp32 conversions of the rotary and paged-cache kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace sep {

// (cos, sin) of the angle pos * f with the arithmetic of SepCache's kernels (k_sepcache.cu), so that
// a key rotated here and one rotated there agree: the angle is formed in fp64 and reduced to
// [-pi, pi] by subtracting the nearest multiple of 2 pi (fp64), then the fp32 sincosf of the
// reduced angle is taken. The error is about 1e-7 absolute, from rounding the reduced angle.
__device__ __forceinline__ void rope_angle(long long pos, double f, float* cs, float* sn) {
  constexpr double kTwoPi = 6.283185307179586, kInvTwoPi = 0.15915494309189535;
  const double x = __dmul_rn((double)pos, f);
  const double r = __fma_rn(-rint(__dmul_rn(x, kInvTwoPi)), kTwoPi, x);
  sincosf((float)r, sn, cs);
}

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) {
  return __float2half_rn(x);
}
template <>
__device__ __forceinline__ float from_float<float>(float x) {
  return x;
}

}  // namespace sep
