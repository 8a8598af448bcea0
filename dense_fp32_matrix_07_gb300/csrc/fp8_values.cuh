// Values to 8 bits and their blocks' scales, as all quantising kernels make them.
#pragma once

#include "experts.cuh"

#include <cuda_fp8.h>

namespace sgemm_gb300 {

// Magnitudes as unsigned integers: they order like the floats, with NaN above
// infinity, so that a NaN in a block wins the maximum.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

struct Scale {
    float inv, scale;
};

__device__ __forceinline__ Scale scale_of(uint32_t amax)
{
    float a = __uint_as_float(amax);
    if (a < kFp8Least) a = kFp8Least;   // false for NaN
    return Scale{__fdiv_rn(kFp8Max, a), __fdiv_rn(a, kFp8Max)};
}

// Four values to four bytes (cvt.rn.satfinite.e4m3x2.f32 keeps NaN).
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

}  // namespace sgemm_gb300
