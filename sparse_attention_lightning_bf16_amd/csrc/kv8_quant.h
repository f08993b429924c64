// Rows of values into a page of e4m3 codes with one scale: shared by
// appending to the cache and by moving kept tokens to new pages.
#pragma once

#include "common.h"

namespace lix {

constexpr float kE4M3Max = 448.0f;

// The smallest power of two s >= top / 448, not below 2^-60, for a finite
// top >= 0.  448 = 1.75 * 2^8: the exponent of top less 8, one more if top's
// significand is above 1.75; exact, no division.
__device__ __forceinline__ float page_scale(float top) {
    const uint32_t u = __float_as_uint(top);
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, -60);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Four values as e4m3 bytes, rounded to nearest even; NaN stays NaN.  SATURATE:
// values beyond 448 become 448; without it they have to be within.
template <bool SATURATE>
__device__ __forceinline__ uint32_t e4m3_quad(const float (&x)[4]) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = x[i];
        if (SATURATE) y[i] = y[i] > kE4M3Max ? kE4M3Max : y[i] < -kE4M3Max ? -kE4M3Max : y[i];   // NaN compares false
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
    return (uint32_t)w;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void e4m3_quad_to_f32(uint32_t w, float (&x)[4]) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[0] = lo.x;
    x[1] = lo.y;
    x[2] = hi.x;
    x[3] = hi.y;
}

constexpr float kInf = __builtin_inff();

// max(top, |x|) over finite x: infinities and NaN leave top as it is.
__device__ __forceinline__ float finite_top(float top, float x) {
    const float m = fabsf(x);
    return m < kInf ? fmaxf(top, m) : top;
}

// Maximum over the 256 threads of a workgroup; `part` holds 4 floats of LDS
// that no thread is still reading.
__device__ __forceinline__ float workgroup_max(float v, float* part) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
}

}  // namespace lix
