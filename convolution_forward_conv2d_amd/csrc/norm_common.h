// norm_common.h -- pieces shared by the norms: sums over a workgroup and rows written in e4m3.
#pragma once

#include "linear_common.h"

namespace miconv {

constexpr float E4M3_MAX = 448.0f;

template <int WAVES> __device__ __forceinline__ float block_sum(float v, float* part)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if constexpr (WAVES == 1) return v;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s += part[w];
    return s;
}

template <int WAVES> __device__ __forceinline__ float block_max(float v, float* part)
{
    // fmaxf drops a NaN: it comes back through the rows' own values
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    if constexpr (WAVES == 1) return v;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s = fmaxf(s, part[w]);
    return s;
}

// y / scale as y * inv * shift: 1 / scale overflows below 2^-128, and a zero times that is no number.
__device__ __forceinline__ void store8_e4m3(uint8_t* p, int nv, const float (&v)[8], float inv, float shift)
{
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t[i] = v[i] * shift * inv;
        t[i] = t[i] != t[i] ? t[i] : fminf(fmaxf(t[i], -E4M3_MAX), E4M3_MAX);
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int q = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * h], t[4 * h + 1], 0, false);
        w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t[4 * h + 2], t[4 * h + 3], q, true);
    }
    if (nv >= 8) {
        __builtin_memcpy(p, w, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < nv) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

}  // namespace miconv
