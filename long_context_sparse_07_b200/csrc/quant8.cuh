// quant8.cuh -- the e4m3 storage rule of the 8-bit projections: a block of
// values shares the scale max(amax / 448, 2^-126), a value's code is value /
// scale rounded to nearest even.
#pragma once

#include <float.h>

#include "common.cuh"

namespace csa {

// Largest of m and two magnitudes; a NaN wins.
__device__ __forceinline__ float max_mag(float m, float2 v)
{
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(v.x), "f"(v.y));
    return m;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(a), "f"(b));
    return a;
}

// Scale of a block with the largest magnitude m (a NaN stays one).
__device__ __forceinline__ float block_scale(float m)
{
    const float s = m / 448.0f;
    return s < FLT_MIN ? FLT_MIN : s;
}

__device__ __forceinline__ uint32_t codes_2(float2 q)
{
    return (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
}

// 4 NW codes, one to a byte, of values of a block with scale s, each from the
// correctly rounded float32 quotient v / s. Between 2^-100 and 2^100 (where no
// step below under- or overflows) the quotient is taken as Markstein's theorem
// gives it: with r the rounded reciprocal and q = v r, q + r (v - q s) rounds
// to the rounded quotient (P. Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990): three packed instructions for
// two values. Other scales (NaN among them) divide. (v r alone turns ties
// around: 7 x 1.5625 over a scale of 7 is 1.5625 + 2^-23, the next code up.)
template <int NW>
__device__ __forceinline__ void codes_of(const float2 *v, float s, uint32_t (&w)[NW])
{
    if (s >= 0x1p-100f && s <= 0x1p100f) {
        const float r = 1.f / s;
        const float2 r2 = make_float2(r, r), s2 = make_float2(-s, -s);
#pragma unroll
        for (int i = 0; i < NW; i++) {
            uint32_t h[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float2 x = v[2 * i + e], q = __fmul2_rn(x, r2);
                h[e] = codes_2(__ffma2_rn(__ffma2_rn(q, s2, x), r2, q));
            }
            w[i] = h[0] | h[1] << 16;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NW; i++)
            w[i] = codes_2(make_float2(v[2 * i].x / s, v[2 * i].y / s)) |
                   codes_2(make_float2(v[2 * i + 1].x / s, v[2 * i + 1].y / s)) << 16;
    }
}

}  // namespace csa
