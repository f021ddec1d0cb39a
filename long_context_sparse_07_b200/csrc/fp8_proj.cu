// fp8_proj.cu -- product of e4m3 activations and weights with block scales
// (csa_fp8_proj):
//   r[t, j] = sum_b As[t, b] Ws[j / 128, b] sum_{k in block b} A[t, k] W[j, k],
// blocks b of 128 inputs, float32 sums; bf16, float32 or e4m3 results.
//
// CUDA cores: a block of threads owns 32 tokens x 128 features, a warp four
// of the tokens with all 128 features (so that an output scale's block lies in
// one warp). Operands are decoded to float in shared memory 32 inputs at a
// time; each block of 128 inputs is summed by itself, then scaled and added.
#include <float.h>

#include "common.cuh"
#include "kernels.h"

namespace csa {

namespace {

constexpr int PM = 32, PN = 128, PK = 32, PB = 128;
constexpr int PTHREADS = 256;

__global__ void __launch_bounds__(PTHREADS)
fp8_proj_kernel(const Fp8ProjArgs a)
{
    __shared__ float sa[PK][PM + 4], sw[PK][PN + 4];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int nb = (a.K + PB - 1) / PB, nt = (a.N + PN - 1) / PN;
    const int64_t lda = (int64_t)a.groups * a.K, ldo = (int64_t)a.groups * a.N;
    const int64_t m0 = (int64_t)(blockIdx.x / (nt * a.groups)) * PM;
    const int g = blockIdx.x / nt % a.groups;
    const int n0 = blockIdx.x % nt * PN;              // first feature, within the group
    const uint8_t *A = a.A + (int64_t)g * a.K;
    const uint8_t *W = a.W + (int64_t)g * a.N * a.K;
    const float *As = a.As + (int64_t)g * nb;
    const float *Ws = a.Ws + ((int64_t)g * a.N + n0) / PB * nb;
    float acc[4][4] = {};
    for (int b = 0; b < nb; b++) {
        float p[4][4] = {};
        for (int k0 = b * PB; k0 < min(a.K, (b + 1) * PB); k0 += PK) {
            __syncthreads();
            for (int i = threadIdx.x; i < (PM + PN) * PK / 4; i += PTHREADS) {
                const int r = i / (PK / 4), k = i % (PK / 4) * 4;
                const bool is_a = r < PM;
                const int64_t row = is_a ? m0 + r : (int64_t)n0 + r - PM;
                uint32_t u = 0;
                if (row < (is_a ? a.M : (int64_t)a.N) && k0 + k < a.K)
                    u = *(const uint32_t *)((is_a ? A + row * lda : W + row * a.K) + k0 + k);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float v = e4m3_to_float((uint8_t)(u >> (8 * e)));
                    if (is_a)
                        sa[k + e][r] = v;
                    else
                        sw[k + e][r - PM] = v;
                }
            }
            __syncthreads();
#pragma unroll 8
            for (int k = 0; k < PK; k++) {
                const float4 x = *(const float4 *)&sa[k][ty * 4];
                const float4 w = *(const float4 *)&sw[k][tx * 4];
                const float xv[4] = {x.x, x.y, x.z, x.w}, wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        p[i][j] = fmaf(xv[i], wv[j], p[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int64_t t = m0 + ty * 4 + i;
            const float s = t < a.M ? As[t * a.groups * nb + b] * Ws[b] : 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++)
                acc[i][j] = fmaf(p[i][j], s, acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t t = m0 + ty * 4 + i;
        const int64_t o = t * ldo + (int64_t)g * a.N + n0 + tx * 4;
        float s = 1.f;
        if (a.out_dt == CSA_E4M3) {
            uint32_t m = 0;                           // features behind the last one are zero
#pragma unroll
            for (int j = 0; j < 4; j++)
                m = max(m, __float_as_uint(acc[i][j]) & 0x7fffffffu);
#pragma unroll
            for (int f = 16; f > 0; f >>= 1)
                m = max(m, __shfl_xor_sync(0xffffffffu, m, f));
            s = __uint_as_float(m) / 448.0f;
            if (s < FLT_MIN)
                s = FLT_MIN;
            if (tx == 0 && t < a.M)
                a.out_scale[t * ((ldo + PB - 1) / PB) + ((int64_t)g * a.N + n0) / PB] = s;
        }
        if (t >= a.M)
            continue;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (n0 + tx * 4 + j >= a.N)
                break;
            if (a.out_dt == CSA_F32)
                ((float *)a.out)[o + j] = acc[i][j];
            else if (a.out_dt == CSA_BF16)
                ((__nv_bfloat16 *)a.out)[o + j] = __float2bfloat16_rn(acc[i][j]);
            else
                ((uint8_t *)a.out)[o + j] = (uint8_t)float2_to_e4m3x2(acc[i][j] / s, 0.f);
        }
    }
}

}  // namespace

cudaError_t launch_fp8_proj(const Fp8ProjArgs &a, unsigned *err, cudaStream_t s)
{
    (void)err;
    const int64_t tiles = (a.M + PM - 1) / PM * ((a.N + PN - 1) / PN) * a.groups;
    if (tiles > INT32_MAX)
        return cudaErrorInvalidConfiguration;
    fp8_proj_kernel<<<(unsigned)tiles, PTHREADS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace csa
