// norm_quant.cu -- 8-bit storage of the projections' operands: the residual's
// addition, RMSNorm and e4m3 output in one call (csa_add_norm_quant), and a
// weight's e4m3 codes in 128 x 128 blocks (csa_quantize_weight).
//
// Per row of d values:
//   s = x + residual,  v = s / sqrt(mean_j s_j^2 + eps) * gamma,
//   a_b = max(max_{j in b} |v_j| / 448, 2^-126) per block b of 128 channels,
//   code_j = e4m3(v_j / a_b), rounded to nearest even.
// Both kernels stream: HBM bytes bound them.
#include <float.h>

#include "common.cuh"
#include "kernels.h"

namespace csa {

namespace {

constexpr int kBlock = 128;       // values that share a scale (along a row)
constexpr int kThreads = 256;

// 8 consecutive values, as float.
__device__ __forceinline__ void load_8(const __nv_bfloat16 *p, float *v) { load8(p, v); }
__device__ __forceinline__ void load_8(const float *p, float *v)
{
    load4(p, v);
    load4(p + 4, v + 4);
}

__device__ __forceinline__ void store_8(__nv_bfloat16 *p, const float *v)
{
    uint4 u;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; i++)
        h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = u;
}
__device__ __forceinline__ void store_8(float *p, const float *v)
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Magnitude as an unsigned integer: ordered like the magnitude, a NaN above all.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Scale of a block whose largest magnitude has the bits m (a NaN stays one).
__device__ __forceinline__ float block_scale(uint32_t m)
{
    const float s = __uint_as_float(m) / 448.0f;
    return s < FLT_MIN ? FLT_MIN : s;
}

__device__ __forceinline__ uint2 codes_8(const float *v, float s)
{
    uint16_t c[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
        c[i] = float2_to_e4m3x2(v[2 * i] / s, v[2 * i + 1] / s);
    return make_uint2(c[0] | (uint32_t)c[1] << 16, c[2] | (uint32_t)c[3] << 16);
}

// One block of threads per row, the row read once for the sum of squares and
// once (from cache) for the outputs; 16 threads of 8 values hold a scale's block.
template <typename T>
__global__ void __launch_bounds__(kThreads)
add_norm_quant_kernel(const T *x, const T *residual, const float *__restrict__ gamma, int d,
                      int normalise, float eps, T *total, T *y, uint8_t *codes, float *scale)
{
    __shared__ float part[kThreads / 32];
    const int64_t base = (int64_t)blockIdx.x * d;
    const int nb = (d + kBlock - 1) / kBlock;
    float inv = 1.f;
    if (normalise) {
        float ss = 0.f;
        for (int j = threadIdx.x * 8; j < d; j += kThreads * 8) {
            float v[8], r[8];
            load_8(x + base + j, v);
            if (residual)
                load_8(residual + base + j, r);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float s = residual ? v[e] + r[e] : v[e];
                ss += s * s;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x >> 5] = ss;
        __syncthreads();
        ss = 0.f;
        for (int i = 0; i < kThreads / 32; i++)
            ss += part[i];
        inv = 1.f / sqrtf(ss / d + eps);
    }
    for (int j0 = 0; j0 < d; j0 += kThreads * 8) {
        const int j = j0 + threadIdx.x * 8;
        const bool live = j < d;
        float v[8], r[8];
        uint32_t m = 0;
        if (live) {
            load_8(x + base + j, v);
            if (residual) {
                load_8(residual + base + j, r);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    v[e] += r[e];
                if (total)
                    store_8(total + base + j, v);
            }
            if (normalise) {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    v[e] = v[e] * inv * (gamma ? gamma[j + e] : 1.f);
            }
            if (y)
                store_8(y + base + j, v);
#pragma unroll
            for (int e = 0; e < 8; e++)
                m = max(m, mag(v[e]));
        }
        if (codes) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (live) {
                const float s = block_scale(m);
                *reinterpret_cast<uint2 *>(codes + base + j) = codes_8(v, s);
                if (j % kBlock == 0)
                    scale[(int64_t)blockIdx.x * nb + j / kBlock] = s;
            }
        }
    }
}

// One block of threads per 128 x 128 block of the weight: 16 threads of 8
// values to a row, 16 rows at a time, held in registers between the maximum
// and the codes.
template <typename T>
__global__ void __launch_bounds__(kThreads)
quantize_weight_kernel(const T *__restrict__ W, int64_t N, int K, uint8_t *__restrict__ codes,
                       float *__restrict__ scale)
{
    __shared__ uint32_t part[kThreads / 32];
    const int kb = blockIdx.x;
    const int64_t n0 = (int64_t)blockIdx.y * kBlock;
    const int col = kb * kBlock + (threadIdx.x & 15) * 8;
    float v[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int64_t row = n0 + i * 16 + (threadIdx.x >> 4);
        if (row < N && col < K) {
            load_8(W + row * K + col, v[i]);
#pragma unroll
            for (int e = 0; e < 8; e++)
                m = max(m, mag(v[i][e]));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; i++)
        m = max(m, part[i]);
    const float s = block_scale(m);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int64_t row = n0 + i * 16 + (threadIdx.x >> 4);
        if (row < N && col < K)
            *reinterpret_cast<uint2 *>(codes + row * K + col) = codes_8(v[i], s);
    }
    if (threadIdx.x == 0)
        scale[(int64_t)blockIdx.y * gridDim.x + kb] = s;
}

}  // namespace

cudaError_t launch_add_norm_quant(const AddNormQuantArgs &a, cudaStream_t s)
{
    const unsigned grid = (unsigned)a.rows;
    if (a.dt == CSA_BF16)
        add_norm_quant_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(
            (const __nv_bfloat16 *)a.x, (const __nv_bfloat16 *)a.residual, a.gamma, a.d,
            a.normalise, a.eps, (__nv_bfloat16 *)a.total, (__nv_bfloat16 *)a.y, a.codes, a.scale);
    else
        add_norm_quant_kernel<float><<<grid, kThreads, 0, s>>>(
            (const float *)a.x, (const float *)a.residual, a.gamma, a.d, a.normalise, a.eps,
            (float *)a.total, (float *)a.y, a.codes, a.scale);
    return cudaGetLastError();
}

cudaError_t launch_quantize_weight(const QuantWeightArgs &a, cudaStream_t s)
{
    // row blocks beyond the grid's y limit go in further launches
    const int64_t nbn = (a.N + kBlock - 1) / kBlock;
    const unsigned nbk = (unsigned)((a.K + kBlock - 1) / kBlock);
    constexpr int64_t kMaxY = 65535;
    for (int64_t b0 = 0; b0 < nbn; b0 += kMaxY) {
        const int64_t nb = nbn - b0 < kMaxY ? nbn - b0 : kMaxY;
        const int64_t row0 = b0 * kBlock, rows = a.N - row0;
        const dim3 grid(nbk, (unsigned)nb);
        if (a.dt == CSA_BF16)
            quantize_weight_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(
                (const __nv_bfloat16 *)a.W + row0 * a.K, rows, a.K, a.codes + row0 * a.K,
                a.scale + b0 * nbk);
        else
            quantize_weight_kernel<float><<<grid, kThreads, 0, s>>>(
                (const float *)a.W + row0 * a.K, rows, a.K, a.codes + row0 * a.K,
                a.scale + b0 * nbk);
    }
    return cudaGetLastError();
}

}  // namespace csa
