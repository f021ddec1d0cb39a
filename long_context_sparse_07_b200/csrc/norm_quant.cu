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

// Quotients by one block's scale, each the correctly rounded float32 v / s.
// Between 2^-100 and 2^100 (where no step below under- or overflows) as
// Markstein's theorem gives it: with r the rounded reciprocal and q = v r,
// q + r (v - q s) rounds to the rounded quotient (P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990); three
// FMA-pipe instructions a value, where a division each left the weight's
// kernel bound by arithmetic. Other scales (NaN among them) divide.
struct Quotient {
    float s, r;
    bool fast;
    __device__ __forceinline__ explicit Quotient(float scale)
        : s(scale), r(1.f / scale), fast(scale >= 0x1p-100f && scale <= 0x1p100f) {}
    __device__ __forceinline__ float quick(float v) const
    {
        const float q = v * r;
        return fmaf(fmaf(-q, s, v), r, q);
    }
};

__device__ __forceinline__ uint2 codes_8(const float *v, const Quotient &q)
{
    uint16_t c[4];
    if (q.fast) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            c[i] = float2_to_e4m3x2(q.quick(v[2 * i]), q.quick(v[2 * i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            c[i] = float2_to_e4m3x2(v[2 * i] / q.s, v[2 * i + 1] / q.s);
    }
    return make_uint2(c[0] | (uint32_t)c[1] << 16, c[2] | (uint32_t)c[3] << 16);
}

// 16 bytes that are read once: past L1.
__device__ __forceinline__ uint4 load_once(const void *p) { return __ldcs((const uint4 *)p); }

// 8 consecutive values as they lie in memory.
template <typename T> struct Raw8 {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; i++)
            u[i] = load_once((const uint4 *)p + i);
    }
    __device__ __forceinline__ void floats(float *v) const
    {
        const uint32_t *w = (const uint32_t *)u;
#pragma unroll
        for (int e = 0; e < 8; e++)
            v[e] = sizeof(T) == 4 ? __uint_as_float(w[e])
                                  : __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
};

// Largest magnitude of a scale's block: the 16 lanes of a half warp.
__device__ __forceinline__ uint32_t half_warp_max(uint32_t m)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// s of CH chunks of 8 values (chunk i at j + i * step), all loads in flight
// together; zeros behind the row's end.
template <typename T, int CH>
__device__ __forceinline__ void load_sums(const T *x, const T *residual, int64_t base, int d,
                                          int j, int step, float (&v)[CH][8])
{
    Raw8<T> a[CH], b[CH];
#pragma unroll
    for (int i = 0; i < CH; i++)
        if (j + i * step < d)
            a[i].load(x + base + j + i * step);
    if (residual) {
#pragma unroll
        for (int i = 0; i < CH; i++)
            if (j + i * step < d)
                b[i].load(residual + base + j + i * step);
    }
#pragma unroll
    for (int i = 0; i < CH; i++) {
        if (j + i * step < d) {
            a[i].floats(v[i]);
            if (residual) {
                float r[8];
                b[i].floats(r);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    v[i][e] += r[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++)
                v[i][e] = 0.f;
        }
    }
}

// Rows of up to 8 CH tpr values, tpr threads (a multiple of 32) to a row and
// blockDim / tpr rows to a block. A thread holds CH chunks of 8 values, tpr
// chunks apart, from the one read to the outputs (HOLD), so that each byte
// crosses HBM once and only the sum of squares is exchanged; 16 lanes hold a
// scale's block. Rows too long for the registers are read a second time.
template <typename T, int CH, bool HOLD>
__global__ void __launch_bounds__(HOLD ? 512 : 1024)
add_norm_quant_kernel(const T *x, const T *residual, const float *__restrict__ gamma, int64_t rows,
                      int d, int tpr, float eps, T *total, T *y, uint8_t *codes, float *scale)
{
    __shared__ float part[32];
    const int sub = threadIdx.x % tpr;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const int64_t base = row * d;
    const int nb = (d + kBlock - 1) / kBlock;
    const int dl = row < rows ? d : 0;                // nothing of rows behind the last
    float v[CH][8];
    float ss = 0.f;
    for (int j0 = 0; j0 < (HOLD ? 1 : d); j0 += CH * tpr * 8) {
        load_sums<T, CH>(x, residual, base, dl, j0 + sub * 8, tpr * 8, v);
#pragma unroll
        for (int i = 0; i < CH; i++)
#pragma unroll
            for (int e = 0; e < 8; e++)
                ss = fmaf(v[i][e], v[i][e], ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (tpr > 32) {
        const int w0 = (threadIdx.x - sub) >> 5;
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x >> 5] = ss;
        __syncthreads();
        ss = 0.f;
        for (int i = 0; i < tpr / 32; i++)
            ss += part[w0 + i];
    }
    const float inv = 1.f / sqrtf(ss / d + eps);
    for (int j0 = 0; j0 < (HOLD ? 1 : d); j0 += CH * tpr * 8) {
        if (!HOLD)
            load_sums<T, CH>(x, residual, base, dl, j0 + sub * 8, tpr * 8, v);
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const int j = j0 + (i * tpr + sub) * 8;
            const bool live = j < dl;
            uint32_t m = 0;
            if (live) {
                if (total)
                    store_8(total + base + j, v[i]);
                float g[8];
                if (gamma)
                    load_8(gamma + j, g);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    v[i][e] = v[i][e] * inv * (gamma ? g[e] : 1.f);
                if (y)
                    store_8(y + base + j, v[i]);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    m = max(m, mag(v[i][e]));
            }
            if (codes) {
                m = half_warp_max(m);
                if (live) {
                    const float s = block_scale(m);
                    *reinterpret_cast<uint2 *>(codes + base + j) = codes_8(v[i], Quotient(s));
                    if (j % kBlock == 0)
                        scale[row * nb + j / kBlock] = s;
                }
            }
        }
    }
}

// Without the norm every block of 128 channels stands by itself: a half warp
// takes CH of them at a time.
template <typename T, int CH>
__global__ void __launch_bounds__(kThreads)
add_quant_kernel(const T *x, const T *residual, int64_t rows, int d, T *total, T *y,
                 uint8_t *codes, float *scale)
{
    const int nb = (d + kBlock - 1) / kBlock;
    const int64_t blocks = rows * nb;
    constexpr int kHalves = kThreads / 16;
    const int64_t first = (int64_t)blockIdx.x * kHalves * CH + threadIdx.x / 16;
    Raw8<T> a[CH], b[CH];
    int64_t at[CH];                                   // this thread's chunk, -1 for none
#pragma unroll
    for (int i = 0; i < CH; i++) {
        const int64_t g = first + i * kHalves;
        const int64_t row = g / nb;
        const int j = (int)(g - row * nb) * kBlock + (threadIdx.x & 15) * 8;
        at[i] = g < blocks && j < d ? row * d + j : -1;
        if (at[i] >= 0) {
            a[i].load(x + at[i]);
            if (residual)
                b[i].load(residual + at[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < CH; i++) {
        float v[8];
        uint32_t m = 0;
        if (at[i] >= 0) {
            a[i].floats(v);
            if (residual) {
                float r[8];
                b[i].floats(r);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    v[e] += r[e];
                if (total)
                    store_8(total + at[i], v);
            }
            if (y)
                store_8(y + at[i], v);
#pragma unroll
            for (int e = 0; e < 8; e++)
                m = max(m, mag(v[e]));
        }
        if (codes) {
            m = half_warp_max(m);
            if (at[i] >= 0) {
                const float s = block_scale(m);
                *reinterpret_cast<uint2 *>(codes + at[i]) = codes_8(v, Quotient(s));
                if ((threadIdx.x & 15) == 0)
                    scale[first + i * kHalves] = s;
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
    const Quotient q(s);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int64_t row = n0 + i * 16 + (threadIdx.x >> 4);
        if (row < N && col < K)
            *reinterpret_cast<uint2 *>(codes + row * K + col) = codes_8(v[i], q);
    }
    if (threadIdx.x == 0)
        scale[(int64_t)blockIdx.y * gridDim.x + kb] = s;
}

template <typename T, int CH, bool HOLD>
void launch_norm(const AddNormQuantArgs &a, int tpr, int rpb, cudaStream_t s)
{
    add_norm_quant_kernel<T, CH, HOLD><<<(unsigned)((a.rows + rpb - 1) / rpb), tpr * rpb, 0, s>>>(
        (const T *)a.x, (const T *)a.residual, a.gamma, a.rows, a.d, tpr, a.eps, (T *)a.total,
        (T *)a.y, a.codes, a.scale);
}

template <typename T>
cudaError_t launch_add_norm_quant_t(const AddNormQuantArgs &a, cudaStream_t s)
{
    if (!a.normalise) {
        constexpr int CH = 4;
        const int64_t blocks = a.rows * ((a.d + kBlock - 1) / kBlock);
        const int64_t grid = (blocks + kThreads / 16 * CH - 1) / (kThreads / 16 * CH);
        if (grid > INT32_MAX)
            return cudaErrorInvalidConfiguration;
        add_quant_kernel<T, CH><<<(unsigned)grid, kThreads, 0, s>>>(
            (const T *)a.x, (const T *)a.residual, a.rows, a.d, (T *)a.total, (T *)a.y, a.codes,
            a.scale);
        return cudaGetLastError();
    }
    const int warps = (a.d + 255) / 256;              // of 8 values a lane
    if (warps <= 8) {
        const int tpr = 32 * ((warps + 1) / 2);
        launch_norm<T, 2, true>(a, tpr, 256 / tpr, s);
    } else if (warps <= 64) {
        const int tpr = 32 * ((warps + 3) / 4);
        launch_norm<T, 4, true>(a, tpr, tpr < 256 ? 256 / tpr : 1, s);
    } else {
        launch_norm<T, 2, false>(a, 1024, 1, s);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_norm_quant(const AddNormQuantArgs &a, cudaStream_t s)
{
    return a.dt == CSA_BF16 ? launch_add_norm_quant_t<__nv_bfloat16>(a, s)
                            : launch_add_norm_quant_t<float>(a, s);
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
