// norm_quant.cu -- 8-bit storage of the projections' operands: the residual's
// addition, RMSNorm and e4m3 output in one call (csa_add_norm_quant), and a
// weight's e4m3 codes in 128 x 128 blocks (csa_quantize_weight).
//
// Per row of d values:
//   s = x + residual,  v = s / sqrt(mean_j s_j^2 + eps) * gamma,
//   a_b = max(max_{j in b} |v_j| / 448, 2^-126) per block b of 128 channels,
//   code_j = e4m3(v_j / a_b), rounded to nearest even.
// HBM bytes bound these kernels as long as a value costs few instructions: at
// 3 bytes a value (unnormed bf16) an SM has about 16 issue slots for each.
// Hence packed pairs of float32 (one instruction for two values), quotients
// without a division, and 16 consecutive values to a lane, so that a scale's
// block is 8 lanes and its maximum three shuffles for every 16 values. A lane's
// values are whole sectors of 32 bytes, moved by one instruction each where the
// buffers are aligned so (in halves, 16384 x 4096 float32 takes 158 us in place
// of 130). Measured in a graph: 65536 x 4096 bf16 with residual and total 293 us
// (6.4 TB/s, the copy rate; 500 us with a division a value and each row read
// twice), the unnormed 4096 x 32768 69 us (5.9 TB/s), a weight of 32768 x 1024
// 18.2 us (5.5 TB/s), 8 rows of 4096 3 us (the launch).
#include "common.cuh"
#include "kernels.h"
#include "quant8.cuh"
#include "tc.cuh"

namespace csa {

namespace {

constexpr int kBlock = 128;       // values that share a scale (along a row)
constexpr int kThreads = 256;
constexpr int kLane = 16;         // consecutive values of a lane
constexpr int kPairs = kLane / 2;

// 16 consecutive values as they lie in memory, moved as sectors of 32 bytes
// where the buffers' alignment allows (`wide`), else in halves.
template <typename T> struct Raw {
    uint4 u[sizeof(T)];
    __device__ __forceinline__ void load(const T *p, bool wide)
    {
        const uint4 *q = (const uint4 *)p;
        if (wide) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); i += 2)
                asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(u[i].x), "=r"(u[i].y), "=r"(u[i].z), "=r"(u[i].w),
                               "=r"(u[i + 1].x), "=r"(u[i + 1].y), "=r"(u[i + 1].z),
                               "=r"(u[i + 1].w)
                             : "l"(q + i)
                             : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); i++)
                u[i] = q[i];
        }
    }
    __device__ __forceinline__ void store(T *p, bool wide) const
    {
        uint4 *q = (uint4 *)p;
        if (wide) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); i += 2)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q + i),
                             "r"(u[i].x), "r"(u[i].y), "r"(u[i].z), "r"(u[i].w), "r"(u[i + 1].x),
                             "r"(u[i + 1].y), "r"(u[i + 1].z), "r"(u[i + 1].w)
                             : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); i++)
                q[i] = u[i];
        }
    }
    __device__ __forceinline__ float2 pair(int i) const
    {
        const uint32_t *w = (const uint32_t *)u;
        if (sizeof(T) == 4)
            return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
};

__device__ __forceinline__ void store_16(__nv_bfloat16 *p, const float2 (&v)[kPairs], bool wide)
{
    Raw<__nv_bfloat16> r;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const __nv_bfloat162 h = __float22bfloat162_rn(v[4 * i + e]);
            w[e] = *(const uint32_t *)&h;
        }
        r.u[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    r.store(p, wide);
}
__device__ __forceinline__ void store_16(float *p, const float2 (&v)[kPairs], bool wide)
{
    Raw<float> r;
#pragma unroll
    for (int i = 0; i < 4; i++)
        r.u[i] = make_uint4(__float_as_uint(v[2 * i].x), __float_as_uint(v[2 * i].y),
                            __float_as_uint(v[2 * i + 1].x), __float_as_uint(v[2 * i + 1].y));
    r.store(p, wide);
}

// Largest magnitude of a scale's block: 16 values of each of 8 lanes.
__device__ __forceinline__ float block_max(const float2 (&v)[kPairs], float m = 0.f)
{
#pragma unroll
    for (int i = 0; i < kPairs; i++)
        m = max_mag(m, v[i]);
    return m;
}

__device__ __forceinline__ float eight_lane_max(float m)
{
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

__device__ __forceinline__ uint4 codes_16(const float2 (&v)[kPairs], float s)
{
    uint32_t w[4];
    codes_of<4>(v, s, w);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 16 gains from gamma + j: only 4-byte aligned in general.
__device__ __forceinline__ void load_gains(const float *gamma, int j, bool aligned,
                                           float2 (&g)[kPairs])
{
    if (aligned) {
#pragma unroll
        for (int e = 0; e < kPairs; e += 2) {
            const float4 f = *(const float4 *)(gamma + j + 2 * e);
            g[e] = make_float2(f.x, f.y);
            g[e + 1] = make_float2(f.z, f.w);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kPairs; e++)
            g[e] = make_float2(gamma[j + 2 * e], gamma[j + 2 * e + 1]);
    }
}

// Sum over a row's tpr threads: 8, 16 or a multiple of 32. `part` is this
// call's own place of 32 floats. Threads of other rows take part as well.
__device__ __forceinline__ float row_sum(float ss, int tpr, int sub, float *part)
{
    for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1)
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
    return ss;
}

// The outputs of one lane piece whose values are normed already (but for
// total, which the caller writes); every lane of the warp calls it.
template <typename T>
__device__ __forceinline__ void write_piece(const float2 (&v)[kPairs], bool live, int64_t base,
                                            int j, int64_t row, int nb, T *y, uint8_t *codes,
                                            float *scale, bool wide)
{
    if (live && y)
        store_16(y + base + j, v, wide);
    if (codes) {
        const float m = eight_lane_max(block_max(v));
        if (live) {
            const float s = block_scale(m);
            *reinterpret_cast<uint4 *>(codes + base + j) = codes_16(v, s);
            if (j % kBlock == 0)
                scale[row * nb + j / kBlock] = s;
        }
    }
}

// Rows of up to 16 tpr values, tpr threads to a row and blockDim / tpr rows at
// a time; the grid is resident and strides over the rows. A thread's 16 values
// stay in its registers from the one read to the outputs, so that each byte
// crosses HBM once and only the sum of squares is exchanged, and its 16 gains
// for all its rows (read per row they cost more L1 traffic than the row). The
// next row is read while this one is written: x before the sums are exchanged,
// the residual after them (both before: 340 against 294 us for 65536 x 4096
// bf16, with reads and writes crowding each other; a
// call without a residual, RES = false, takes 201 us, with a test of the pointer
// in the loop 267).
// A few longer rows are each cut over a cluster of thread blocks (CLUSTER; `cut`
// values a block), which add their sums of squares in the order of their ranks:
// one row of 32768 takes 4.2 us in a graph, read twice by one block 7.6 us.
constexpr int min_blocks(int size, int most, bool res)
{
    // as many registers as the loop takes without spilling much
    return size == 2 ? (most == 512 ? 2 : 1) : most == 256 ? (res ? 2 : 3) : 1;
}

template <typename T, bool CLUSTER, int MOST, bool RES>
__global__ void __launch_bounds__(MOST, min_blocks(sizeof(T), MOST, RES))
add_norm_quant_kernel(const T *x, const T *residual, const float *gamma,
                      bool gamma_aligned, int64_t rows, int d, int tpr, int cut, int ranks,
                      float eps, T *total, T *y, uint8_t *codes, float *scale, bool wide)
{
    __shared__ float part[2][32];
    __shared__ float sums[2];
    const int rank = CLUSTER ? (int)tc::cluster_rank() : 0;
    const int sub = threadIdx.x % tpr;
    const int rpb = blockDim.x / tpr;
    const int j = rank * cut + sub * kLane;
    const int nb = (d + kBlock - 1) / kBlock;
    const bool in = j < d && sub * kLane < cut;
    float2 g[kPairs];
#pragma unroll
    for (int e = 0; e < kPairs; e++)
        g[e] = make_float2(1.f, 1.f);
    tc::grid_let_next();
    tc::grid_wait();
    if (gamma && in)
        load_gains(gamma, j, gamma_aligned, g);
    Raw<T> a, b;
    const int64_t stride = (int64_t)gridDim.x / ranks * rpb, mine = threadIdx.x / tpr;
    int64_t r0 = (int64_t)(blockIdx.x / ranks) * rpb;  // the block's first row
    auto read_x = [&](int64_t row) {
        if (row < rows && in)
            a.load(x + row * d + j, wide);
    };
    auto read_residual = [&](int64_t row) {
        if (RES && row < rows && in)
            b.load(residual + row * d + j, wide);
    };
    read_x(r0 + mine);
    read_residual(r0 + mine);
    for (int parity = 0; r0 < rows; r0 += stride, parity ^= 1) {
        const int64_t row = r0 + mine, base = row * d;
        const bool live = row < rows && in;
        float2 v[kPairs];
        float2 ss2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < kPairs; e++) {
            v[e] = make_float2(0.f, 0.f);
            if (live)
                v[e] = RES ? __fadd2_rn(a.pair(e), b.pair(e)) : a.pair(e);
            ss2 = __ffma2_rn(v[e], v[e], ss2);
        }
        read_x(row + stride);
        if (RES && live && total)
            store_16(total + base + j, v, wide);
        float ss = row_sum(ss2.x + ss2.y, tpr, sub, part[parity]);
        read_residual(row + stride);
        if (CLUSTER) {
            // the place of one row is written again two rows later, when every
            // block has passed the next row's barrier and so read this one
            if (threadIdx.x == 0)
                sums[parity] = ss;
            __syncwarp();
            tc::cluster_sync();
            ss = 0.f;
            for (int q = 0; q < ranks; q++)
                ss += tc::cluster_ld(&sums[parity], q);
        }
        const float inv = rsqrtf(ss / d + eps);
#pragma unroll
        for (int e = 0; e < kPairs; e++)
            v[e] = __fmul2_rn(__fmul2_rn(v[e], make_float2(inv, inv)), g[e]);
        write_piece(v, live, base, j, row, nb, y, codes, scale, wide);
    }
    if (CLUSTER) {
        // no block leaves while another may still read its sums
        __syncwarp();
        tc::cluster_sync();
    }
}

// Many rows too long for a block's registers, one to a block, are read a second
// time (from L2) for the outputs; the cluster's barrier a row would cost more
// (4096 rows of 32768: 343 against 195 us).
constexpr int kLongThreads = 512;

template <typename T, bool RES>
__global__ void __launch_bounds__(kLongThreads, sizeof(T) == 2 ? 2 : 1)
add_norm_quant_long_kernel(const T *x, const T *residual, const float *gamma,
                           bool gamma_aligned, int d, float eps, T *total, T *y, uint8_t *codes,
                           float *scale, bool wide)
{
    constexpr int kStep = kLongThreads * kLane;
    __shared__ float part[32];
    const int64_t row = blockIdx.x, base = row * d;
    const int nb = (d + kBlock - 1) / kBlock;
    const int first = threadIdx.x * kLane;
    Raw<T> a, b;
    auto read = [&](int j) {
        if (j < d) {
            a.load(x + base + j, wide);
            if (RES)
                b.load(residual + base + j, wide);
        }
    };
    // the piece read last, and the next one on its way
    float2 v[kPairs], ss2 = make_float2(0.f, 0.f);
    auto take = [&](int j) {
#pragma unroll
        for (int e = 0; e < kPairs; e++) {
            v[e] = make_float2(0.f, 0.f);
            if (j < d)
                v[e] = RES ? __fadd2_rn(a.pair(e), b.pair(e)) : a.pair(e);
        }
        read(j + kStep);
    };
    tc::grid_let_next();
    tc::grid_wait();
    read(first);
    for (int j = first; j - first < d; j += kStep) {
        take(j);
#pragma unroll
        for (int e = 0; e < kPairs; e++)
            ss2 = __ffma2_rn(v[e], v[e], ss2);
    }
    read(first);
    const float ss = row_sum(ss2.x + ss2.y, kLongThreads, threadIdx.x, part);
    const float inv = rsqrtf(ss / d + eps);
    for (int j = first; j - first < d; j += kStep) {
        take(j);
        if (RES && j < d && total)
            store_16(total + base + j, v, wide);
#pragma unroll
        for (int e = 0; e < kPairs; e++)
            v[e] = __fmul2_rn(v[e], make_float2(inv, inv));
        if (gamma && j < d) {
            float2 g[kPairs];
            load_gains(gamma, j, gamma_aligned, g);
#pragma unroll
            for (int e = 0; e < kPairs; e++)
                v[e] = __fmul2_rn(v[e], g[e]);
        }
        write_piece(v, j < d, base, j, row, nb, y, codes, scale, wide);
    }
}

// Without the norm every block of 128 channels stands by itself: 8 lanes take
// CH of them at a time. FLAT: d is a multiple of 128, so that block g of the
// whole array is values 128 g ..
template <typename T, int CH, bool FLAT>
__global__ void __launch_bounds__(kThreads)
add_quant_kernel(const T *x, const T *residual, int64_t rows, int d, T *total, T *y,
                 uint8_t *codes, float *scale, bool wide)
{
    const int nb = (d + kBlock - 1) / kBlock;
    const int64_t blocks = rows * nb;
    constexpr int kEights = kThreads / 8;
    const int64_t first = (int64_t)blockIdx.x * kEights * CH + threadIdx.x / 8;
    const int off = (threadIdx.x & 7) * kLane;
    const int64_t row0 = FLAT ? 0 : first / nb;
    const unsigned col0 = FLAT ? 0u : (unsigned)(first - row0 * nb);
    int64_t at[CH];                                   // this thread's piece, -1 for none
#pragma unroll
    for (int i = 0; i < CH; i++) {
        const int64_t g = first + i * kEights;
        if (FLAT) {
            at[i] = g < blocks ? g * kBlock + off : -1;
        } else {
            const unsigned c = col0 + i * kEights, up = c / nb;
            const int j = (int)(c - up * nb) * kBlock + off;
            at[i] = g < blocks && j < d ? (row0 + up) * d + j : -1;
        }
    }
    tc::grid_let_next();
    tc::grid_wait();
    float2 v[CH][kPairs];
    {
        Raw<T> a[CH], b[CH];
#pragma unroll
        for (int i = 0; i < CH; i++) {
            if (at[i] >= 0) {
                a[i].load(x + at[i], wide);
                if (residual)
                    b[i].load(residual + at[i], wide);
            }
        }
#pragma unroll
        for (int i = 0; i < CH; i++)
#pragma unroll
            for (int e = 0; e < kPairs; e++) {
                v[i][e] = make_float2(0.f, 0.f);
                if (at[i] >= 0)
                    v[i][e] = residual ? __fadd2_rn(a[i].pair(e), b[i].pair(e)) : a[i].pair(e);
            }
    }
#pragma unroll
    for (int i = 0; i < CH; i++) {
        if (at[i] >= 0) {
            if (total)
                store_16(total + at[i], v[i], wide);
            if (y)
                store_16(y + at[i], v[i], wide);
        }
        if (codes) {
            const float m = eight_lane_max(block_max(v[i]));
            if (at[i] >= 0) {
                const float s = block_scale(m);
                *reinterpret_cast<uint4 *>(codes + at[i]) = codes_16(v[i], s);
                if (off == 0)
                    scale[first + i * kEights] = s;
            }
        }
    }
}

// One block of threads per 128 x 128 block of the weight: 8 lanes to a row,
// four pieces of 16 values a thread, held as they were read between the
// maximum and the codes (in bf16 few enough registers for four such blocks on
// an SM, which hide each other's barrier).
constexpr int kPieces = kBlock * kBlock / (kThreads * kLane);
constexpr int kRowStep = kThreads / 8;

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
quantize_weight_kernel(const T *W, int64_t N, int K, uint8_t *codes, float *scale, bool wide)
{
    __shared__ float part[kThreads / 32];
    const int kb = blockIdx.x;
    const int64_t n0 = (int64_t)blockIdx.y * kBlock + (threadIdx.x >> 3);
    const int col = kb * kBlock + (threadIdx.x & 7) * kLane;
    tc::grid_let_next();
    tc::grid_wait();
    Raw<T> a[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; i++) {
        if (n0 + i * kRowStep < N && col < K)
            a[i].load(W + (n0 + i * kRowStep) * K + col, wide);
        else
            a[i] = Raw<T>{};
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; i++)
#pragma unroll
        for (int e = 0; e < kPairs; e++)
            m = max_mag(m, a[i].pair(e));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; i++)
        m = max_nan(m, part[i]);
    const float s = block_scale(m);
#pragma unroll
    for (int i = 0; i < kPieces; i++) {
        if (n0 + i * kRowStep < N && col < K) {
            float2 v[kPairs];
#pragma unroll
            for (int e = 0; e < kPairs; e++)
                v[e] = a[i].pair(e);
            *reinterpret_cast<uint4 *>(codes + (n0 + i * kRowStep) * K + col) = codes_16(v, s);
        }
    }
    if (threadIdx.x == 0)
        scale[(int64_t)blockIdx.y * gridDim.x + kb] = s;
}

// Rows are whole sectors of 32 bytes (16 values), so only the bases count.
bool sectors(const void *p, const void *q = nullptr, const void *r = nullptr,
             const void *s = nullptr)
{
    return (((uintptr_t)p | (uintptr_t)q | (uintptr_t)r | (uintptr_t)s) & 31u) == 0;
}

template <typename T, bool FLAT>
cudaError_t launch_quant(const AddNormQuantArgs &a, cudaStream_t s)
{
    constexpr int CH = 2;
    const int64_t blocks = a.rows * ((a.d + kBlock - 1) / kBlock);
    const int64_t grid = (blocks + kThreads / 8 * CH - 1) / (kThreads / 8 * CH);
    if (grid > INT32_MAX)
        return cudaErrorInvalidConfiguration;
    return launch_early(add_quant_kernel<T, CH, FLAT>, dim3((unsigned)grid), kThreads, 0, 1, s,
                        (const T *)a.x, (const T *)a.residual, a.rows, a.d, (T *)a.total, (T *)a.y,
                        a.codes, a.scale, sectors(a.x, a.residual, a.total, a.y));
}

template <typename T, bool CLUSTER, int MOST, bool RES>
cudaError_t launch_norm_rows(const AddNormQuantArgs &a, int tpr, int rpb, int cut, int ranks,
                        cudaStream_t s)
{
    int dev = 0, sms = 148, per_sm = 1;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t want = (a.rows + rpb - 1) / rpb;
    if (want * ranks > sms) {
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
            &per_sm, add_norm_quant_kernel<T, CLUSTER, MOST, RES>, tpr * rpb, 0);
        if (e != cudaSuccess)
            return e;
    }
    const int64_t room = (int64_t)sms * per_sm / ranks;
    return launch_early(add_norm_quant_kernel<T, CLUSTER, MOST, RES>,
                        dim3((unsigned)((want < room ? want : room) * ranks)), tpr * rpb, 0, ranks, s,
                        (const T *)a.x, (const T *)a.residual, a.gamma,
                        ((uintptr_t)a.gamma & 15u) == 0, a.rows, a.d, tpr, cut, ranks, a.eps,
                        (T *)a.total, (T *)a.y, a.codes, a.scale,
                        sectors(a.x, a.residual, a.total, a.y));
}

template <typename T, bool CLUSTER, int MOST>
cudaError_t launch_norm(const AddNormQuantArgs &a, int tpr, int rpb, int cut, int ranks,
                        cudaStream_t s)
{
    return a.residual ? launch_norm_rows<T, CLUSTER, MOST, true>(a, tpr, rpb, cut, ranks, s)
                      : launch_norm_rows<T, CLUSTER, MOST, false>(a, tpr, rpb, cut, ranks, s);
}

template <typename T>
cudaError_t launch_add_norm_quant_t(const AddNormQuantArgs &a, cudaStream_t s)
{
    if (!a.normalise)
        return a.d % kBlock == 0 ? launch_quant<T, true>(a, s) : launch_quant<T, false>(a, s);
    const int pieces = a.d / kLane;
    if (pieces <= 512) {
        const int tpr = pieces <= 8 ? 8 : pieces <= 16 ? 16 : (pieces + 31) / 32 * 32;
        if constexpr (sizeof(T) == 4)
            if (tpr <= 256)
                return launch_norm<T, false, 256>(a, tpr, 256 / tpr, a.d, 1, s);
        return launch_norm<T, false, 512>(a, tpr, tpr <= 256 ? 256 / tpr : 1, a.d, 1, s);
    }
    // whole scale blocks to each thread block of the cluster, 4096 values at a
    // time as long as eight blocks suffice
    const int nb = (a.d + kBlock - 1) / kBlock;
    int ranks = 2;
    while (ranks < 8 && (nb + ranks - 1) / ranks > 32)
        ranks *= 2;
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (a.rows * ranks > sms) {                       // no longer at once by clusters
        // resident rows up to 16384 (4096 of them: 85 us, read twice 107); in
        // float32 they would spill
        if constexpr (sizeof(T) == 2)
            if (pieces <= 1024)
                return launch_norm<T, false, 1024>(a, (pieces + 31) / 32 * 32, 1, a.d, 1, s);
        const auto kernel =
            a.residual ? add_norm_quant_long_kernel<T, true> : add_norm_quant_long_kernel<T, false>;
        return launch_early(kernel, dim3((unsigned)a.rows), kLongThreads, 0, 1, s, (const T *)a.x,
                            (const T *)a.residual, a.gamma, ((uintptr_t)a.gamma & 15u) == 0, a.d,
                            a.eps, (T *)a.total, (T *)a.y, a.codes, a.scale,
                            sectors(a.x, a.residual, a.total, a.y));
    }
    const int blocks = (nb + ranks - 1) / ranks;
    return launch_norm<T, true, 512>(a, (blocks * (kBlock / kLane) + 31) / 32 * 32, 1, blocks * kBlock,
                                ranks, s);
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
        cudaError_t e;
        if (a.dt == CSA_BF16)
            e = launch_early(quantize_weight_kernel<__nv_bfloat16>, grid, kThreads, 0, 1, s,
                             (const __nv_bfloat16 *)a.W + row0 * a.K, rows, a.K,
                             a.codes + row0 * a.K, a.scale + b0 * nbk, sectors(a.W));
        else
            e = launch_early(quantize_weight_kernel<float>, grid, kThreads, 0, 1, s,
                             (const float *)a.W + row0 * a.K, rows, a.K, a.codes + row0 * a.K,
                             a.scale + b0 * nbk, sectors(a.W));
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace csa
