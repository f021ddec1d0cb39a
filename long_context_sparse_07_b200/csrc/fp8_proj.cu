// fp8_proj.cu -- product of e4m3 activations and weights with block scales
// (csa_fp8_proj):
//   r[t, j] = sum_b As[t, b] Ws[j / 128, b] sum_{k in block b} A[t, k] W[j, k],
// blocks b of 128 inputs, float32 sums; bf16, float32 or e4m3 results.
//
// The first two kernels feed the 5th-generation tensor cores (kind::f8f6f4) from
// a TMA ring whose stages are one block of 128 inputs: the products of a block
// are summed in tensor memory from zero, and the epilogue warps add the block's
// sum, times its scale, to float32 registers while the next block's MMAs run
// into another tensor-memory buffer. (The scales are arbitrary floats, one per
// token and block, so they cannot ride in the MMA itself.)
//
// proj_rows_kernel (many tokens): tokens on the MMA's M axis, so that an
// epilogue thread owns one token and multiplies a block's sums by one scale;
// large calls by pairs of thread blocks (cta_group::2).
// proj_cols_kernel (9 to 32 tokens, and more over long rows): features on the M
// axis and tokens on N, so that one token costs a 16-wide MMA and not a 128-row
// one; the blocks of inputs are split over a cluster of thread blocks, whose
// partial results are added through distributed shared memory in the order of
// their ranks.
// proj_few_kernel (up to 8 tokens): warp MMAs straight from global memory.
// form_of says where one gives way to the next.
//
// All are launched so that they may start while the call before them ends (the
// projections of a step follow one another); the two for few tokens bring their
// weights into L2 meanwhile. In a graph the norm and projections of one token
// (13 launches) take 36.6 us so, 47.0 without the weights' prefetch and 51.2
// with plain launches; of 32 tokens 52, 53.5 and 70 us.
//
// Every wait is bounded, and a warp's lanes give up together; on expiry the
// kernel records CSA_ERR_TIMEOUT, lets its copies and products land and returns.
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "quant8.cuh"
#include "tc.cuh"
#include "tma_host.h"

namespace csa {

namespace {

constexpr int PB = 128;            // inputs per scale block = K of a ring stage
constexpr int UK = 32;             // K of one 8-bit MMA

struct ProjDev {
    const float *As, *Ws;
    void *out;
    float *out_scale;
    unsigned *err;
    int64_t M, ldo;                // ldo = groups N
    int N, K, groups, nb, las, nbo;  // las = groups nb, nbo = ceil(ldo / 128)
    csa_dtype out_dt;
    bool tma_out;
};

__device__ __forceinline__ uint32_t bf16_2(float a, float b)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *(const uint32_t *)&p;
}

// ------------------------------------------------------------ many tokens

// Tiles of 128 tokens x 128 features, or (PAIR) of 256 x 256 by two thread
// blocks whose tensor cores work as one: a block brings 128 tokens and half of
// the features, and holds the sums of its tokens and all features. Warp 0 issues
// the TMA loads, warps 1 and 2 (of the leader) in turn the MMAs of a block of
// inputs, warp 3 copies the scales, the epilogue warps each own a TMEM lane
// quarter (32 tokens) and CW features. A block's MMAs go in units of 128
// features, of which tensor memory holds four.
// What the form of a pair's tile answers to (grouped output projection, 16384
// tokens x 8 groups of 4096 -> 1024, in a graph; the board's power cap holds the
// clock near 1.55 GHz during one call, 1.2 to 1.4 during many):
// - One block's tile of 128 x 256 is bound by shared memory: per block of inputs
//   the loads write 48 KB and the MMAs read 48 KB, 750 cycles at 128 bytes a
//   cycle where the MMAs take 512. A pair writes 32 KB in each block. 545 us
//   became 510 us, now 470 to 495 (2.2 to 2.3 PFLOP/s): 806 cycles a block of
//   inputs, with the end of its tile in them (rows of 1024 inputs: 980 in bf16,
//   1140 in e4m3). Without the FMAs they are 754 (840, 845), without the MMAs 749
//   (937, 1088, at 1.93 GHz), with the loads and barriers alone 659 (748, 691).
// - From an accumulator's last MMA to the next one into it pass about 1100
//   cycles of barriers, besides its draining, which two whole-block buffers do
//   not cover: units of half a block, with two buffers each, made 302 us of 316
//   on 32768 x 8192 x 1024 (e4m3 results).
// - An issuer goes on only when its last MMA has started, and then needs some
//   450 cycles for its next barriers and issues, which the other's MMAs hide.
// - Adding the sums is bound by instructions: 128 x 256 float32 FMAs a block are
//   256 of the FMA pipe's cycles, and every warp pays its barriers and addresses
//   a block. Eight warps of 128 features, on the registers that the first
//   warpgroup gives up (40 + 2 x 232 = 3 x 168), take 510 us, sixteen of 64
//   features 590 us.
// - Scales are copied to shared memory as far ahead as the operands (read by the
//   epilogue itself, or by a warp that loads and then stores them, their latency
//   was the pace: 1000 cycles a block).
// - Results leave through shared memory by TMA stores that run beside the next
//   tile's products (stored from the registers, 32 rows to a store instruction, a
//   tile's results held its epilogue for 6400 cycles).
// - A code is the float32 sum's correctly rounded quotient, as everywhere: the
//   sum times the scale's reciprocal alone takes two FMAs less for two values
//   (289 against 301 us for the e4m3 call above), but turns ties around.
// Sustained, the same call takes 550 to 590 us.
template <bool PAIR> struct Rows {
    static constexpr int TN = PAIR ? 256 : 128;       // features of a tile
    static constexpr int TM = PAIR ? 256 : 128;       // tokens of a tile
    static constexpr int STAGES = PAIR ? 4 : 5;
    static constexpr int UPB = TN / 128;              // units of TM x 128 of a block
    static constexpr int NBUF = 4;                    // units that tensor memory holds
    // Barriers of landed blocks: twice the stages. An issuer sees every second
    // block only, and a wait tells a barrier's phases apart by their parity, so
    // that each barrier has to have the same issuer for good.
    static constexpr int FULLS = 2 * STAGES;
    static constexpr int CW = PAIR ? 128 : 64;        // features of an epilogue warp
    static constexpr int EPI = 4 * TN / CW;
    static constexpr int THREADS = 128 + 32 * EPI;
    static constexpr int REGS_DOWN = 40, REGS_UP = 232;   // of PAIR's warpgroups
    static constexpr uint32_t A_BYTES = 128 * PB, B_BYTES = 128 * PB;   // of each block
    static constexpr int UROWS = 128 / UPB;           // features a block brings to a unit
    static constexpr uint32_t OUT_BYTES = 64 * CW;    // of each epilogue warp: store boxes
    // scales of a block: when those of block it are copied, its ring stage is
    // free, so block it - STAGES is multiplied, which took the buffer of the
    // block NBUF / UPB earlier, which therefore is drained
    static constexpr int SRING = PAIR ? 8 : 16;
    static_assert(SRING >= STAGES + NBUF / UPB, "scales are overwritten only after their use");
    static constexpr int SLOT = 128 + 4;              // 128 tokens', the features' blocks'
    static constexpr size_t SMEM = 1024 + STAGES * (A_BYTES + B_BYTES) + EPI * OUT_BYTES +
                                   SRING * SLOT * 4 + EPI * 32 * 4 + 512;
};

template <bool PAIR>
__global__ void __launch_bounds__(Rows<PAIR>::THREADS, 1)
proj_rows_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                 const __grid_constant__ CUtensorMap tmO, const ProjDev a)
{
    using R = Rows<PAIR>;
    constexpr int TN = R::TN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sA = sm;
    uint8_t *sB = sm + R::STAGES * R::A_BYTES;
    uint8_t *sO = sB + R::STAGES * R::B_BYTES;
    float *sS = (float *)(sO + R::EPI * R::OUT_BYTES);
    float *sM = sS + R::SRING * R::SLOT;                    // largest magnitudes [epilogue warp][32]
    uint64_t *full = (uint64_t *)(sM + R::EPI * 32), *empty = full + R::FULLS;
    uint64_t *accf = empty + R::STAGES, *acce = accf + R::NBUF, *done = acce + R::NBUF;
    uint64_t *scaled = done + 1;                      // the second block's scales landed
    uint32_t *tmem_slot = (uint32_t *)(scaled + R::SRING);
    int *abort_flag = (int *)(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t mt = (uint32_t)((a.M + R::TM - 1) / R::TM), nt = (uint32_t)((a.N + TN - 1) / TN);
    const uint32_t ntiles = a.groups * mt * nt;       // below 2^31
    // this block's place in its pair, and the pair's (or block's) among all
    const int rank = PAIR ? (int)tc::cluster_rank() : 0;
    const uint32_t first = PAIR ? blockIdx.x / 2 : blockIdx.x;
    const uint32_t stride = PAIR ? gridDim.x / 2 : gridDim.x;

    if (threadIdx.x == 0) {
        for (int i = 0; i < R::FULLS; i++)
            // the loads (in the leader both blocks'), each lane's scales, and word
            // that the other block's scales are there
            tc::mbar_init(&full[i], 1 + 32 + (PAIR ? 1 : 0));
        for (int i = 0; i < R::SRING; i++)
            tc::mbar_init(&scaled[i], 32);
        for (int i = 0; i < R::STAGES; i++)
            tc::mbar_init(&empty[i], 1);
        for (int i = 0; i < R::NBUF; i++) {
            tc::mbar_init(&accf[i], 1);
            tc::mbar_init(&acce[i], 8);               // epilogue warps of a unit
        }
        tc::mbar_init(done, 2);                       // both issuers
        tc::fence_mbar_init();
        *abort_flag = 0;
        tc::tma_prefetch_desc(&tmA);
        tc::tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tc::tmem_alloc_pair(tmem_slot, 512);
            tc::tmem_relinquish_pair();
        } else {
            tc::tmem_alloc(tmem_slot, 512);
            tc::tmem_relinquish();
        }
    }
    tc::fence_before();
    __syncthreads();
    if constexpr (PAIR)
        tc::cluster_sync();                           // the other block's barriers stand
    tc::fence_after();
    tc::grid_let_next();
    tc::grid_wait();
    const uint32_t tmem = *tmem_slot;
    volatile int *abortv = abort_flag;
    // tile t -> (group, m tile, n tile), n fastest: the blocks working at one
    // time share their tokens through L2
    auto coords = [&](uint32_t t, int &grp, int &mi, int &ni) {
        const uint32_t r = t / nt;
        ni = (int)(t - r * nt);
        grp = (int)(r / mt);
        mi = (int)(r - grp * mt);
    };

    auto commit = [](uint64_t *bar) {
        if constexpr (PAIR)
            tc::mma_commit_pair(bar);
        else
            tc::mma_commit(bar);
    };

    if (warp < 4) {
        if constexpr (PAIR)
            tc::regs_down<R::REGS_DOWN>();
        if (warp == 0) {
            // ---------------- operands
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t t = first; t < ntiles && ok; t += stride) {
                int grp, mi, ni;
                coords(t, grp, mi, ni);
                const int ax = grp * a.K, ay = mi * R::TM + rank * 128;
                const int wy = grp * a.N + ni * TN + rank * R::UROWS;
                for (int b = 0; b < a.nb; b++, it++) {
                    const int st = it % R::STAGES;
                    if (it >= R::STAGES &&
                        !tc::mbar_wait_warp(&empty[st], ((it / R::STAGES) - 1) & 1, abortv)) {
                        ok = false;
                        break;
                    }
                    if (tc::elect_one()) {
                        uint64_t *landed = &full[it % R::FULLS];
                        if constexpr (PAIR) {
                            if (rank == 0)
                                tc::mbar_arrive_expect_tx(landed, 2 * (R::A_BYTES + R::B_BYTES));
                            const uint32_t at = tc::cluster_map(landed, 0);
                            tc::tma_load_2d_pair(sA + st * R::A_BYTES, &tmA, at, ax + b * PB, ay);
#pragma unroll
                            for (int h = 0; h < R::UPB; h++)
                                tc::tma_load_2d_pair(sB + st * R::B_BYTES + h * R::UROWS * PB, &tmW,
                                                     at, b * PB, wy + h * 128);
                        } else {
                            tc::mbar_arrive_expect_tx(landed, R::A_BYTES + R::B_BYTES);
                            tc::tma_load_2d(sA + st * R::A_BYTES, &tmA, landed, ax + b * PB, ay);
                            tc::tma_load_2d(sB + st * R::B_BYTES, &tmW, landed, b * PB, wy);
                        }
                    }
                    __syncwarp();
                }
            }
            if (!ok && lane == 0) {
                *abort_flag = 1;
                report(a.err, CSA_ERR_TIMEOUT, K_FP8_PROJ, blockIdx.x, 0);
            }
            // let the copies in flight land before the block exits (the leader
            // knows of both blocks')
            volatile int never = 0;
            for (uint32_t j = it > R::STAGES ? it - R::STAGES : 0; j < it; j++) {
                if (rank == 0)
                    static_cast<void>(tc::mbar_wait(&full[j % R::FULLS], (j / R::FULLS) & 1, &never,
                                                    200000000ull));
                // and the leader's commits arrive
                if (PAIR)
                    static_cast<void>(tc::mbar_wait(&empty[j % R::STAGES], (j / R::STAGES) & 1,
                                                    &never, 200000000ull));
            }
        } else if (warp == 3) {
            // ---------------- scales: four tokens' to a lane, and the features'
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t t = first; t < ntiles && ok; t += stride) {
                int grp, mi, ni;
                coords(t, grp, mi, ni);
                const int64_t r0 = (int64_t)mi * R::TM + rank * 128 + lane;
                const int rows = (int)(a.M - r0 < 128 ? a.M - r0 : 128);   // may be negative
                const float *as = a.As + (rows > 0 ? r0 * a.las + (int64_t)grp * a.nb : 0);
                const bool has_w = lane < TN / 128 && ni * TN + lane * 128 < a.N;
                const float *ws =
                    a.Ws + (has_w ? (int64_t)((grp * a.N + ni * TN) / PB + lane) * a.nb : 0);
                for (int b = 0; b < a.nb; b++, it++) {
                    const int st = it % R::STAGES;
                    if (it >= R::STAGES &&
                        !tc::mbar_wait_warp(&empty[st], ((it / R::STAGES) - 1) & 1, abortv)) {
                        ok = false;
                        break;
                    }
                    // zeros (from any valid address) behind the last row and feature
                    float *slot = sS + it % R::SRING * R::SLOT;
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        tc::cp_async4(slot + i * 32 + lane,
                                      i * 32 < rows ? as + (int64_t)i * 32 * a.las + b : a.As,
                                      i * 32 < rows ? 4 : 0);
                    if (lane < TN / 128)
                        tc::cp_async4(slot + 128 + lane, ws + b, has_w ? 4 : 0);
                    tc::cp_async_arrive(rank == 0 ? &full[it % R::FULLS] : &scaled[it % R::SRING]);
                }
            }
            if (!ok && lane == 0) {
                *abort_flag = 1;
                report(a.err, CSA_ERR_TIMEOUT, K_FP8_PROJ, blockIdx.x, 6);
            }
            tc::cp_async_wait_all();
        } else if (rank == 0) {
            // ---------------- MMA issuers: the whole warp runs the loop (so that
            // what it computes stays in uniform registers), one lane issues
            constexpr uint32_t idesc = tc::idesc_e4m3(R::TM, 128);
            const uint64_t dA = tc::sdesc_sw128(tc::smem_u32(sA)), dB = tc::sdesc_sw128(tc::smem_u32(sB));
            const uint32_t total = (ntiles - first + stride - 1) / stride * a.nb;
            bool ok = true;
            for (uint32_t it = warp - 1; it < total; it += 2) {
                const uint32_t st = it % R::STAGES, buf0 = it * R::UPB % R::NBUF;
                const uint32_t pa = (it * R::UPB / R::NBUF - 1) & 1, pf = (it / R::FULLS) & 1;
                uint64_t *landed = &full[it % R::FULLS];
                // all barriers tried before any answer is used: one round trip to
                // shared memory
                bool free[R::UPB];
#pragma unroll
                for (int h = 0; h < R::UPB; h++)
                    free[h] = it * R::UPB < R::NBUF || tc::mbar_test_wait(&acce[buf0 + h], pa);
                const bool in = tc::mbar_test_wait(landed, pf);
#pragma unroll
                for (int h = 0; h < R::UPB; h++)
                    free[h] = tc::warp_agrees(free[h]);
                ok = tc::warp_agrees(in) || tc::mbar_wait_warp(landed, pf, abortv);
#pragma unroll
                for (int h = 0; h < R::UPB; h++) {
                    ok = ok && (free[h] || tc::mbar_wait_warp(&acce[buf0 + h], pa, abortv));
                    if (!ok)
                        break;
                    tc::fence_after();
                    if (tc::elect_one()) {
                        const uint32_t d = tmem + (buf0 + h) * 128;
                        const uint64_t da = dA + ((st * R::A_BYTES) >> 4);
                        const uint64_t db = dB + ((st * R::B_BYTES + h * R::UROWS * PB) >> 4);
#pragma unroll
                        for (int kk = 0; kk < PB / UK; kk++) {
                            if constexpr (PAIR)
                                tc::mma_f8_pair(d, da + (kk * UK >> 4), db + (kk * UK >> 4), idesc,
                                                kk != 0);
                            else
                                tc::mma_f8(d, da + (kk * UK >> 4), db + (kk * UK >> 4), idesc,
                                           kk != 0);
                        }
                        if (h == R::UPB - 1)
                            commit(&empty[st]);
                        commit(&accf[buf0 + h]);
                    }
                    __syncwarp();
                }
                if (!ok)
                    break;
            }
            if (!ok && lane == 0) {
                *abort_flag = 1;
                report(a.err, CSA_ERR_TIMEOUT, K_FP8_PROJ, blockIdx.x, 1);
            }
            __syncwarp();
            if (tc::elect_one()) {
                if constexpr (PAIR)
                    tc::mma_commit_pair_own(done);
                else
                    tc::mma_commit(done);
            }
            __syncwarp();
            volatile int never = 0;
            static_cast<void>(tc::mbar_wait(done, 0, &never, 200000000ull));
        } else if (warp == 1) {
            // ---------------- the second block's word to the leader: a block's MMAs
            // wait for both blocks' scales, so that they are there when the sums
            // are, and nobody runs ahead of them
            const uint32_t total = (ntiles - first + stride - 1) / stride * a.nb;
            bool ok = true;
            for (uint32_t it = 0; it < total && ok; it++) {
                ok = tc::mbar_wait_warp(&scaled[it % R::SRING], (it / R::SRING) & 1, abortv);
                if (ok && tc::elect_one())
                    tc::mbar_arrive_cluster(tc::cluster_map(&full[it % R::FULLS], 0));
                __syncwarp();
            }
            if (!ok && lane == 0) {
                *abort_flag = 1;
                report(a.err, CSA_ERR_TIMEOUT, K_FP8_PROJ, blockIdx.x, 7);
            }
        }
        __syncwarp();
    } else {
        if constexpr (PAIR)
            tc::regs_up<R::REGS_UP>();
        // ---------------- epilogue: lane quarter warp % 4 = 32 tokens, the
        // features c0 .. c0 + CW - 1 of the tile
        constexpr int CW = R::CW, BOXES = CW / 64;    // boxes of a warp: 32 tokens x 128 bytes
        const int e = warp - 4, q4 = warp & 3, c0 = (e >> 2) * CW;
        const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16) + c0 % 128;
        const uint32_t acce0 = PAIR ? tc::cluster_map(acce, 0) : 0u;   // the leader's
        uint8_t *stage = sO + e * R::OUT_BYTES;
        // barrier with the warp of the other half of a scale's block (CW = 64)
        const int other = 1 + (e >> 3) * 4 + q4;
        uint32_t it = 0;
        bool sums = false;                            // block it seen to be summed
        auto look = [&] {
            const uint32_t u = it * R::UPB + c0 / 128;  // this warp's unit of block it
            sums = tc::mbar_test_wait(&accf[u % R::NBUF], (u / R::NBUF) & 1);
        };
        for (uint32_t t = first; t < ntiles; t += stride) {
            float2 acc[CW / 2];
#pragma unroll
            for (int j = 0; j < CW / 2; j++)
                acc[j] = make_float2(0.f, 0.f);
            bool ok = true;
            look();
            for (int b = 0; b < a.nb; b++) {
                const uint32_t u = it * R::UPB + c0 / 128, buf = u % R::NBUF;
                ok = tc::warp_agrees(sums) ||
                     tc::mbar_wait_warp(&accf[buf], (u / R::NBUF) & 1, abortv);
                if (!ok)
                    break;
                tc::fence_after();
                uint32_t v[2][32];
                tc::tmem_ld32(lane_addr + buf * 128, v[0]);
                const float *slot = sS + it % R::SRING * R::SLOT;
                const float s = slot[q4 * 32 + lane] * slot[128 + c0 / 128];
                const float2 s2 = make_float2(s, s);
                it++;
#pragma unroll
                for (int c = 0; c < CW / 32; c++) {
                    tc::tmem_ld_wait(v[c & 1]);
                    if (c + 1 < CW / 32) {
                        tc::tmem_ld32(lane_addr + buf * 128 + (c + 1) * 32, v[(c + 1) & 1]);
                    } else {
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (PAIR)
                                tc::mbar_arrive_cluster(acce0 + buf * 8);
                            else
                                tc::mbar_arrive(&acce[buf]);
                        }
                        look();                       // answered while the last sums are added
                    }
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        acc[c * 16 + j] =
                            __ffma2_rn(make_float2(__uint_as_float(v[c & 1][2 * j]),
                                                   __uint_as_float(v[c & 1][2 * j + 1])),
                                       s2, acc[c * 16 + j]);
                }
            }
            if (!ok) {
                *abort_flag = 1;
                report(a.err, CSA_ERR_TIMEOUT, K_FP8_PROJ, blockIdx.x, 2);
            }
            int grp, mi, ni;
            coords(t, grp, mi, ni);
            const int n0 = ni * TN + c0;              // first feature, within the group
            const int cols = a.N - n0 < CW ? a.N - n0 : CW;   // may be negative
            const int col = grp * a.N + n0, y0 = mi * R::TM + rank * 128 + q4 * 32;
            // in the store's 128-byte swizzle: piece p of row r at p ^ r % 8
            auto put = [&](uint8_t *box, int piece, uint32_t w0, uint32_t w1, uint32_t w2,
                           uint32_t w3) {
                *(uint4 *)(box + lane * 128 + ((piece ^ (lane & 7)) << 4)) =
                    make_uint4(w0, w1, w2, w3);
            };
            auto send = [&](const uint8_t *box, int from) {
                if (lane == 0 && y0 < a.M && from < cols)
                    tc::tma_store_2d(&tmO, box, col + from, y0);
            };
            if (a.out_dt == CSA_E4M3) {
                // features behind the last have sums of zero, which an infinite
                // scale makes NaN
                if (cols < CW)
#pragma unroll
                    for (int j = 0; j < CW / 2; j++)
                        if (2 * j >= cols)             // N is a multiple of 16
                            acc[j] = make_float2(0.f, 0.f);
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < CW / 2; j++)
                    m = max_mag(m, acc[j]);
                uint8_t *box = stage;
                if (lane == 0)
                    tc::bulk_wait_read();
                if constexpr (CW == 64) {
                    // a scale's block is two warps': both fill the first one's box
                    box = sO + (e & ~4) * R::OUT_BYTES;
                    sM[e * 32 + lane] = m;
                    if (tc::named_bar_or(other, 64, !ok))
                        break;
                    m = max_nan(m, sM[(e ^ 4) * 32 + lane]);
                } else {
                    __syncwarp();
                    if (!ok)
                        break;
                }
                const bool lead = CW == 128 || (e & 4) == 0;
                const float sc = block_scale(m);
                if (lead && y0 + lane < a.M && cols > 0)
                    a.out_scale[(int64_t)(y0 + lane) * a.nbo + col / 128] = sc;
                uint32_t w[CW / 4];
                codes_of<CW / 4>(acc, sc, w);
#pragma unroll
                for (int j = 0; j < CW / 16; j++)
                    put(box, (lead ? 0 : 4) + j, w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                tc::fence_async_shared();
                if constexpr (CW == 64)
                    tc::named_bar_sync(other, 64);
                else
                    __syncwarp();
                if (lead) {
                    send(box, 0);
                    if (lane == 0)
                        tc::bulk_commit();
                }
                continue;
            }
            if (!ok)
                break;
            // 64 features to a box in bf16, 32 in float32, whose warp goes twice
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const bool half = a.out_dt == CSA_BF16;
                if (h && half)
                    break;
                if (lane == 0)
                    tc::bulk_wait_read();
                __syncwarp();
                if (half) {
#pragma unroll
                    for (int j = 0; j < CW / 8; j++)
                        put(stage + j / 8 * 4096, j % 8, bf16_2(acc[4 * j].x, acc[4 * j].y),
                            bf16_2(acc[4 * j + 1].x, acc[4 * j + 1].y),
                            bf16_2(acc[4 * j + 2].x, acc[4 * j + 2].y),
                            bf16_2(acc[4 * j + 3].x, acc[4 * j + 3].y));
                } else {
#pragma unroll
                    for (int j = 0; j < CW / 8; j++) {
                        const float2 p = acc[h * CW / 4 + 2 * j], q = acc[h * CW / 4 + 2 * j + 1];
                        put(stage + j / 8 * 4096, j % 8, __float_as_uint(p.x), __float_as_uint(p.y),
                            __float_as_uint(q.x), __float_as_uint(q.y));
                    }
                }
                if (a.tma_out) {
                    tc::fence_async_shared();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < BOXES; i++)
                        send(stage + i * 4096, h * CW / 2 + i * (half ? 64 : 32));
                    if (lane == 0)
                        tc::bulk_commit();
                } else {
                    // rows that no tensor map describes (not a multiple of 16 bytes):
                    // 32 lanes store a box's row
                    __syncwarp();
#pragma unroll 1
                    for (int r = 0; r < 32 && y0 + r < a.M; r++) {
#pragma unroll
                        for (int i = 0; i < BOXES; i++) {
                            const uint32_t w = *(const uint32_t *)(stage + i * 4096 + r * 128 +
                                                                   ((lane >> 2 ^ (r & 7)) << 4) +
                                                                   (lane & 3) * 4);
                            const int f = half ? i * 64 + 2 * lane : h * CW / 2 + i * 32 + lane;
                            const int64_t o = (int64_t)(y0 + r) * a.ldo + col + f;
                            if (!half) {
                                if (f < cols)
                                    ((uint32_t *)a.out)[o] = w;
                            } else {
                                if (f < cols)
                                    ((uint16_t *)a.out)[o] = (uint16_t)w;
                                if (f + 1 < cols)
                                    ((uint16_t *)a.out)[o + 1] = (uint16_t)(w >> 16);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (lane == 0)
            tc::bulk_wait_all();
    }
    tc::fence_before();
    __syncthreads();
    if constexpr (PAIR)
        tc::cluster_sync();                           // nothing more arrives from the other block
    if (warp == 1) {
        tc::fence_after();
        if constexpr (PAIR)
            tc::tmem_dealloc_pair(tmem, 512);
        else
            tc::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------ few tokens

// Tiles of 128 features x TT tokens, the blocks of inputs split over the
// cluster's thread blocks. Warps as above, with four epilogue warps (a lane
// quarter = 32 features each); an epilogue thread owns one feature and all TT
// tokens. In the end a warp takes one token at a time and adds the cluster's
// partial results of its 128 features. Two blocks of threads fit an SM.
constexpr int kMaxSplit = 8;       // thread blocks of a cluster

template <int TT> struct Cols {
    static constexpr int STAGES = TT == 64 ? 4 : 5;
    static constexpr int FULLS = 2 * STAGES;          // as above
    static constexpr int NBUF = 4;
    static constexpr int THREADS = 256;
    static constexpr uint32_t W_BYTES = 128 * PB, T_BYTES = TT * PB;
    static constexpr uint32_t TMEM = NBUF * TT;
    static constexpr int SRING = STAGES + NBUF;       // as above
    static constexpr int SLOT = TT + 4;               // the tokens' scales, the features'
    static constexpr size_t RING = STAGES * (W_BYTES + T_BYTES);
    static constexpr size_t SMEM = 1024 + RING + SRING * SLOT * 4 + 256;
    static_assert(RING >= (size_t)TT * 128 * 4, "partial results reuse the ring");
};

template <int TT>
__global__ void __launch_bounds__(Cols<TT>::THREADS, 2)
proj_cols_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                 const ProjDev a, const int split)
{
    using C = Cols<TT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sW = sm;
    uint8_t *sT = sm + C::STAGES * C::W_BYTES;
    float *sS = (float *)(sm + C::RING);
    uint64_t *full = (uint64_t *)(sS + C::SRING * C::SLOT), *empty = full + C::FULLS;
    uint64_t *accf = empty + C::STAGES, *acce = accf + C::NBUF, *done = acce + C::NBUF;
    uint32_t *tmem_slot = (uint32_t *)(done + 1);
    int *abort_flag = (int *)(tmem_slot + 1);
    float *partial = (float *)sm;                     // [TT][128], once the ring is drained

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = split > 1 ? (int)tc::cluster_rank() : 0;
    const uint32_t tile = blockIdx.x / split;
    const uint32_t ft = (a.N + 127) / 128, tt = (uint32_t)((a.M + TT - 1) / TT);
    const int n0 = (int)(tile % ft) * 128;            // first feature, within the group
    const int t0 = (int)(tile / ft % tt) * TT;        // first token
    const int grp = (int)(tile / ft / tt);
    const int b0 = (int)((int64_t)a.nb * rank / split);
    const int b1 = (int)((int64_t)a.nb * (rank + 1) / split);
    const uint32_t nblk = (uint32_t)(b1 - b0);
    const int64_t fb = ((int64_t)grp * a.N + n0) / PB;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::FULLS; i++)
            tc::mbar_init(&full[i], 1 + 32);          // the TMA loads, each lane's scales
        for (int i = 0; i < C::STAGES; i++)
            tc::mbar_init(&empty[i], 1);
        for (int i = 0; i < C::NBUF; i++) {
            tc::mbar_init(&accf[i], 1);
            tc::mbar_init(&acce[i], 4);
        }
        tc::mbar_init(done, 2);                       // both issuers
        tc::fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, C::TMEM);
        tc::tmem_relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    tc::grid_let_next();
    // the weight does not wait for the call before this one; as much as the ring
    // holds (all of it: 12.0 against 11.0 us for 8 x 32768 x 1024 alone and cold)
    if (warp == 4 && tc::elect_one())
        for (int b = b0; b < b1 && b < b0 + C::STAGES; b++)
            tc::prefetch_l2_2d(&tmW, b * PB, grp * a.N + n0);
    tc::grid_wait();
    const uint32_t tmem = *tmem_slot;
    volatile int *abortv = abort_flag;

    if (warp == 0 || warp == 3) {
        // ---------------- operands (warp 0) and scales (warp 3)
        const int rows = (int)(a.M - t0 < TT ? a.M - t0 : TT);
        const float *as = a.As + (lane < rows ? (int64_t)(t0 + lane) * a.las : 0) +
                          (int64_t)grp * a.nb + b0;
        const float *ws = a.Ws + fb * a.nb + b0;
        uint32_t it = 0;
        for (; it < nblk; it++) {
            const uint32_t st = it % C::STAGES;
            if (it >= C::STAGES &&
                !tc::mbar_wait_warp(&empty[st], ((it / C::STAGES) - 1) & 1, abortv)) {
                if (lane == 0) {
                    *abort_flag = 1;
                    report(a.err, CSA_ERR_TIMEOUT, K_FP8_PROJ, blockIdx.x, 3);
                }
                break;
            }
            uint64_t *landed = &full[it % C::FULLS];
            if (warp == 0) {
                if (tc::elect_one()) {
                    const int x = (b0 + (int)it) * PB;
                    tc::mbar_arrive_expect_tx(landed, C::W_BYTES + C::T_BYTES);
                    tc::tma_load_2d(sW + st * C::W_BYTES, &tmW, landed, x, grp * a.N + n0);
                    tc::tma_load_2d(sT + st * C::T_BYTES, &tmA, landed, grp * a.K + x, t0);
                }
                __syncwarp();
            } else {
                // zeros (from any valid address) behind the last token
                float *slot = sS + it % C::SRING * C::SLOT;
#pragma unroll
                for (int i = 0; i < TT; i += 32)
                    if (i + lane < TT)
                        tc::cp_async4(slot + i + lane,
                                      i + lane < rows ? as + (int64_t)i * a.las + it : a.As,
                                      i + lane < rows ? 4 : 0);
                if (lane == 0)
                    tc::cp_async4(slot + TT, ws + it, 4);
                tc::cp_async_arrive(landed);
            }
        }
        // let the copies in flight land before the block exits
        volatile int never = 0;
        if (warp == 3)
            tc::cp_async_wait_all();
        else
            for (uint32_t j = it > C::STAGES ? it - C::STAGES : 0; j < it; j++)
                static_cast<void>(tc::mbar_wait(&full[j % C::FULLS], (j / C::FULLS) & 1, &never,
                                                200000000ull));
    } else if (warp < 3) {
        // ---------------- MMA issuers
        constexpr uint32_t idesc = tc::idesc_e4m3(128, TT);
        const uint64_t dW = tc::sdesc_sw128(tc::smem_u32(sW)), dT = tc::sdesc_sw128(tc::smem_u32(sT));
        for (uint32_t it = warp - 1; it < nblk; it += 2) {
            const uint32_t st = it % C::STAGES, buf = it % C::NBUF;
            const uint32_t pa = (it / C::NBUF - 1) & 1, pf = (it / C::FULLS) & 1;
            uint64_t *landed = &full[it % C::FULLS];
            const bool empty_buf = it < C::NBUF || tc::mbar_test_wait(&acce[buf], pa);
            const bool in = tc::mbar_test_wait(landed, pf);
            const bool free = tc::warp_agrees(empty_buf);
            bool ok = tc::warp_agrees(in) || tc::mbar_wait_warp(landed, pf, abortv);
            ok = ok && (free || tc::mbar_wait_warp(&acce[buf], pa, abortv));
            if (!ok) {
                if (lane == 0) {
                    *abort_flag = 1;
                    report(a.err, CSA_ERR_TIMEOUT, K_FP8_PROJ, blockIdx.x, 4);
                }
                break;
            }
            tc::fence_after();
            if (tc::elect_one()) {
                const uint64_t dw = dW + ((st * C::W_BYTES) >> 4), dt = dT + ((st * C::T_BYTES) >> 4);
#pragma unroll
                for (int kk = 0; kk < PB / UK; kk++)
                    tc::mma_f8(tmem + buf * TT, dw + (kk * UK >> 4), dt + (kk * UK >> 4), idesc,
                               kk != 0);
                tc::mma_commit(&empty[st]);
                tc::mma_commit(&accf[buf]);
            }
            __syncwarp();
        }
        __syncwarp();
        if (tc::elect_one())
            tc::mma_commit(done);
        __syncwarp();
        volatile int never = 0;
        static_cast<void>(tc::mbar_wait(done, 0, &never, 200000000ull));
    } else {
        // ---------------- epilogue: feature n0 + 32 (warp % 4) + lane
        constexpr int CH = TT < 32 ? TT : 32;          // columns per load
        const int q4 = warp & 3;
        const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16);
        float2 acc[TT / 2];
#pragma unroll
        for (int j = 0; j < TT / 2; j++)
            acc[j] = make_float2(0.f, 0.f);
        for (uint32_t it = 0; it < nblk; it++) {
            const uint32_t buf = it % C::NBUF;
            if (!tc::mbar_wait_warp(&accf[buf], (it / C::NBUF) & 1, abortv)) {
                *abort_flag = 1;
                report(a.err, CSA_ERR_TIMEOUT, K_FP8_PROJ, blockIdx.x, 5);
                break;
            }
            tc::fence_after();
            // landed before the MMAs of this block were let go
            const float *slot = sS + it % C::SRING * C::SLOT;
            const float2 w = make_float2(slot[TT], slot[TT]);
#pragma unroll
            for (int c = 0; c < TT / CH; c++) {
                uint32_t v[CH];
                tc::tmem_get(lane_addr + buf * TT + c * CH, v);
#pragma unroll
                for (int j = 0; j < CH; j += 4) {
                    const float4 x = *(const float4 *)&slot[c * CH + j];
                    float2 &lo = acc[(c * CH + j) / 2], &hi = acc[(c * CH + j) / 2 + 1];
                    lo = __ffma2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])),
                                    __fmul2_rn(make_float2(x.x, x.y), w), lo);
                    hi = __ffma2_rn(
                        make_float2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])),
                        __fmul2_rn(make_float2(x.z, x.w), w), hi);
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(&acce[buf]);
        }
        // the last accumulator's commit covers every MMA of its issuer, the one
        // before the other's: the ring is drained
#pragma unroll
        for (int j = 0; j < TT / 2; j++) {
            partial[2 * j * 128 + q4 * 32 + lane] = acc[j].x;
            partial[(2 * j + 1) * 128 + q4 * 32 + lane] = acc[j].y;
        }
    }
    tc::fence_before();
    __syncthreads();
    if (split > 1)
        tc::cluster_sync();
    // token t0 + j, features n0 + 4 lane .. + 3
    const int nw = C::THREADS / 32;
    for (int j = rank + split * warp; j < TT && t0 + j < a.M; j += split * nw) {
        const float *src = partial + j * 128 + lane * 4;
        float4 v;
        if (split > 1) {
            float4 u[kMaxSplit];                       // all in flight before the first is added
#pragma unroll
            for (int p = 0; p < kMaxSplit; p++)
                if (p < split)
                    u[p] = tc::cluster_ld4(src, p);
            v = u[0];
#pragma unroll
            for (int p = 1; p < kMaxSplit; p++)
                if (p < split)
                    v = make_float4(v.x + u[p].x, v.y + u[p].y, v.z + u[p].z, v.w + u[p].w);
        } else {
            v = *(const float4 *)src;
        }
        const int cols = a.N - n0 - lane * 4;         // features of this lane that exist
        const int64_t t = t0 + j, o = t * a.ldo + (int64_t)grp * a.N + n0 + lane * 4;
        if (a.out_dt == CSA_E4M3) {
            // features behind the last have sums of zero, which an infinite scale
            // makes NaN; N is a multiple of 16
            if (cols <= 0)
                v = make_float4(0.f, 0.f, 0.f, 0.f);
            const float2 p[2] = {make_float2(v.x, v.y), make_float2(v.z, v.w)};
            float m = max_mag(max_mag(0.f, p[0]), p[1]);
#pragma unroll
            for (int f = 16; f > 0; f >>= 1)
                m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, f));
            const float s = block_scale(m);
            uint32_t w[1];
            codes_of<1>(p, s, w);
            if (lane == 0)
                a.out_scale[t * a.nbo + fb] = s;
            if (cols > 0)
                *(uint32_t *)((uint8_t *)a.out + o) = w[0];
        } else if (a.ldo % 4 == 0) {
            if (cols > 0) {
                if (a.out_dt == CSA_BF16)
                    *(uint2 *)((__nv_bfloat16 *)a.out + o) =
                        make_uint2(bf16_2(v.x, v.y), bf16_2(v.z, v.w));
                else
                    *(float4 *)((float *)a.out + o) = v;
            }
        } else {
            const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (i < cols) {
                    if (a.out_dt == CSA_BF16)
                        ((__nv_bfloat16 *)a.out)[o + i] = __float2bfloat16_rn(e[i]);
                    else
                        ((float *)a.out)[o + i] = e[i];
                }
            }
        }
    }
    // no block leaves while another may still read its shared memory
    if (split > 1) {
        __syncwarp();
        tc::cluster_sync();
    }
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, C::TMEM);
    }
}

// ------------------------------------------------------------ very few tokens

// Up to 8 tokens: the weight's bytes are all that counts, and what a call waits
// for. A warp takes 16 features and a share of the input blocks: 16-byte loads
// of the weight straight into the fragments of 16 x 8 x 32 warp MMAs (no tensor
// memory to allocate, no ring to fill: one token by 1024 x 4096 takes 3.3 us in
// a graph, against 4.0 us through the kernel above), the loads of four blocks
// in flight before the first is used. Which inputs share an MMA does not matter
// as long as both operands agree: lane (g, t) = (lane / 4, lane % 4) holds
// inputs 16 t .. 16 t + 15 of every 64, eight for each of two MMAs, of features
// g and g + 8 and of token g. A block of threads is rg groups of 16 features x
// ks shares of the inputs, whose sums meet in shared memory in the order of the
// shares.
constexpr int kFewTokens = 8, kFewWarps = 16, kFewAhead = 4;
constexpr int kFewLd = kFewTokens + 1;                // padded against bank conflicts

__device__ __forceinline__ uint4 ld_stream(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ void mma_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__global__ void __launch_bounds__(32 * kFewWarps)
proj_few_kernel(const uint8_t *A, const uint8_t *W, const ProjDev a,
                const int ks)
{
    extern __shared__ float sums[];                   // [ks][16 rg][kFewLd]
    tc::grid_let_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rg = blockDim.x / 32 / ks, share = warp / rg, group = warp % rg;
    const int rows = 16 * rg;                         // features of the block
    const int ft = (a.N + rows - 1) / rows;
    const int grp = blockIdx.x / ft, n0 = blockIdx.x % ft * rows;
    const int f0 = n0 + 16 * group;                   // the warp's first feature, in its group
    const int b0 = (int)((int64_t)a.nb * share / ks), b1 = (int)((int64_t)a.nb * (share + 1) / ks);
    const int M = (int)a.M;
    const bool r0 = f0 + g < a.N, r1 = f0 + g + 8 < a.N, tok = g < M;
    const uint8_t *w0 = W + ((int64_t)grp * a.N + (r0 ? f0 + g : 0)) * a.K;
    const uint8_t *w1 = W + ((int64_t)grp * a.N + (r1 ? f0 + g + 8 : 0)) * a.K;
    const uint8_t *x0 = A + ((int64_t)(tok ? g : 0) * a.groups + grp) * a.K;
    const float *as = a.As + (int64_t)grp * a.nb;
    const float *ws = a.Ws + ((int64_t)grp * a.N + (f0 < a.N ? f0 : 0)) / PB * a.nb;
    // the weight does not wait for the call before this one
    for (int k = b0 * PB + (lane & 7) * PB; k < b1 * PB && k < a.K; k += 8 * PB)
#pragma unroll
        for (int r = lane >> 3; r < 16; r += 4)
            if (f0 + r < a.N)
                tc::prefetch_l2(W + ((int64_t)grp * a.N + f0 + r) * a.K + k);
    tc::grid_wait();
    const uint4 zero = make_uint4(0, 0, 0, 0);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};              // (feature g + 8 (e / 2), token 2 t + e % 2)
    for (int b = b0; b < b1; b += kFewAhead) {
        uint4 wa[kFewAhead][2], wb[kFewAhead][2];
        float sw[kFewAhead], sa[kFewAhead][2];
#pragma unroll
        for (int i = 0; i < kFewAhead; i++) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int k = (b + i) * PB + h * 64 + t * 16;
                const bool in = b + i < b1 && k < a.K;
                wa[i][h] = in && r0 ? ld_stream(w0 + k) : zero;
                wb[i][h] = in && r1 ? ld_stream(w1 + k) : zero;
            }
            sw[i] = b + i < b1 ? ws[b + i] : 0.f;
#pragma unroll
            for (int e = 0; e < 2; e++)
                sa[i][e] =
                    b + i < b1 && 2 * t + e < M ? as[(int64_t)(2 * t + e) * a.las + b + i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kFewAhead; i++) {
            if (b + i >= b1)
                break;
            float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int k = (b + i) * PB + h * 64 + t * 16;
                const uint4 x = tok && k < a.K ? *(const uint4 *)(x0 + k) : zero;
                mma_16x8x32(p, wa[i][h].x, wb[i][h].x, wa[i][h].y, wb[i][h].y, x.x, x.y);
                mma_16x8x32(p, wa[i][h].z, wb[i][h].z, wa[i][h].w, wb[i][h].w, x.z, x.w);
            }
#pragma unroll
            for (int e = 0; e < 4; e++)
                acc[e] = fmaf(p[e], sa[i][e & 1] * sw[i], acc[e]);
        }
    }
    float *mine = sums + (share * rows + 16 * group) * kFewLd;
#pragma unroll
    for (int e = 0; e < 4; e++)
        mine[(g + 8 * (e >> 1)) * kFewLd + 2 * t + (e & 1)] = acc[e];
    __syncthreads();
    for (int i = threadIdx.x; i < rows * M; i += blockDim.x) {
        const int m = i / rows, f = i - m * rows;
        if (n0 + f >= a.N)
            continue;
        float v = 0.f;
        for (int q = 0; q < ks; q++)
            v += sums[(q * rows + f) * kFewLd + m];
        const int64_t o = m * a.ldo + (int64_t)grp * a.N + n0 + f;
        if (a.out_dt == CSA_BF16)
            ((__nv_bfloat16 *)a.out)[o] = __float2bfloat16_rn(v);
        else
            ((float *)a.out)[o] = v;
    }
}

// ------------------------------------------------------------ launches

int sm_count()
{
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

template <bool PAIR>
cudaError_t launch_rows(const Fp8ProjArgs &g, ProjDev d, int sms, cudaStream_t s)
{
    using R = Rows<PAIR>;
    CUtensorMap tmA, tmW, tmO;
    if (!make_tmap_2d(&tmA, g.A, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)g.M,
                      (uint64_t)g.groups * g.K, 128) ||
        !make_tmap_2d(&tmW, g.W, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)d.ldo, (uint64_t)g.K,
                      R::UROWS))
        return cudaErrorInvalidValue;
    const int es = g.out_dt == CSA_F32 ? 4 : g.out_dt == CSA_BF16 ? 2 : 1;
    d.tma_out = d.ldo * es % 16 == 0;
    tmO = tmA;
    if (d.tma_out &&
        !make_tmap_2d(&tmO, g.out,
                      g.out_dt == CSA_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                      : g.out_dt == CSA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                      es, (uint64_t)g.M, (uint64_t)d.ldo, 32))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(proj_rows_kernel<PAIR>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)R::SMEM);
    if (e != cudaSuccess)
        return e;
    const int64_t tiles = (g.M + R::TM - 1) / R::TM * ((g.N + R::TN - 1) / R::TN) * g.groups;
    if (tiles > INT32_MAX)
        return cudaErrorInvalidConfiguration;
    if (PAIR) {
        // the warpgroups' shares (regs_down, regs_up) come out of the launch's
        // registers: with fewer the epilogue would wait for ever
        static std::atomic<int> known{0};             // any thread's call may be the first
        int regs = known;
        if (!regs) {
            cudaFuncAttributes f;
            if ((e = cudaFuncGetAttributes(&f, proj_rows_kernel<PAIR>)) != cudaSuccess)
                return e;
            known = regs = f.numRegs;
        }
        if (regs * R::THREADS < 128 * R::REGS_DOWN + (R::THREADS - 128) * R::REGS_UP)
            return cudaErrorInvalidConfiguration;
    }
    const int64_t room = PAIR ? sms / 2 : sms;
    return launch_early(proj_rows_kernel<PAIR>,
                        dim3((unsigned)((tiles < room ? tiles : room) * (PAIR ? 2 : 1))), R::THREADS,
                        R::SMEM, PAIR ? 2 : 1, s, tmA, tmW, tmO, d);
}

template <int TT>
cudaError_t launch_cols(const Fp8ProjArgs &g, ProjDev d, int sms, cudaStream_t s)
{
    using C = Cols<TT>;
    CUtensorMap tmA, tmW;
    if (!make_tmap_2d(&tmA, g.A, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)g.M,
                      (uint64_t)g.groups * g.K, TT) ||
        !make_tmap_2d(&tmW, g.W, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)d.ldo, (uint64_t)g.K,
                      128))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(proj_cols_kernel<TT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess)
        return e;
    const int64_t tiles = (g.M + TT - 1) / TT * ((g.N + 127) / 128) * g.groups;
    if (tiles > INT32_MAX / kMaxSplit)
        return cudaErrorInvalidConfiguration;
    // a block to every SM, and a second one where enough blocks of inputs are left
    // for each (16 tokens by 8192 x 8192: 21.2 against 19.1 us with two; by 4096 x
    // 4096, four blocks each: 8.5 and 8.5; 64 tokens by 4096 x 8192: 16.1 against
    // 14.3; 333 by 1000 x 2064: 9.7 and 9.7). Of the splits 1, 2, 4 and 8 the rule
    // takes the best or one within 3 % in each of 20 sizes from 12 to 333 tokens,
    // 512 to 12288 features and 2048 to 16384 inputs.
    int split = 1;
    while (split < kMaxSplit && split * 2 <= d.nb &&
           (tiles * split * 2 <= sms ||
            (tiles * split <= sms && d.nb >= split * 2 * (TT == 64 ? 4 : 8))))
        split *= 2;
    return launch_early(proj_cols_kernel<TT>, dim3((unsigned)(tiles * split)), C::THREADS, C::SMEM,
                        split, s, tmA, tmW, d, split);
}

cudaError_t launch_few(const Fp8ProjArgs &g, const ProjDev &d, int sms, cudaStream_t s)
{
    // shares of the inputs until every SM has eight warps
    const int64_t tiles = (int64_t)g.groups * ((g.N + 15) / 16);
    int ks = 1;
    while (ks < kFewWarps && 2 * ks <= d.nb && tiles * ks < 8 * (int64_t)sms)
        ks *= 2;
    const int rg = ks >= 8 ? 1 : 8 / ks;
    const int64_t blocks = (int64_t)g.groups * ((g.N + 16 * rg - 1) / (16 * rg));
    return launch_early(proj_few_kernel, dim3((unsigned)blocks), 32 * rg * ks,
                        ks * 16 * rg * kFewLd * 4, 1, s, g.A, g.W, d, ks);
}

Fp8ProjForm form_of(const Fp8ProjArgs &g, int sms)
{
    const int64_t nb = (g.K + PB - 1) / PB, weight = (int64_t)g.groups * g.N * g.K;
    // Up to 8 tokens take the kernel that waits least, but for e4m3 results (a
    // scale's 128 features would have to share a block), where the ring's kernel
    // fills the SMs without clusters (8 tokens by 8192 x 1024: 3.6 against 4.3 us;
    // by 20000 x 4096: 33.5 against 21.0) and for weights that it streams better
    // (by 8192 x 2048: 5.0 against 5.4; by 8192 x 8192: 16.7 against 14.9).
    const int64_t ft = ((g.N + 127) / 128) * (int64_t)g.groups;
    if (g.M <= kFewTokens && g.out_dt != CSA_E4M3 && 2 * ft <= sms && weight <= (32 << 20))
        return PROJ_FEW;
    if (g.M <= 16)
        return PROJ_COLS_16;
    if (g.M <= 32)
        return PROJ_COLS_32;
    // More tokens take the row kernel, unless long rows over few tiles leave a
    // cluster several SMs to a tile: four of them (128 tokens by 1024 x 2048: 8.7
    // against 7.4 us, by 1024 x 4096: 13.1 against 9.0), or two where the rows are
    // longer (333 tokens by 1000 x 2304: 9.2 against 9.5, x 2816: 10.2 against
    // 10.0, x 4096: 13.1 against 11.5; the same turn between 2560 and 3200 inputs
    // for 256 x 2048, 500 x 768, 1000 x 384, 180 x 2000, 64 x 8192 and 300 x 1280)
    // or start off a sector of 32 bytes, which costs the row kernel's loads more
    // (333 tokens by 1000 x 2048: 8.7 against 9.0, x 2064: 10.5 against 9.7; 256 by
    // 2048 x 2064: 10.5 and 10.5, x 2576: 12.3 against 11.3; 1000 by 384 x 2064: 10.5
    // against 10.0).
    const int64_t cols_tiles = (g.M + 63) / 64 * ft;
    if (nb >= 16 && (g.K % 32 == 0 && nb < 24 ? 4 : 2) * cols_tiles <= sms)
        return PROJ_COLS_64;
    // A pair's tile is four of a single block's and takes 16/9 of its time on two
    // SMs (4096 tokens by 2048 x 4096: 40.1 us in four rounds against 35.1 in two;
    // 1536 by 4096 x 4096: 31.0 in three against 36.3 in two).
    const int64_t one = (g.M + 127) / 128 * ft;
    const int64_t two = (g.M + 255) / 256 * ((g.N + 255) / 256) * g.groups;
    return 16 * ((two + sms / 2 - 1) / (sms / 2)) < 9 * ((one + sms - 1) / sms) ? PROJ_PAIRS
                                                                              : PROJ_TILES;
}

}  // namespace

Fp8ProjForm fp8_proj_form(const Fp8ProjArgs &g) { return form_of(g, sm_count()); }

cudaError_t launch_fp8_proj(const Fp8ProjArgs &g, unsigned *err, cudaStream_t s)
{
    ProjDev d;
    d.As = g.As;
    d.Ws = g.Ws;
    d.out = g.out;
    d.out_scale = g.out_scale;
    d.err = err;
    d.M = g.M;
    d.ldo = (int64_t)g.groups * g.N;
    d.N = g.N;
    d.K = g.K;
    d.groups = g.groups;
    d.nb = (g.K + PB - 1) / PB;
    d.las = g.groups * d.nb;
    d.nbo = (int)((d.ldo + PB - 1) / PB);
    d.out_dt = g.out_dt;
    d.tma_out = false;
    const int sms = sm_count();
    switch (form_of(g, sms)) {
    case PROJ_FEW:
        return launch_few(g, d, sms, s);
    case PROJ_COLS_16:
        return launch_cols<16>(g, d, sms, s);
    case PROJ_COLS_32:
        return launch_cols<32>(g, d, sms, s);
    case PROJ_COLS_64:
        return launch_cols<64>(g, d, sms, s);
    case PROJ_PAIRS:
        return launch_rows<true>(g, d, sms, s);
    default:
        return launch_rows<false>(g, d, sms, s);
    }
}

}  // namespace csa
