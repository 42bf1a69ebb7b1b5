// gated.cu -- the gated feed-forward block of an MXFP8 expert in one kernel per
// direction:
//   pmn_w1_gemm_swiglu_mxfp8           gate and up projections, silu(gate) * up,
//                                      MXFP8 of h (and of h^T, and bf16 y)
//   pmn_dh_gemm_swiglu_backward_mxfp8  dH = dY . W2, SwiGLU's gradient, MXFP8 of
//                                      dY1 and of dY1^T
// The products run on the 5th-generation tensor cores (block-scaled tcgen05 MMA,
// float32 accumulators in TMEM); everything after them is done on the
// accumulators, so y, h and dH never make a round trip through memory at a wider
// type than the one they are kept in.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/pmn.h"
#include "numerics.cuh"
#include "sm100.cuh"

using namespace pmn;
using namespace pmn::sm100;

uint64_t pmn_wait_limit_ns();  // gemm.cu: the limit of every bounded device wait

namespace {

__device__ int g_gated_error = 0;

constexpr int BM = 128;
constexpr int MAX_GROUPS = 1024;
constexpr int EW = 8;                       // epilogue warps, two per TMEM lane quadrant
constexpr int THREADS = 128 + 32 * EW;
constexpr uint32_t TMEM_COLS = 512;
constexpr int TP = 17;                      // row pitch (floats) of a warp's transposition buffer
constexpr int TP_BYTES = 32 * TP * 4;

// One tile: 128 routed rows of an expert times TBN rows of its weight.  Forward:
// TBN / 2 gate rows and the TBN / 2 up rows of the same columns of h; backward:
// TBN columns of dH.  A stage holds 128 bytes of K of both operands (TMA,
// 128-byte swizzle) and their scale factors in the 32 x 128-bit form that
// tcgen05.cp copies into TMEM.
template <bool BWD, int TBN>
struct Cfg {
    static constexpr int HB = BWD ? TBN : TBN / 2;  // columns of h (dH) per tile
    static constexpr int NCH = HB / 32;             // 32-column chunks (MX blocks) of the epilogue
    static constexpr int RB = (TBN + 127) / 128;    // 128-row scale blocks of B
    static constexpr int A_BYTES = BM * 128, B_BYTES = TBN * 128, SF_BYTES = 512 * (1 + RB);
    static constexpr int STAGE_BYTES = (A_BYTES + B_BYTES + SF_BYTES + 1023) / 1024 * 1024;
    static constexpr int STAGES = TBN == 256 ? 4 : TBN == 128 ? 5 : 7;
    static constexpr uint32_t SF_COLS = 4 * (1 + RB);
    static constexpr int ACC = 2 * TBN + STAGES * (int)SF_COLS <= (int)TMEM_COLS ? 2 : 1;  // accumulators
    static constexpr uint32_t SF_COL0 = ACC * TBN;
    static constexpr int NR = 4 + TBN / 32;         // scale rows per lane
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EW * TP_BYTES + 1024 + (MAX_GROUPS + 1) * 4;
    static_assert(SF_COL0 + STAGES * SF_COLS <= TMEM_COLS, "TMEM budget");
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

struct Args {
    const int32_t *offsets;
    int groups;
    int64_t m, f, k;         // routed rows, columns of h, contraction length
    const uint8_t *sa, *sb;  // scales, k / 32 bytes per row
    int64_t b_rows;          // rows of B of all experts
    uint8_t *out, *out_sc, *out_t, *out_t_sc;
    uint16_t *y;             // forward: written (or NULL); backward: read
    uint64_t wait_ns;
};

struct Tile {
    int g;
    int64_t m0, row_end;
    int h0;  // first column of h
};

template <bool BWD, int TBN>
__device__ __forceinline__ Tile get_tile(int t, const Args &p, const int *s_cum, int &gc)
{
    while (gc + 1 < p.groups && s_cum[gc + 1] <= t) ++gc;  // every role walks its tiles upwards
    constexpr int HB = Cfg<BWD, TBN>::HB;
    const int nt = (int)((p.f + HB - 1) / HB);
    const int local = t - s_cum[gc], mi = local / nt;
    Tile ti;
    ti.g = gc;
    ti.m0 = __ldg(p.offsets + gc) + (int64_t)mi * BM;
    ti.row_end = __ldg(p.offsets + gc + 1);
    ti.h0 = (local - mi * nt) * HB;
    return ti;
}

__device__ __forceinline__ void latch_error(int bit) { atomicOr(&g_gated_error, bit); }

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    const bool ok = mbar_wait(bar, parity, limit_ns);
    return __all_sync(0xFFFFFFFFu, ok) != 0;  // warp-uniform, also on a timeout
}

// Instruction descriptor of the block-scaled MMA: E4M3 operands, E8M0 scales,
// M = 128, N = TBN; sf_id selects the scale byte of the 32-deep K step.
template <int TBN>
__device__ __forceinline__ uint32_t make_idesc(uint32_t sf_id)
{
    return (sf_id << 4) | ((uint32_t)(TBN >> 3) << 17) | (1u << 23) | ((uint32_t)(BM >> 4) << 24) | (sf_id << 29);
}

// Four values times 2^-e -> four E4M3 bytes, nearest even.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float s)
{
    return cvt_e4m3x2_rn(__fmul_rn(a, s), __fmul_rn(b, s)) | (cvt_e4m3x2_rn(__fmul_rn(c, s), __fmul_rn(d, s)) << 16);
}

// MXFP8 of one row's 32 columns held by this thread.
__device__ __forceinline__ void store_row_block(const float (&v)[32], uint8_t *q, uint8_t *sc)
{
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) amax = fmaxf(amax, fabsf(v[j]));
    const int e = mx_exponent_448(amax);
    const float s = exp2_neg(e);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = e4m3x4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], s);
    uint4 *o = reinterpret_cast<uint4 *>(q);
    o[0] = make_uint4(w[0], w[1], w[2], w[3]);
    o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    *sc = (uint8_t)(e + 127);
}

// MXFP8 along the rows of a warp's 32 x 32 block (lane = row, v[j] = column j),
// in two halves of 16 columns through shared memory: lane l takes column l % 16
// and rows 16 (l / 16) .. + 15, so a column's block lies in lanes l and l + 16.
// q, sc: the block's first column in the transposed tensor, at its first row.
__device__ __forceinline__ void store_col_blocks(const float (&v)[32], float *buf, uint8_t *q, uint8_t *sc,
                                                 int64_t pitch, int lane)
{
    const int c = lane & 15, hi = lane >> 4;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) buf[lane * TP + j] = v[16 * half + j];
        __syncwarp();
        float u[16];
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            u[i] = buf[(16 * hi + i) * TP + c];
            amax = fmaxf(amax, fabsf(u[i]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 16));
        const int e = mx_exponent_448(amax);
        const float s = exp2_neg(e);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = e4m3x4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3], s);
        const int64_t col = 16 * half + c;
        *reinterpret_cast<uint4 *>(q + col * pitch + 16 * hi) = make_uint4(w[0], w[1], w[2], w[3]);
        if (hi == 0) sc[col * (pitch / 32)] = (uint8_t)(e + 127);
    }
}

// One persistent kernel per call, one CTA per SM:
//   warp 0     one lane loads the operands' code tiles by TMA
//   warp 2     scale factors: 16 bytes of each row cover four stages; they are
//              read a group of four stages ahead and written in the form that
//              tcgen05.cp expects
//   warp 1     one lane copies a stage's scale factors into TMEM and issues its
//              MMAs (copies and MMAs of one thread execute in order)
//   warps 4..  epilogue, one row per thread and 32 columns at a time
// Every wait is bounded: on a timeout an error bit is latched and the CTA winds
// down.
template <bool BWD, int TBN>
__global__ void __launch_bounds__(THREADS, 1)
    gated_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Args p)
{
    using C = Cfg<BWD, TBN>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *stages = smem;
    float *tbuf = reinterpret_cast<float *>(smem + STAGES * C::STAGE_BYTES);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * C::STAGE_BYTES + EW * TP_BYTES);
    const uint32_t bar_full = smem_u32(bars), bar_empty = bar_full + 8 * STAGES, bar_sfr = bar_empty + 8 * STAGES;
    const uint32_t bar_acc_full = bar_sfr + 8 * STAGES, bar_acc_empty = bar_acc_full + 16;
    const uint32_t bar_drain = bar_acc_empty + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 3 * STAGES + 5);
    int *s_abort = reinterpret_cast<int *>(tmem_slot + 1);
    int *s_total = s_abort + 1;
    int *s_cum = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(bars) + 1024);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
            mbar_init(bar_sfr + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_acc_full + 8 * b, 1);
            mbar_init(bar_acc_empty + 8 * b, EW);
        }
        mbar_init(bar_drain, 1);
        *s_abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 0) {
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 1) {
        // tiles of each group and their running sum, 32 groups at a time; offsets
        // that are not monotone, in range and (with column blocks) multiples of
        // 32 run no tile
        const int nt = (int)((p.f + C::HB - 1) / C::HB);
        const bool cols = p.out_t != nullptr;
        int base = 0;
        bool good = true;
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
            const int g = g0 + lane;
            int lo = 0, hi = 0;
            if (g < p.groups) {
                lo = __ldg(p.offsets + g);
                hi = __ldg(p.offsets + g + 1);
                if (lo < 0 || hi < lo || hi > p.m || (cols && ((lo | hi) & 31))) good = false;
            }
            good = __all_sync(0xFFFFFFFFu, good);
            if (!good) break;
            int n = (hi - lo + BM - 1) / BM * nt, sum = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += v;
            }
            if (g < p.groups) s_cum[g] = base + sum - n;
            base += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        if (lane == 0) {
            s_cum[p.groups] = base;
            *s_total = good ? base : 0;
            if (!good && blockIdx.x == 0) latch_error(PMN_DEVERR_BAD_OFFSETS);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = *s_total;
    const int nks = (int)(p.k / 128);

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer
            uint32_t stage = 0, phase = 0, issued = 0, last = 0;
            int gc = 0;
            for (int t = blockIdx.x; t < total && !*(volatile int *)s_abort; t += gridDim.x) {
                const Tile ti = get_tile<BWD, TBN>(t, p, s_cum, gc);
                const int64_t brow = (int64_t)ti.g * (BWD ? p.f : 2 * p.f) + ti.h0;
                for (int ks = 0; ks < nks; ++ks) {
                    if (!mbar_wait(bar_empty + 8 * stage, phase ^ 1, p.wait_ns)) {
                        *(volatile int *)s_abort = 1;
                        latch_error(PMN_DEVERR_WAIT_TIMEOUT);
                        break;
                    }
                    uint8_t *st = stages + stage * C::STAGE_BYTES;
                    const uint32_t fb = bar_full + 8 * stage;
                    mbar_arrive_expect_tx(fb, C::A_BYTES + C::B_BYTES);
                    tma_load_2d(smem_u32(st), &tmA, fb, ks * 128, (int32_t)ti.m0);
                    tma_load_2d(smem_u32(st + C::A_BYTES), &tmB, fb, ks * 128, (int32_t)brow);
                    if (!BWD)
                        tma_load_2d(smem_u32(st + C::A_BYTES + C::B_BYTES / 2), &tmB, fb, ks * 128, (int32_t)(brow + p.f));
                    issued |= 1u << stage;
                    last = (last & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // no copy may still be landing when the CTA ends
            for (int s = 0; s < STAGES; ++s)
                if (issued & (1u << s)) (void)mbar_wait(bar_full + 8 * s, (last >> s) & 1u, 1000000000ull);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------------------------------------------- scale factors
        // Block b (A, then the 128-row blocks of B), lane r, word j: the four
        // scale bytes of row 32 j + r of the stage's 128-deep K range.
        const int64_t pitch = p.k / 32;
        const int groups4 = nks / 4;  // k is a multiple of 512
        int t = blockIdx.x, q = 0, gc = 0;
        Tile ti;
        if (t < total) ti = get_tile<BWD, TBN>(t, p, s_cum, gc);
        auto fetch = [&](uint4 (&v)[C::NR]) {
            if (t >= total) return;
            const int64_t brow = (int64_t)ti.g * (BWD ? p.f : 2 * p.f) + ti.h0;
#pragma unroll
            for (int j = 0; j < C::NR; ++j) {
                int64_t row;
                const uint8_t *base;
                bool ok;
                if (j < 4) {
                    row = ti.m0 + 32 * j + lane;
                    base = p.sa;
                    ok = row < p.m;
                } else {
                    const int n = 32 * (j - 4);  // row of B within the tile
                    row = brow + n + lane + (!BWD && n >= C::HB ? p.f - C::HB : 0);
                    base = p.sb;
                    ok = row < p.b_rows;
                }
                v[j] = make_uint4(0u, 0u, 0u, 0u);
                if (ok) v[j] = __ldg(reinterpret_cast<const uint4 *>(base + row * pitch + 16 * q));
            }
            if (++q == groups4) {
                q = 0;
                t += gridDim.x;
                if (t < total) ti = get_tile<BWD, TBN>(t, p, s_cum, gc);
            }
        };
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        auto put = [&](const uint4 (&v)[C::NR]) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                ok = ok && warp_wait(bar_empty + 8 * stage, phase ^ 1, p.wait_ns);
                if (!ok || __any_sync(0xFFFFFFFFu, *(volatile int *)s_abort != 0)) {
                    if (!ok && lane == 0) {
                        *(volatile int *)s_abort = 1;
                        latch_error(PMN_DEVERR_WAIT_TIMEOUT);
                    }
                    ok = false;
                    return;
                }
                uint4 *sf = reinterpret_cast<uint4 *>(stages + stage * C::STAGE_BYTES + C::A_BYTES + C::B_BYTES) + lane;
                sf[0] = make_uint4(u4_word(v[0], s), u4_word(v[1], s), u4_word(v[2], s), u4_word(v[3], s));
#pragma unroll
                for (int b = 0; b < C::RB; ++b) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = 4 + 4 * b + j < C::NR ? u4_word(v[4 + 4 * b + j], s) : 0u;
                    sf[32 * (1 + b)] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_sfr + 8 * stage);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        };
        int64_t left = 0;  // groups of four stages of this CTA
        for (int u = blockIdx.x; u < total; u += gridDim.x) left += groups4;
        uint4 v0[C::NR], v1[C::NR];
        fetch(v0);
        while (ok && left > 0) {
            fetch(v1);
            put(v0);
            if (--left <= 0 || !ok) break;
            fetch(v0);
            put(v1);
            --left;
        }
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, abuf = 0, aphase = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                if (!mbar_wait(bar_acc_empty + 8 * abuf, aphase ^ 1, p.wait_ns) || *(volatile int *)s_abort) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + abuf * TBN;
                for (int ks = 0; ks < nks; ++ks) {
                    if (!mbar_wait(bar_full + 8 * stage, phase, p.wait_ns) ||
                        !mbar_wait(bar_sfr + 8 * stage, phase, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    uint8_t *st = stages + stage * C::STAGE_BYTES;
                    const uint32_t sf = smem_u32(st + C::A_BYTES + C::B_BYTES);
                    const uint32_t sfa = tmem + C::SF_COL0 + stage * C::SF_COLS, sfb = sfa + 4;
#pragma unroll
                    for (int b = 0; b < 1 + C::RB; ++b)
                        tc_cp_32x128b_warpx4(sfa + 4 * b, smem_desc(sf + 512 * b, 0, 128, 0));
                    const uint32_t a = smem_u32(st), b = smem_u32(st + C::A_BYTES);
#pragma unroll
                    for (int s = 0; s < 4; ++s)  // 32 of K per MMA inside the 128-byte swizzled rows
                        mma_mxfp8(d, smem_desc(a + 32 * s, 16, 1024, 2), smem_desc(b + 32 * s, 16, 1024, 2),
                                  make_idesc<TBN>((uint32_t)s), sfa, sfb, (ks > 0 || s > 0) ? 1u : 0u);
                    tc_commit(bar_empty + 8 * stage);
                    if (ks == nks - 1) tc_commit(bar_acc_full + 8 * abuf);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (++abuf == C::ACC) {
                    abuf = 0;
                    aphase ^= 1;
                }
            }
            if (!ok && !*(volatile int *)s_abort) {
                *(volatile int *)s_abort = 1;
                latch_error(PMN_DEVERR_WAIT_TIMEOUT);
            }
            tc_commit(bar_drain);  // every tcgen05 operation of this thread has completed
            (void)mbar_wait(bar_drain, 0, 1000000000ull);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------- epilogue
        // Warp w reads accumulator lanes (rows) 32 (w % 4) .. + 31 and every
        // second 32-column chunk.
        const int quad = warp & 3, half = (warp - 4) >> 2;
        float *buf = tbuf + (warp - 4) * (32 * TP);
        uint32_t abuf = 0, aphase = 0;
        int gc = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x) {
            const Tile ti = get_tile<BWD, TBN>(t, p, s_cum, gc);
            const int64_t row0 = ti.m0 + 32 * quad, row = row0 + lane;
            const bool valid = row < ti.row_end;
            const bool any = row0 < ti.row_end;  // with column blocks: all 32 rows or none
            if (!warp_wait(bar_acc_full + 8 * abuf, aphase, p.wait_ns)) {
                if (lane == 0) {
                    *(volatile int *)s_abort = 1;
                    latch_error(PMN_DEVERR_WAIT_TIMEOUT);
                }
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(32 * quad) << 16) + abuf * TBN;
#pragma unroll 1
            for (int c = half; c < C::NCH; c += 2) {
                const int64_t col = ti.h0 + 32 * c;
                const bool on = any && col < p.f;
                float v[32];
                if constexpr (!BWD) {
                    float u[32];
                    tmem_ld_32x32b_x32(acc + 32 * c, reinterpret_cast<uint32_t(&)[32]>(v));
                    tmem_ld_32x32b_x32(acc + C::HB + 32 * c, reinterpret_cast<uint32_t(&)[32]>(u));
                    tmem_ld_wait();
                    if (on) {
                        if (p.y && valid) {
#pragma unroll
                            for (int part = 0; part < 2; ++part) {
                                uint4 *o = reinterpret_cast<uint4 *>(p.y + row * 2 * p.f + part * p.f + col);
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    uint32_t w[4];
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const float *x = (part ? u : v) + 8 * j + 2 * i;
                                        const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[0], x[1]);
                                        w[i] = *reinterpret_cast<const uint32_t *>(&b2);
                                    }
                                    o[j] = make_uint4(w[0], w[1], w[2], w[3]);
                                }
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = silu_mul(v[j], u[j]);
                        if (valid) store_row_block(v, p.out + row * p.f + col, p.out_sc + row * (p.f / 32) + col / 32);
                        if (p.out_t)
                            store_col_blocks(v, buf, p.out_t + col * p.m + row0, p.out_t_sc + col * (p.m / 32) + row0 / 32,
                                             p.m, lane);
                    }
                } else {
                    uint4 gw[4], uw[4];
                    if (on) {
                        const uint4 *yg = reinterpret_cast<const uint4 *>(p.y + row * 2 * p.f + col);
                        const uint4 *yu = reinterpret_cast<const uint4 *>(p.y + row * 2 * p.f + p.f + col);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            gw[j] = __ldg(yg + j);
                            uw[j] = __ldg(yu + j);
                        }
                    }
                    tmem_ld_32x32b_x32(acc + 32 * c, reinterpret_cast<uint32_t(&)[32]>(v));
                    tmem_ld_wait();
                    if (on) {
                        float du[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const uint32_t a = u4_word(gw[j >> 3], (j >> 1) & 3), b = u4_word(uw[j >> 3], (j >> 1) & 3);
                            const float g = __uint_as_float((j & 1) ? (a & 0xFFFF0000u) : (a << 16));
                            const float u = __uint_as_float((j & 1) ? (b & 0xFFFF0000u) : (b << 16));
                            const float s = __fdividef(1.0f, __fadd_rn(1.0f, __expf(-g)));
                            const float ds = __fmul_rn(v[j], s);
                            du[j] = __fmul_rn(ds, g);
                            v[j] = __fmul_rn(__fmul_rn(ds, u), fmaf(g, __fsub_rn(1.0f, s), 1.0f));
                        }
                        const int64_t f2 = 2 * p.f;
                        store_row_block(v, p.out + row * f2 + col, p.out_sc + row * (f2 / 32) + col / 32);
                        store_row_block(du, p.out + row * f2 + p.f + col, p.out_sc + row * (f2 / 32) + (p.f + col) / 32);
                        store_col_blocks(v, buf, p.out_t + col * p.m + row0, p.out_t_sc + col * (p.m / 32) + row0 / 32,
                                         p.m, lane);
                        store_col_blocks(du, buf, p.out_t + (p.f + col) * p.m + row0,
                                         p.out_t_sc + (p.f + col) * (p.m / 32) + row0 / 32, p.m, lane);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_acc_empty + 8 * abuf);
            if (++abuf == C::ACC) {
                abuf = 0;
                aphase ^= 1;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

// ====================================================================== host
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// E4M3 bytes [rows, k] in boxes of 128 bytes x box_rows, 128-byte swizzle; rows
// past the end read as zeros.
bool make_map(CUtensorMap *m, const void *base, uint64_t k, uint64_t rows, uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {k, rows}, strides[1] = {k};
    cuuint32_t box[2] = {128, box_rows}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <bool BWD, int TBN>
pmn_status launch(const uint8_t *a, const uint8_t *b, const Args &args, cudaStream_t s)
{
    using C = Cfg<BWD, TBN>;
    CUtensorMap ma, mb;
    if (!make_map(&ma, a, (uint64_t)args.k, (uint64_t)args.m, BM) ||
        !make_map(&mb, b, (uint64_t)args.k, (uint64_t)args.b_rows, BWD ? TBN : TBN / 2))
        return PMN_ERR_CUDA;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        return PMN_ERR_CUDA;
    auto kern = gated_kernel<BWD, TBN>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
        return PMN_ERR_CUDA;
    kern<<<(unsigned)sms, THREADS, C::SMEM_BYTES, s>>>(ma, mb, args);
    return cudaGetLastError() == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

// What both directions ask of their sizes and operands.
pmn_status check_common(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b, const uint8_t *b_scales,
                        const int32_t *offsets, int num_experts, int64_t total_rows, int64_t f, int64_t k)
{
    if (num_experts <= 0 || num_experts > MAX_GROUPS || total_rows < 0 || total_rows >= (int64_t(1) << 31) || f <= 0 ||
        f % 128 != 0 || k <= 0 || k % 512 != 0 || k >= (int64_t(1) << 31) || f >= (int64_t(1) << 28))
        return PMN_ERR_INVALID_ARG;
    if ((int64_t)num_experts * 2 * f >= (int64_t(1) << 31)) return PMN_ERR_INVALID_ARG;  // rows of B: a TMA coordinate
    // tiles are counted in 32 bits
    if ((total_rows / BM + num_experts) * (f / 16) >= (int64_t(1) << 31)) return PMN_ERR_UNSUPPORTED;
    if (total_rows == 0) return PMN_OK;  // nothing to read: NULL operands allowed
    if (!a || !a_scales || !b || !b_scales || !offsets) return PMN_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(a_scales) || !aligned16(b) || !aligned16(b_scales) || ((uintptr_t)offsets & 3u))
        return PMN_ERR_INVALID_ARG;
    return PMN_OK;
}

}  // namespace

// The library's device error word is read through pmn_get_device_error, which
// collects each translation unit's word.
pmn_status pmn_take_gated_device_error(cudaStream_t s, int *bits)
{
    int host = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbolAsync(&host, g_gated_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return PMN_ERR_CUDA;
    if (host != 0 &&
        (cudaMemcpyToSymbolAsync(g_gated_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
         cudaStreamSynchronize(s) != cudaSuccess))
        return PMN_ERR_CUDA;
    *bits = host;
    return PMN_OK;
}

extern "C" pmn_status pmn_w1_gemm_swiglu_mxfp8(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b,
                                               const uint8_t *b_scales, const int32_t *offsets, int num_experts,
                                               int64_t total_rows, int64_t f, int64_t k, uint8_t *out,
                                               uint8_t *out_scales, uint8_t *out_t, uint8_t *out_t_scales, void *y_out,
                                               void *stream)
{
    const pmn_status st = check_common(a, a_scales, b, b_scales, offsets, num_experts, total_rows, f, k);
    if (st != PMN_OK || total_rows == 0) return st;
    if ((out_t != nullptr) != (out_t_scales != nullptr) || (out_t && total_rows % 32 != 0)) return PMN_ERR_INVALID_ARG;
    if (!out || !out_scales || !aligned16(out) || !aligned16(out_t) || !aligned16(y_out)) return PMN_ERR_INVALID_ARG;
    const Args args{offsets, num_experts, total_rows, f, k, a_scales, b_scales, (int64_t)num_experts * 2 * f,
                    out, out_scales, out_t, out_t_scales, static_cast<uint16_t *>(y_out), pmn_wait_limit_ns()};
    return launch<false, 256>(a, b, args, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" pmn_status pmn_dh_gemm_swiglu_backward_mxfp8(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b,
                                                        const uint8_t *b_scales, const void *y, const int32_t *offsets,
                                                        int num_experts, int64_t total_rows, int64_t f, int64_t k,
                                                        uint8_t *out, uint8_t *out_scales, uint8_t *out_t,
                                                        uint8_t *out_t_scales, void *stream)
{
    const pmn_status st = check_common(a, a_scales, b, b_scales, offsets, num_experts, total_rows, f, k);
    if (st != PMN_OK || total_rows == 0) return st;
    if (total_rows % 32 != 0) return PMN_ERR_INVALID_ARG;
    if (!y || !out || !out_scales || !out_t || !out_t_scales || !aligned16(y) || !aligned16(out) || !aligned16(out_t))
        return PMN_ERR_INVALID_ARG;
    const Args args{offsets, num_experts, total_rows, f, k, a_scales, b_scales, (int64_t)num_experts * f,
                    out, out_scales, out_t, out_t_scales, static_cast<uint16_t *>(const_cast<void *>(y)),
                    pmn_wait_limit_ns()};
    return launch<true, 256>(a, b, args, reinterpret_cast<cudaStream_t>(stream));
}
