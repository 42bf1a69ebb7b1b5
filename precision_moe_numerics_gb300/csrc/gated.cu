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
// An epilogue warp's shared memory: 32 rows x 32 columns of bf16 gate and up
// (2 x 2 KB), and 2 KB through which blocks are transposed and codes are staged
// for TMA stores.
constexpr int Y_BYTES = 4096, T_BYTES = 2048, WARP_BYTES = Y_BYTES + T_BYTES;

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
    static constexpr int STAGES = TBN >= 192 ? 4 : TBN == 128 ? 5 : 7;
    static constexpr uint32_t SF_COLS = 4 * (1 + RB);
    static constexpr int ACC = 2 * TBN + STAGES * (int)SF_COLS <= (int)TMEM_COLS ? 2 : 1;  // accumulators
    static constexpr uint32_t SF_COL0 = ACC * TBN;
    static constexpr int NR = 4 + TBN / 32;         // scale rows per lane
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EW * WARP_BYTES + 1024 + (MAX_GROUPS + 1) * 4;
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

// Largest magnitude of the thread's values -> E8M0 exponent and 2^-e.
__device__ __forceinline__ float block_scale(float amax, uint8_t &byte)
{
    const int e = mx_exponent_448(amax);
    byte = (uint8_t)(e + 127);
    return exp2_neg(e);
}

// MXFP8 of one row's 32 columns held by this thread.
__device__ __forceinline__ void row_block(const float (&v)[32], uint4 (&q)[2], uint8_t &sc)
{
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) amax = fmaxf(amax, fabsf(v[j]));
    const float s = block_scale(amax, sc);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = e4m3x4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], s);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// 16-byte piece `i` of row `r` in a box of 32 rows x 32 bytes (TMA's 32-byte
// swizzle) or x 64 bytes (64-byte swizzle): eight lanes that access one piece of
// eight consecutive rows meet eight different bank groups.
__device__ __forceinline__ int box32(int r, int i) { return 32 * r + 16 * (i ^ ((r >> 2) & 1)); }
__device__ __forceinline__ int box64(int r, int i) { return 64 * r + 16 * (i ^ ((r >> 1) & 3)); }

// Largest magnitude over the warp's lanes (NaN ignored, as fmaxf does).
__device__ __forceinline__ uint32_t warp_absmax(float v)
{
    float m;
    asm("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return __float_as_uint(m);
}

// MXFP8 along the rows of a warp's 32 x 32 block (lane = row, v[j] = column j).
// A column's maximum is one reduction over the lanes, so the values are scaled
// and converted where they are and only bytes are transposed: through shared
// memory (rows 36 bytes apart: conflict-free both ways), lane 4 k + r then holds
// columns 4 k .. 4 k + 3, rows 8 r .. 8 r + 7.
// The exponent rule of mx_exponent_448 on the bits M of the maximum: with
// t = (M + 0x1FFFFF) >> 23 (a carry where M's fraction is above 1.75) and t >= 8,
// e = t - 135, so the scale byte is t - 8 and 2^-e has the exponent field 262 - t.
// q: the block's first column at its first row; pitch: bytes between columns.
__device__ __forceinline__ void col_blocks(const float (&v)[32], uint8_t *buf, uint8_t *q, int64_t pitch, uint8_t &sc,
                                           int lane)
{
    uint32_t sb[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float y[4];
        uint32_t t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[i] = max(min(warp_absmax(v[4 * k + i]), 0x7F800000u), 0x04000000u) + 0x1FFFFFu;  // (all NaN: as infinity)
            y[i] = __fmul_rn(v[4 * k + i], __uint_as_float(0x83000000u - (t[i] & 0xFF800000u)));
        }
        *reinterpret_cast<uint32_t *>(buf + 36 * lane + 4 * k) =
            cvt_e4m3x2_rn(y[0], y[1]) | (cvt_e4m3x2_rn(y[2], y[3]) << 16);
        sb[k] = __byte_perm(__byte_perm(t[0] << 1, t[1] << 1, 0x0073), __byte_perm(t[2] << 1, t[3] << 1, 0x0073), 0x5410) -
                0x08080808u;
    }
    __syncwarp();
    const int k = lane >> 2, r = lane & 3;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint32_t *>(buf + 36 * (8 * r + i) + 4 * k);
    __syncwarp();
    uint2 o[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 4 x 4 bytes each
        const uint32_t a = __byte_perm(w[4 * h], w[4 * h + 1], 0x5140), b = __byte_perm(w[4 * h + 2], w[4 * h + 3], 0x5140);
        const uint32_t c = __byte_perm(w[4 * h], w[4 * h + 1], 0x7362), d = __byte_perm(w[4 * h + 2], w[4 * h + 3], 0x7362);
        (h ? o[0].y : o[0].x) = __byte_perm(a, b, 0x5410);
        (h ? o[1].y : o[1].x) = __byte_perm(a, b, 0x7632);
        (h ? o[2].y : o[2].x) = __byte_perm(c, d, 0x5410);
        (h ? o[3].y : o[3].x) = __byte_perm(c, d, 0x7632);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint2 *>(q + (4 * k + i) * pitch + 8 * r) = o[i];
    const uint32_t s01 = k & 1 ? sb[1] : sb[0], s23 = k & 1 ? sb[3] : sb[2], s45 = k & 1 ? sb[5] : sb[4],
                   s67 = k & 1 ? sb[7] : sb[6];
    const uint32_t lo = k & 2 ? s23 : s01, hi = k & 2 ? s67 : s45;
    sc = (uint8_t)((k & 4 ? hi : lo) >> (8 * r));
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
    gated_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmY, const Args p)
{
    using C = Cfg<BWD, TBN>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *stages = smem;
    uint8_t *wbuf = smem + STAGES * C::STAGE_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * C::STAGE_BYTES + EW * WARP_BYTES);
    const uint32_t bar_full = smem_u32(bars), bar_empty = bar_full + 8 * STAGES, bar_sfr = bar_empty + 8 * STAGES;
    const uint32_t bar_acc_full = bar_sfr + 8 * STAGES, bar_acc_empty = bar_acc_full + 16;
    const uint32_t bar_drain = bar_acc_empty + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 3 * STAGES + 5 + EW);
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
        for (int w = 0; w < EW; ++w) mbar_init(bar_drain + 8 + 8 * w, 1);
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
        // second 32-column chunk.  Its global accesses are TMA boxes of 32 rows x
        // 32 columns (a row-per-thread access would touch 32 lines per
        // instruction); only the rows of a 32-row slice that an expert's end cuts
        // are stored one by one.
        const int quad = warp & 3, half = (warp - 4) >> 2;
        uint8_t *ybuf = wbuf + (warp - 4) * WARP_BYTES, *tb = ybuf + Y_BYTES;
        const uint32_t yb = smem_u32(ybuf), tbs = smem_u32(tb), bar_y = bar_drain + 8 + 8 * (warp - 4);
        uint32_t abuf = 0, aphase = 0, yphase = 0;
        int gc = 0;
        bool ok = true;
        // backward: gate and up of the next chunk are on their way while a chunk
        // is worked on
        int yt = blockIdx.x, yc = half, ygc = 0;
        bool pending = false;
        Tile yti;
        if (BWD && yt < total) yti = get_tile<BWD, TBN>(yt, p, s_cum, ygc);
        auto fetch_y = [&]() {
            if (yt >= total) return;
            if (yti.m0 + 32 * quad < yti.row_end && yti.h0 + 32 * yc < p.f) {
                pending = true;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar_y, Y_BYTES);
                    tma_load_2d(yb, &tmY, bar_y, yti.h0 + 32 * yc, (int32_t)yti.m0 + 32 * quad);
                    tma_load_2d(yb + Y_BYTES / 2, &tmY, bar_y, (int32_t)p.f + yti.h0 + 32 * yc, (int32_t)yti.m0 + 32 * quad);
                }
            }
            yc += 2;
            if (yc >= C::NCH) {
                yc = half;
                yt += gridDim.x;
                if (yt < total) yti = get_tile<BWD, TBN>(yt, p, s_cum, ygc);
            }
        };
        // shared memory that TMA stores still read may be written again
        auto stores_read = [&]() {
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
        };
        auto publish = [&]() {  // written by all lanes -> visible to TMA
            fence_proxy_async_smem();
            __syncwarp();
        };
        // one output's row codes into a staging box, and its scale bytes
        auto put_row = [&](const float (&v)[32], int box, int64_t row, int64_t col, int64_t width, bool valid, bool full) {
            uint4 q[2];
            uint8_t sc;
            row_block(v, q, sc);
            if (full) {
                *reinterpret_cast<uint4 *>(tb + 1024 * box + box32(lane, 0)) = q[0];
                *reinterpret_cast<uint4 *>(tb + 1024 * box + box32(lane, 1)) = q[1];
            } else if (valid) {
                uint4 *o = reinterpret_cast<uint4 *>(p.out + row * width + col);
                o[0] = q[0];
                o[1] = q[1];
            }
            if (valid) p.out_sc[row * (width / 32) + col / 32] = sc;
        };
        // one output's column blocks
        auto put_cols = [&](const float (&v)[32], int64_t row0, int64_t col) {
            uint8_t sc;
            col_blocks(v, tb, p.out_t + col * p.m + row0, p.m, sc, lane);
            p.out_t_sc[(col + lane) * (p.m / 32) + row0 / 32] = sc;
        };
        if (BWD) fetch_y();
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Tile ti = get_tile<BWD, TBN>(t, p, s_cum, gc);
            const int64_t row0 = ti.m0 + 32 * quad, row = row0 + lane;
            const bool valid = row < ti.row_end, any = row0 < ti.row_end, full = row0 + 32 <= ti.row_end;
            ok = warp_wait(bar_acc_full + 8 * abuf, aphase, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(32 * quad) << 16) + abuf * TBN;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_acc_empty + 8 * abuf);
            };
            if (half >= C::NCH) release();
#pragma unroll 1
            for (int c = half; c < C::NCH; c += 2) {
                const int64_t col = ti.h0 + 32 * c;
                const bool on = any && col < p.f;
                float v[32], u[32];
                if constexpr (!BWD) {
                    tmem_ld_32x32b_x32(acc + 32 * c, reinterpret_cast<uint32_t(&)[32]>(v));
                    tmem_ld_32x32b_x32(acc + C::HB + 32 * c, reinterpret_cast<uint32_t(&)[32]>(u));
                    tmem_ld_wait();
                    if (c + 2 >= C::NCH) release();
                    if (!on) continue;
                    stores_read();
                    if (p.y) {  // y in bf16 for the backward pass
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t w[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float *x = (part ? u : v) + 8 * j + 2 * i;
                                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[0], x[1]);
                                    w[i] = *reinterpret_cast<const uint32_t *>(&b2);
                                }
                                const uint4 q = make_uint4(w[0], w[1], w[2], w[3]);
                                if (full) *reinterpret_cast<uint4 *>(ybuf + part * (Y_BYTES / 2) + box64(lane, j)) = q;
                                else if (valid) *reinterpret_cast<uint4 *>(p.y + row * 2 * p.f + part * p.f + col + 8 * j) = q;
                            }
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = silu_mul(v[j], u[j]);
                    put_row(v, 0, row, col, p.f, valid, full);
                    if (full) {
                        publish();
                        if (lane == 0) {
                            tma_store_2d(&tmO, tbs, (int32_t)col, (int32_t)row0);
                            if (p.y) {
                                tma_store_2d(&tmY, yb, (int32_t)col, (int32_t)row0);
                                tma_store_2d(&tmY, yb + Y_BYTES / 2, (int32_t)(p.f + col), (int32_t)row0);
                            }
                            bulk_commit_group();
                        }
                    }
                    if (p.out_t) {
                        stores_read();
                        put_cols(v, row0, col);
                    }
                } else {
                    uint4 gw[4], uw[4];
                    if (on) {
                        ok = warp_wait(bar_y, yphase, p.wait_ns);
                        if (!ok) break;
                        pending = false;
                        yphase ^= 1;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            gw[j] = *reinterpret_cast<const uint4 *>(ybuf + box64(lane, j));
                            uw[j] = *reinterpret_cast<const uint4 *>(ybuf + Y_BYTES / 2 + box64(lane, j));
                        }
                        __syncwarp();
                    }
                    fetch_y();
                    tmem_ld_32x32b_x32(acc + 32 * c, reinterpret_cast<uint32_t(&)[32]>(v));
                    tmem_ld_wait();
                    if (c + 2 >= C::NCH) release();
                    if (!on) continue;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const uint32_t a = u4_word(gw[j >> 3], (j >> 1) & 3), b = u4_word(uw[j >> 3], (j >> 1) & 3);
                        const float gt = __uint_as_float((j & 1) ? (a & 0xFFFF0000u) : (a << 16));
                        const float up = __uint_as_float((j & 1) ? (b & 0xFFFF0000u) : (b << 16));
                        const float s = __fdividef(1.0f, __fadd_rn(1.0f, __expf(-gt)));
                        const float ds = __fmul_rn(v[j], s);
                        u[j] = __fmul_rn(ds, gt);
                        v[j] = __fmul_rn(__fmul_rn(ds, up), fmaf(gt, __fsub_rn(1.0f, s), 1.0f));
                    }
                    stores_read();
                    put_row(v, 0, row, col, 2 * p.f, true, true);
                    put_row(u, 1, row, p.f + col, 2 * p.f, true, true);
                    publish();
                    if (lane == 0) {
                        tma_store_2d(&tmO, tbs, (int32_t)col, (int32_t)row0);
                        tma_store_2d(&tmO, tbs + 1024, (int32_t)(p.f + col), (int32_t)row0);
                        bulk_commit_group();
                    }
                    stores_read();
                    put_cols(v, row0, col);
                    put_cols(u, row0, p.f + col);
                }
            }
            if (++abuf == C::ACC) {
                abuf = 0;
                aphase ^= 1;
            }
        }
        if (!ok && lane == 0) {
            *(volatile int *)s_abort = 1;
            latch_error(PMN_DEVERR_WAIT_TIMEOUT);
        }
        if (BWD && pending) (void)warp_wait(bar_y, yphase, 1000000000ull);  // a copy may still be landing
        if (lane == 0) bulk_wait_group_all();
        __syncwarp();
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

// A row-major tensor [rows, width] of bytes or bf16 values; out-of-range elements of
// a loaded box read as zeros, of a stored box are not written.
bool make_map(CUtensorMap *m, const void *base, bool bf16, uint64_t width, uint64_t rows, uint32_t box_w,
              uint32_t box_rows, CUtensorMapSwizzle swizzle)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {width, rows}, strides[1] = {width * (bf16 ? 2 : 1)};
    cuuint32_t box[2] = {box_w, box_rows}, es[2] = {1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base),
              dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <bool BWD, int TBN>
pmn_status launch(const uint8_t *a, const uint8_t *b, const Args &args, cudaStream_t s)
{
    using C = Cfg<BWD, TBN>;
    const uint64_t m = (uint64_t)args.m, f = (uint64_t)args.f, k = (uint64_t)args.k, w = BWD ? 2 * f : f;
    const auto S32 = CU_TENSOR_MAP_SWIZZLE_32B, S64 = CU_TENSOR_MAP_SWIZZLE_64B, S128 = CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap ma, mb, mo, my;
    if (!make_map(&ma, a, false, k, m, 128, BM, S128) ||
        !make_map(&mb, b, false, k, (uint64_t)args.b_rows, 128, BWD ? TBN : TBN / 2, S128) ||
        !make_map(&mo, args.out, false, w, m, 32, 32, S32))
        return PMN_ERR_CUDA;
    my = mo;  // without y: not used
    if (args.y && !make_map(&my, args.y, true, 2 * f, m, 32, 32, S64)) return PMN_ERR_CUDA;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        return PMN_ERR_CUDA;
    auto kern = gated_kernel<BWD, TBN>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
        return PMN_ERR_CUDA;
    kern<<<(unsigned)sms, THREADS, C::SMEM_BYTES, s>>>(ma, mb, mo, my, args);
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
    return launch<false, 192>(a, b, args, reinterpret_cast<cudaStream_t>(stream));
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
    return launch<true, 192>(a, b, args, reinterpret_cast<cudaStream_t>(stream));
}
