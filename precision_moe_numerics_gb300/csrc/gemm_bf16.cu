// gemm_bf16.cu -- the bf16 products of experts whose row counts are ragged:
//   pmn_grouped_gemm_bf16               rows by expert, or sums over each expert's rows
//   pmn_w1_gemm_swiglu_bf16             gate and up projections and silu(gate) * up
//   pmn_dh_gemm_swiglu_backward_bf16    dH = dY . W2 and SwiGLU's gradient
// One persistent kernel of CTA pairs (tcgen05 kind::f16, float32 accumulators in TMEM).
// The tensor core's M side (256 TMEM lanes of a pair) are the columns of the output -- weight rows, or
// the columns of X in a weight gradient -- and its N side the output's rows, the ragged
// axis: a tile is 32 to 256 of them wide, in steps of 32, so an expert's rows are
// divided evenly and waste less than 32 of them where a tile with rows on the M side wastes up to
// 255.  An accumulator column is then a row of the output, 32 lanes of a warp write 32
// neighbours of it, and the rows behind a segment are simply not stored.
// What bounds it, f 1536, k 4096: the stages' loads, whose time does not fall with the tile's width.  A 64-deep stage of
// 256 rows takes 605 clocks where its MMAs take 512 (one expert's 16384 rows with k = n = 4096: 1.74 PFLOP/s, the
// backward of 16384 rows 138 us); 24 experts of 512 rows, two tiles of 256 each, take 196 us forward, of 384 rows,
// two of 192, 199.  8192 ragged rows, whose tiles are some 195 wide, take 170 us (tensor pipe active 58 %,
// DRAM 57 %; loads and products alone 158, products alone 121).  Float32 weight gradients of the same rows take
// 278 us, 254 where no expert has more than 512 rows; writing their 1.2 GB alone takes 164.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "../../include/pmn.h"
#include "args.cuh"
#include "numerics.cuh"
#include "sm100.cuh"
#include "tensormap.cuh"

using namespace pmn;
using namespace pmn::sm100;

uint64_t pmn_wait_limit_ns();  // gemm.cu: the limit of every bounded device wait

namespace {

__device__ int g_bf16_error = 0;

constexpr int MAX_GROUPS = 1024, MAX_DEVICES = 64;
constexpr uint32_t TMEM_COLS = 512;
constexpr int TILE = 256;        // output columns of a pair's tile, and most rows
constexpr int SIDE_BYTES = 128 * 128;  // a CTA's 128 x 64 of either operand
constexpr int RING_BYTES = 12 * SIDE_BYTES, MAX_SLOTS = 9;
constexpr int EW = 8, THREADS = 128 + 32 * EW;
constexpr int GROUPS = EW / 4;      // of four epilogue warps, which hold a CTA's 128 columns
constexpr int GROUP_BUF = 16384;   // rows on their way to or from memory
constexpr int BUF_OFF = RING_BYTES, BAR_OFF = BUF_OFF + GROUPS * GROUP_BUF;
constexpr int BARRIERS = 3 * MAX_SLOTS + 5 + 4 * GROUPS;
constexpr int CUM_OFF = BAR_OFF + 8 * BARRIERS + 16;
constexpr int SMEM_BYTES = CUM_OFF + (MAX_GROUPS / 32 + 1) * 4;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
constexpr int MT_BLOCK = 8;      // column tiles that share a tile's rows before the next rows are taken
constexpr uint64_t DRAIN_NS = 100000000ull;

// Rows times weights [n, k] and [k, n], the forward with SwiGLU, the gradient of h, sums over rows.
constexpr int ROWS_NK = 0, ROWS_KN = 1, GATED = 2, GATED_BACKWARD = 3, SUMS = 4;

struct Args {
    const int32_t *offsets;
    int groups;
    int64_t rows;      // of the ragged axis, all groups
    int64_t m, n, k;   // SUMS: out [groups, m, n]; else: weight rows n (of h: f), contraction k
    void *out;
    uint16_t *y;       // GATED: written (or NULL); GATED_BACKWARD: read
    uint64_t wait_ns;
};

struct Maps {
    CUtensorMap w;                   // M side
    CUtensorMap x, x64, x32, x16;    // N side: 128, 64, 32, 16 rows (SUMS: x alone, 64 columns of 64 rows)
    CUtensorMap out, y;              // the epilogue's pieces
};

struct Tile {
    int g, width;      // rows, a multiple of 32
    int64_t lo, hi;    // the group's rows
    int64_t r0;        // first output row
    int64_t row_end;   // output rows end here
    int c0;            // first output column of the pair
};

template <int FORM>
struct Form {
    static constexpr bool sums = FORM == SUMS, gated = FORM == GATED, backward = FORM == GATED_BACKWARD;
    static constexpr bool m_major_w = FORM == ROWS_KN || backward || sums;  // the M side's contiguous axis is M
    static constexpr int cols = gated ? TILE / 2 : TILE;                    // output columns of a pair's tile
    static constexpr int ch = backward ? 8 : 16;                            // output rows of an epilogue piece
};

__device__ __forceinline__ int tiles_of(int64_t rows) { return (int)((rows + TILE - 1) / TILE); }

// A last round of few tiles: each is cut into `shares` tiles of fewer rows, so that more pairs
// have one (backward of 16384 rows of one expert, 384 tiles on 76 pairs: 150 us for 139).
struct Tail {
    int full, shares;
};

// Tile t of all (a whole warp asks).  s_cum: row tiles before every 32nd group.
template <int FORM>
__device__ __forceinline__ Tile get_tile(int t, const Args &p, const int *s_cum, const Tail &tail, int lane)
{
    int sub = 0;
    if (t >= tail.full) {
        const int rest = t - tail.full;
        sub = rest % tail.shares;
        t = tail.full + rest / tail.shares;
    }
    using F = Form<FORM>;
    const int mt = (int)((p.n + F::cols - 1) / F::cols), u = t / mt;
    const int b = __popc(__ballot_sync(0xFFFFFFFFu, 32 * lane < p.groups && s_cum[lane] <= u)) - 1, g = 32 * b + lane;
    int lo = 0, hi = 0;
    if (g < p.groups) {
        lo = __ldg(p.offsets + g);
        hi = __ldg(p.offsets + g + 1);
    }
    const int n = g < p.groups ? tiles_of(F::sums ? p.m : hi - lo) : 0;
    int first = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, first, o);
        if (lane >= o) first += v;
    }
    first += s_cum[b] - n;
    // the last group that begins at or before u: those before it without tiles begin there too
    const int at = __popc(__ballot_sync(0xFFFFFFFFu, g < p.groups && first <= u)) - 1;
    Tile ti;
    ti.g = 32 * b + at;
    ti.lo = __shfl_sync(0xFFFFFFFFu, lo, at);
    ti.hi = __shfl_sync(0xFFFFFFFFu, hi, at);
    const int64_t rows = F::sums ? p.m : ti.hi - ti.lo;
    const int nt = tiles_of(rows);
    ti.width = (int)(((rows + nt - 1) / nt + 31) / 32 * 32);
    // column tiles in blocks: the tiles in flight read few rows and few weights
    const int local = t - __shfl_sync(0xFFFFFFFFu, first, at) * mt, block = local / (MT_BLOCK * nt), rest = local - block * MT_BLOCK * nt;
    const int bw = min(MT_BLOCK, mt - block * MT_BLOCK), ri = rest / bw;
    ti.c0 = (block * MT_BLOCK + rest - ri * bw) * F::cols;
    ti.r0 = (F::sums ? 0 : ti.lo) + (int64_t)ri * ti.width;
    ti.row_end = F::sums ? p.m : ti.hi;
    if (t >= tail.full && tail.shares > 1) {
        ti.row_end = min(ti.row_end, ti.r0 + ti.width);
        ti.width = ((ti.width + tail.shares - 1) / tail.shares + 31) / 32 * 32;
        ti.r0 += (int64_t)sub * ti.width;
    }
    return ti;
}

// 64-deep stages of a tile.
template <int FORM>
__device__ __forceinline__ int stages_of(const Tile &ti, const Args &p)
{
    return ti.r0 < ti.row_end ? (int)(((Form<FORM>::sums ? ti.hi - ti.lo : p.k) + 63) / 64) : 0;  // (a share may be empty)
}

// The tensor core truncates each of its additions to float32, an error that grows with their
// number (sums over 16384 rows: 1.9e-5 of their norm, where rounded additions have 1.9e-7; sums of one sign lose
// 1.4 x 2^-24 an addition).  Where the output is float32 too, a tile's sums are therefore made in runs of RUN stages, added
// up in registers and rounded to nearest: 4.8e-7.  RUN 12: 7.3e-7, RUN 4: 2.5e-7; dw1 of 8192 rows of 24 experts takes
// 255 us without runs, 274, 280 and 319 with 12, 8 and 4, the rows' products 2 to 5 % more with 8.
// A bf16 output's rounding, up to 3.9e-3, hides that for as long as K is a layer's width: w1, dx and dh of the training
// batch are 1.65917e-3, 1.65559e-3 and 1.65926e-3 of the norm off with and without runs of 1024 of K, which take
// 170 -> 173, 168 -> 171 and 140 -> 186 us.  Sums over rows have no such bound (2^20 of one sign would be off by 5.4e-3
// before they are rounded): LONG, bf16 outputs of more than LONG_K, has runs of 4096.  (16384 of one sign without
// lose 8.5e-5; dw1 of 8192 rows in bf16 takes 232 us without runs, 239 with these.)
constexpr int64_t LONG_K = 16384;
template <int FORM, typename OUT, bool LONG>
struct Runs {
    static constexpr bool split = LONG || (sizeof(OUT) == 4 && !Form<FORM>::gated && !Form<FORM>::backward);
    static constexpr int RUN = LONG ? 64 : split ? 8 : 1 << 30;
};

// The ring of stages.  A slot holds the weights' 16 KB and the rows: 4 KB of a tile of up to 64,
// 16 KB of up to 256; what is in flight counts (loads and products of the forward of 8192 rows: 3 slots
// of 32 KB 211 us, 4 182, 5 162, 6 158).  A tile of the other kind than the one before starts
// at slot 0, once the stages before it have been read.
template <int FORM>
struct Ring {
    uint32_t kind = 2, slot = 0, phases = 0;  // bit s: parity of slot s's next use
    __device__ __forceinline__ static uint32_t kind_of(const Tile &ti)
    {
        return Form<FORM>::sums || ti.width > 64 ? 1u : 0u;
    }
    __device__ __forceinline__ uint32_t slots() const { return kind == 0 ? 9u : 6u; }
    __device__ __forceinline__ uint32_t bytes() const { return kind == 0 ? 20480u : 32768u; }
    __device__ __forceinline__ uint32_t parity() const { return (phases >> slot) & 1u; }
    __device__ __forceinline__ void enter(const Tile &ti)
    {
        const uint32_t k = kind_of(ti);
        if (k != kind) slot = 0;
        kind = k;
    }
    __device__ __forceinline__ void step()
    {
        phases ^= 1u << slot;
        if (++slot == slots()) slot = 0;
    }
};
static_assert(9 * 20480 <= RING_BYTES && 6 * 32768 <= RING_BYTES, "slots");

__device__ __forceinline__ void latch_error(int bit) { atomicOr(&g_bf16_error, bit); }

__device__ __forceinline__ void tma_3d_pair(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_5d_pair(uint32_t dst, const CUtensorMap *m, uint32_t bar, int a, int b, int c, int d,
                                            int e)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *m, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// The descriptors' high words are constants (smem_desc: 1024 bytes between groups of 8 rows,
// version, 128-byte swizzle); the low ones hold the address and the other stride.
constexpr uint32_t DESC_HIGH = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ void mma_bf16_pair(uint32_t el, uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc,
                                              uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(el), "n"(DESC_HIGH)
        : "memory");
}

__device__ __forceinline__ void store_one(uint16_t *p, float v)
{
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    *p = *reinterpret_cast<const uint16_t *>(&b);
}
__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Roles: warp 0 loads by TMA, warp 1 of the leader issues the pair's MMAs, warp 2 (SUMS) clears
// rows that are not the group's, warps 4.. store.  Every wait is bounded: on a timeout an
// error bit is latched and the CTA winds down.
template <int FORM, typename OUT, bool LONG>
__global__ void __launch_bounds__(THREADS, 1) bf16_kernel(const __grid_constant__ Maps maps, const Args p)
{
    using F = Form<FORM>;
    using R = Runs<FORM, OUT, LONG>;
    constexpr int RUN = R::RUN;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw;
    asm volatile("" : "+l"(smem));
    const uint32_t ring = smem_u32(smem);
    const uint32_t bar_full = ring + BAR_OFF, bar_empty = bar_full + 8 * MAX_SLOTS, bar_land = bar_empty + 8 * MAX_SLOTS;
    const uint32_t bar_acc_full = bar_land + 8 * MAX_SLOTS, bar_acc_empty = bar_acc_full + 16, bar_drain = bar_acc_empty + 16;
    const uint32_t bar_y = bar_drain + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + BAR_OFF + 8 * BARRIERS);
    int *s_abort = reinterpret_cast<int *>(tmem_slot + 1);
    int *s_total = s_abort + 1;
    int *s_cum = reinterpret_cast<int *>(smem + CUM_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int tile0 = blockIdx.x / 2, tstep = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < MAX_SLOTS; ++s) {
            mbar_init(bar_full + 8 * s, F::sums ? 2 : 1);  // SUMS: each CTA's word that its rows are there, and clean
            mbar_init(bar_empty + 8 * s, 1);
            mbar_init(bar_land + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_acc_full + 8 * b, 1);
            mbar_init(bar_acc_empty + 8 * b, 2 * EW);
        }
        mbar_init(bar_drain, 1);
        for (int b = 0; b < 4 * GROUPS; ++b) mbar_init(bar_y + 8 * b, 1);
        *s_abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.x);
    }
    if (warp == 0) {
        __syncwarp();
        tmem_alloc_ct<2>(smem_u32(tmem_slot), TMEM_COLS);
    }
    if (warp == 1) {
        // row tiles before every 32nd group; offsets that are not monotone and in range run no tile
        const int mt = (int)((p.n + F::cols - 1) / F::cols);
        int base = 0;
        bool good = true;
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
            const int g = g0 + lane;
            int lo = 0, hi = 0;
            if (g < p.groups) {
                lo = __ldg(p.offsets + g);
                hi = __ldg(p.offsets + g + 1);
                if (lo < 0 || hi < lo || hi > p.rows) good = false;
            }
            if (lane == 0) s_cum[g0 / 32] = base;
            base += __reduce_add_sync(0xFFFFFFFFu, g < p.groups ? tiles_of(F::sums ? p.m : hi - lo) : 0);
        }
        good = __all_sync(0xFFFFFFFFu, good);
        if (lane == 0) {
            *s_total = good ? base * mt : 0;
            if (!good && blockIdx.x == 0) latch_error(PMN_DEVERR_BAD_OFFSETS);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the pair's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int all = __shfl_sync(0xFFFFFFFFu, *s_total, 0), rest = all % tstep;
    const Tail tail{all - rest, rest > 0 ? min(8, tstep / rest) : 1};
    const int total = tail.full + rest * tail.shares;
    auto give_up = [&]() {  // a wait ran out: every role winds down
        if (lane == 0) {
            *(volatile int *)s_abort = 1;
            latch_error(PMN_DEVERR_WAIT_TIMEOUT);
        }
    };

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        Ring<FORM> at;
        uint32_t issued = 0;
        bool ok = true;
        for (int t = tile0; t < total && ok; t += tstep) {
            const Tile ti = get_tile<FORM>(t, p, s_cum, tail, lane);
            const int nks = stages_of<FORM>(ti, p), half = ti.width / 2;
            const int row = (int)ti.r0 + half * rank;  // of the N side, first accumulator
            if (at.kind != 2 && at.kind != Ring<FORM>::kind_of(ti))
                for (uint32_t s = 0; s < at.slots() && ok; ++s) {
                    ok = warp_wait(bar_empty + 8 * s, ((at.phases >> s) & 1u) ^ 1, p.wait_ns);
                    if (!ok) give_up();
                }
            at.enter(ti);
            for (int ks = 0; ks < nks && ok; ++ks) {
                ok = warp_wait(bar_empty + 8 * at.slot, at.parity() ^ 1, p.wait_ns);
                if (!ok || __any_sync(0xFFFFFFFFu, *(volatile int *)s_abort != 0)) {
                    if (!ok) give_up();
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    const uint32_t w = ring + at.slot * at.bytes(), x = w + SIDE_BYTES, fb = bar_full + 8 * at.slot, lb = leader_addr(fb);
                    const int k = 64 * ks;
                    if constexpr (F::sums) {
                        // Where the group ends inside 16 rows, this CTA's warp 2 clears the rest of them and
                        // reports the stage; else both CTAs report here.
                        const int64_t k0 = ti.lo + k;
                        const int boxes = (half + 63) / 64;
                        if (ti.hi - k0 < 64 && (ti.hi - k0) % 16 != 0) {
                            const uint32_t own = bar_land + 8 * at.slot;
                            mbar_arrive_expect_tx(own, 8192 * (2 + boxes));
                            for (int b = 0; b < 2; ++b) tma_load_2d(w + 8192 * b, &maps.w, own, ti.c0 + 128 * rank + 64 * b, (int)k0);
                            for (int b = 0; b < boxes; ++b) tma_load_2d(x + 8192 * b, &maps.x, own, row + 64 * b, (int)k0);
                        } else {
                            if (rank == 0) mbar_arrive_expect_tx(fb, 2 * 8192 * (2 + boxes));
                            else mbar_arrive_leader(fb);
                            for (int b = 0; b < 2; ++b) tma_load_2d_pair(w + 8192 * b, &maps.w, lb, ti.c0 + 128 * rank + 64 * b, (int)k0);
                            for (int b = 0; b < boxes; ++b) tma_load_2d_pair(x + 8192 * b, &maps.x, lb, row + 64 * b, (int)k0);
                        }
                    } else {
                        if (rank == 0) mbar_arrive_expect_tx(fb, 2 * (SIDE_BYTES + 128 * half));
                        if constexpr (FORM == ROWS_NK) {
                            tma_3d_pair(w, &maps.w, lb, k, ti.c0 + 128 * rank, ti.g);
                        } else if constexpr (FORM == GATED) {
                            tma_5d_pair(w, &maps.w, lb, k, 0, 0, (ti.c0 + 64 * rank) / 16, ti.g);
                        } else {
                            tma_3d_pair(w, &maps.w, lb, ti.c0 + 128 * rank, k, ti.g);
                            tma_3d_pair(w + 8192, &maps.w, lb, ti.c0 + 128 * rank + 64, k, ti.g);
                        }
                        // few boxes: with 16 rows in each the forward of 8192 rows takes 12 % longer
                        if (half & 128) tma_load_2d_pair(x, &maps.x, lb, k, row);
                        if (half & 64) tma_load_2d_pair(x, &maps.x64, lb, k, row);
                        if (half & 32) tma_load_2d_pair(x + 128 * (half & 64), &maps.x32, lb, k, row + (half & 64));
                        if (half & 16) tma_load_2d_pair(x + 128 * (half & 96), &maps.x16, lb, k, row + (half & 96));
                    }
                }
                __syncwarp();
                issued |= 1u << at.slot;
                at.step();
            }
        }
        // no copy may still be landing when the CTA ends; a pair's copies are counted by
        // its leader, and both CTAs end together
        for (int s = 0; s < MAX_SLOTS; ++s)
            if (rank == 0 && (issued & (1u << s))) (void)warp_wait(bar_full + 8 * s, ((at.phases >> s) & 1u) ^ 1, DRAIN_NS);
        if (*(volatile int *)s_abort) {  // one side may have given up before the other: let copies land
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 10000000ull) {
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        // The whole warp walks the loop; one elected lane issues.
        if (rank == 0) {
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0), el = elect_one();
            Ring<FORM> at;
            uint32_t abuf = 0, aphase = 0;
            bool ok = true, ready = false;
            // strides between 64-wide blocks of M (N) where that axis is contiguous: 8192 bytes
            constexpr uint32_t W_LOW = (F::m_major_w ? 8192u >> 4 : 1u) << 16, X_LOW = (F::sums ? 8192u >> 4 : 1u) << 16;
            // 16 of K per MMA: 32 bytes of the swizzled rows where K is contiguous, 16 rows where it is not
            constexpr uint32_t W_STEP = (F::m_major_w ? 2048u : 32u) >> 4, X_STEP = (F::sums ? 2048u : 32u) >> 4;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                ok = warp_wait(bar, parity, p.wait_ns);
                if (!ok) give_up();
                return ok;
            };
            Tile ti, next;
            if (tile0 < total) ti = get_tile<FORM>(tile0, p, s_cum, tail, lane);
            for (int t = tile0; t < total && ok; t += tstep, ti = next) {
                const int nks = stages_of<FORM>(ti, p);
                at.enter(ti);
                const uint32_t bytes = at.bytes() >> 4, base = ring >> 4;
                // D float32, A and B bf16, M = 256
                const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (F::m_major_w ? 1u << 15 : 0u) |
                                       (F::sums ? 1u << 16 : 0u) | ((uint32_t)(ti.width >> 3) << 17) | (16u << 24);
                if (!wait(bar_acc_empty + 8 * abuf, aphase ^ 1) || __any_sync(0xFFFFFFFFu, *(volatile int *)s_abort != 0)) break;
                uint32_t d = tm + abuf * TILE;
                auto next_acc = [&]() {
                    tc_commit_ct<2>(el, bar_acc_full + 8 * abuf);
                    if (++abuf == 2) {
                        abuf = 0;
                        aphase ^= 1;
                    }
                };
                for (int ks = 0; ks < nks; ++ks) {
                    const bool begin = ks % RUN == 0;
                    if (begin && ks > 0) {
                        next_acc();
                        if (!wait(bar_acc_empty + 8 * abuf, aphase ^ 1)) break;
                        d = tm + abuf * TILE;
                    }
                    // asked for a stage ahead, the answer is there when it is needed
                    if (__all_sync(0xFFFFFFFFu, ready) == 0 && !wait(bar_full + 8 * at.slot, at.parity())) break;
                    tc_fence_after();
                    const uint32_t slot = at.slot;
                    at.step();
                    ready = ks + 1 < nks && mbar_test(bar_full + 8 * at.slot, at.parity());
                    const uint32_t w = (base + slot * bytes) | W_LOW, x = (base + slot * bytes + (SIDE_BYTES >> 4)) | X_LOW;
                    const int steps = F::sums ? (int)min((int64_t)4, (ti.hi - ti.lo - 64 * ks + 15) / 16) : 4;
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        if (!F::sums || s < steps) mma_bf16_pair(el, d, w + W_STEP * s, x + X_STEP * s, idesc, !begin || s > 0);
                    tc_commit_ct<2>(el, bar_empty + 8 * slot);
                }
                if (!ok) break;
                next_acc();
                // the next tile is looked up while MMAs run
                if (t + tstep < total) next = get_tile<FORM>(t + tstep, p, s_cum, tail, lane);
            }
            if (elect_one()) tc_commit_own<2>(bar_drain);  // every tcgen05 operation of this warp has completed
            __syncwarp();
            (void)warp_wait(bar_drain, 0, DRAIN_NS);
        }
        __syncwarp();
    } else if (F::sums && warp == 2) {
        // ---------------------------------------------------- rows that are not the group's
        // A last stage of a group that ends inside 16 rows: those up to the next 16 become zeros (another
        // group's rows would enter the sums, and a NaN among them even times zero).
        Ring<FORM> at;
        uint32_t parity = 0;
        bool ok = true;
        for (int t = tile0; t < total && ok; t += tstep) {
            const Tile ti = get_tile<FORM>(t, p, s_cum, tail, lane);
            const int nks = stages_of<FORM>(ti, p), rest = (int)((ti.hi - ti.lo) & 63);
            at.enter(ti);
            for (int ks = 0; ks < nks; ++ks, at.step()) {
                if (ks + 1 < nks || rest % 16 == 0) continue;
                ok = warp_wait(bar_land + 8 * at.slot, (parity >> at.slot) & 1u, p.wait_ns);
                if (!ok) {
                    give_up();
                    break;
                }
                parity ^= 1u << at.slot;
                const int blocks = 2 + (ti.width / 2 + 63) / 64;
                for (int b = 0; b < blocks; ++b) {
                    uint4 *d = reinterpret_cast<uint4 *>(smem + at.slot * at.bytes() + 8192 * b);
                    for (int i = 8 * rest + lane; i < 8 * ((rest + 15) & ~15); i += 32) d[i] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_leader(bar_full + 8 * at.slot);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------- epilogue
        // A lane holds one column of the output, a register one row.  Four warps take every other
        // CH rows of the CTA's 128 columns, put them into shared memory and have TMA write them:
        // the stores then cost the warps nothing and arrive as whole lines (boxes of 32 columns: dw1
        // of 8192 rows 262 us for 252).  Rows behind the segment's end may not be
        // written, so the last few of a segment are stored singly.
        constexpr int CH = F::ch, COLS = F::cols / 2;
        constexpr int PIECE = F::gated ? 8192 : F::backward ? CH * 2 * COLS * 2 : CH * COLS * (int)sizeof(OUT);  // bytes
        constexpr int BUFS = GROUP_BUF / PIECE;
        const int wu = __shfl_sync(0xFFFFFFFFu, warp, 0), quad = wu & 3, group = (wu - 4) >> 2;
        uint8_t *const buf0 = smem + BUF_OFF + group * GROUP_BUF;
        const uint32_t bufs0 = ring + BUF_OFF + group * GROUP_BUF, ybar = bar_y + 32 * group;
        const bool issuer = quad == 0 && lane == 0;
        uint32_t abuf = 0, aphase = 0, n = 0;  // n: pieces so far
        bool ok = true;
        auto pieces_of = [&](const Tile &ti) {
            return ti.c0 + COLS * rank < p.n ? (int)((min((int64_t)ti.width, ti.row_end - ti.r0) + CH - 1) / CH) : 0;
        };
        auto meet = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); };
        // GATED_BACKWARD: gate and up come by TMA too, BUFS - 1 pieces ahead, into the buffer that takes their gradients
        int at = tile0, ac = group;  // tile, piece
        uint32_t asked = 0;
        Tile ahead;
        auto fetch = [&]() {
            while (at < total && ac >= pieces_of(ahead)) {
                ac = group;
                at += tstep;
                if (at < total) ahead = get_tile<FORM>(at, p, s_cum, tail, lane);
            }
            if (at >= total) return;
            if (lane == 0) {
                const uint32_t b = asked % BUFS, bar = ybar + 8 * b;
                mbar_arrive_expect_tx(bar, PIECE);
                tma_load_3d(bufs0 + PIECE * b, &maps.y, bar, ahead.c0 + COLS * rank, 0, (int)ahead.r0 + CH * ac);
            }
            __syncwarp();
            ++asked;
            ac += GROUPS;
        };
        if (F::backward && quad == 0) {
            if (at < total) ahead = get_tile<FORM>(at, p, s_cum, tail, lane);
            for (int i = 0; i < BUFS - 1; ++i) fetch();
        }
        for (int t = tile0; t < total; t += tstep) {
            const Tile ti = get_tile<FORM>(t, p, s_cum, tail, lane);
            const int pieces = pieces_of(ti), col0 = ti.c0 + COLS * rank;
            const bool nothing = F::sums && ti.hi == ti.lo;  // a sum over no rows
            // after a timeout the four warps go on to the end together, without waiting or storing
            auto take = [&]() {
                ok = ok && warp_wait(bar_acc_full + 8 * abuf, aphase, p.wait_ns);
                if (!ok) give_up();
                tc_fence_after();
                return tmem + ((uint32_t)(32 * quad) << 16) + abuf * TILE;
            };
            auto load = [&](uint32_t acc, int c, float(&v)[CH]) {
                if constexpr (CH == 16) tmem_ld_32x32b_x16(acc + CH * c, reinterpret_cast<uint32_t(&)[CH]>(v));
                else tmem_ld_32x32b_x8(acc + CH * c, reinterpret_cast<uint32_t(&)[CH]>(v));
                tmem_ld_wait();
            };
            auto give_back = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_leader(bar_acc_empty + 8 * abuf);
                if (++abuf == 2) {
                    abuf = 0;
                    aphase ^= 1;
                }
            };
            auto emit = [&](int c, float(&v)[CH]) {
                const uint32_t which = n % BUFS;
                uint8_t *const buf = buf0 + PIECE * which;
                if (nothing) {
#pragma unroll
                    for (int j = 0; j < CH; ++j) v[j] = 0.0f;
                }
                const int64_t r0 = ti.r0 + CH * c;
                const int rows = (int)min((int64_t)CH, ti.row_end - r0);
                const bool whole = F::sums || rows == CH;
                if constexpr (F::gated) {
                    // lanes 0 .. 15 gate, 16 .. 31 up of the same 16 columns: the halves trade
                    // values, so that the lower half makes h of the even rows, the upper of the odd
                    const bool up = lane >= 16;
                    const int cl = 16 * quad + (lane & 15), col = col0 + cl;
                    uint16_t *y = reinterpret_cast<uint16_t *>(buf), *h = y + CH * 2 * COLS;  // [CH][2][COLS], [CH][COLS]
#pragma unroll
                    for (int j = 0; j < CH; j += 2) {
                        const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? v[j] : v[j + 1], 16);
                        const float g = up ? got : v[j], u = up ? v[j + 1] : got;
                        store_one(y + (2 * j + up) * COLS + cl, v[j]);
                        store_one(y + (2 * j + 2 + up) * COLS + cl, v[j + 1]);
                        store_one(h + (j + up) * COLS + cl, __fmul_rn(__fmul_rn(g, sigmoid(g)), u));
                    }
                    __syncwarp();
                    if (!whole && ok && col < p.n)
                        for (int j = 0; j < rows; ++j) {
                            if (p.y) p.y[(r0 + j) * 2 * p.n + col + (up ? p.n : 0)] = y[(2 * j + up) * COLS + cl];
                            if (!up) static_cast<uint16_t *>(p.out)[(r0 + j) * p.n + col] = h[j * COLS + cl];
                        }
                } else if constexpr (F::backward) {
                    const int cl = 32 * quad + lane, col = col0 + cl;
                    uint16_t *b = reinterpret_cast<uint16_t *>(buf);  // [CH][2][COLS]: gate, up
                    ok = ok && warp_wait(ybar + 8 * which, (n / BUFS) & 1u, p.wait_ns);
                    if (!ok) give_up();
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        const float g = bf16_value(b[2 * j * COLS + cl]), u = bf16_value(b[(2 * j + 1) * COLS + cl]), dh = v[j];
                        const float s = sigmoid(g), a = __fmul_rn(dh, s);
                        store_one(b + 2 * j * COLS + cl, __fmul_rn(__fmul_rn(a, u), fmaf(g, 1.0f - s, 1.0f)));
                        store_one(b + (2 * j + 1) * COLS + cl, __fmul_rn(a, g));
                    }
                    if (!whole && ok && col < p.n) {
                        uint16_t *o = static_cast<uint16_t *>(p.out) + r0 * 2 * p.n + col;
                        for (int j = 0; j < rows; ++j) {
                            o[j * 2 * p.n] = b[2 * j * COLS + cl];
                            o[j * 2 * p.n + p.n] = b[(2 * j + 1) * COLS + cl];
                        }
                    }
                } else {
                    const int cl = 32 * quad + lane, col = col0 + cl;
                    OUT *b = reinterpret_cast<OUT *>(buf);  // [CH][COLS]
#pragma unroll
                    for (int j = 0; j < CH; ++j) store_one(b + j * COLS + cl, v[j]);
                    if (!whole && ok && col < p.n) {
                        OUT *o = static_cast<OUT *>(p.out) + r0 * p.n + col;
                        for (int j = 0; j < rows; ++j) o[j * p.n] = b[j * COLS + cl];
                    }
                }
                fence_proxy_async_smem();
                if (issuer) bulk_wait_group_read<BUFS - 2>();  // the next piece's buffer has been read
                meet();
                if (quad == 0) {
                    if (lane == 0) {
                        const uint32_t d = bufs0 + PIECE * which;
                        if (whole && ok) {
                            if constexpr (F::gated) {
                                if (p.y) tma_store_3d(&maps.y, d, col0, 0, (int)r0);
                                tma_store_2d(&maps.out, d + CH * 2 * COLS * 2, col0, (int)r0);
                            } else if constexpr (F::backward) {
                                tma_store_3d(&maps.out, d, col0, 0, (int)r0);
                            } else if constexpr (F::sums) {
                                tma_store_3d(&maps.out, d, col0, (int)r0, ti.g);
                            } else {
                                tma_store_2d(&maps.out, d, col0, (int)r0);
                            }
                        }
                        bulk_commit_group();
                    }
                    __syncwarp();
                    if (F::backward && ok) {  // the buffer of the piece before this one
                        if (lane == 0) bulk_wait_group_read<1>();
                        fetch();
                    }
                }
                ++n;
            };
            const int runs = (stages_of<FORM>(ti, p) + RUN - 1) / RUN;
            if (!R::split || runs <= 1) {
                const uint32_t acc = take();
                for (int c = group; c < pieces; c += GROUPS) {
                    float v[CH];
                    load(acc, c, v);
                    emit(c, v);
                }
                give_back();
            } else if constexpr (R::split) {
                constexpr int MOST = TILE / CH / GROUPS;
                float sum[MOST][CH];
#pragma unroll
                for (int i = 0; i < MOST; ++i)
#pragma unroll
                    for (int j = 0; j < CH; ++j) sum[i][j] = -0.0f;
                for (int run = 1; run < runs; ++run) {
                    const uint32_t acc = take();
#pragma unroll
                    for (int i = 0; i < MOST; ++i)
                        if (group + GROUPS * i < pieces) {
                            float v[CH];
                            load(acc, group + GROUPS * i, v);
#pragma unroll
                            for (int j = 0; j < CH; ++j) sum[i][j] = __fadd_rn(sum[i][j], v[j]);
                        }
                    give_back();
                }
                const uint32_t acc = take();
#pragma unroll
                for (int i = 0; i < MOST; ++i)
                    if (group + GROUPS * i < pieces) {
                        float v[CH];
                        load(acc, group + GROUPS * i, v);
#pragma unroll
                        for (int j = 0; j < CH; ++j) v[j] = __fadd_rn(sum[i][j], v[j]);
                        emit(group + GROUPS * i, v);
                    }
                give_back();
            }
        }
        if (F::backward && quad == 0 && !ok)  // loads that nobody waited for may still be landing
            for (int b = 0; b < BUFS; ++b) {
                (void)warp_wait(ybar + 8 * b, 0, DRAIN_NS);
                (void)warp_wait(ybar + 8 * b, 1, DRAIN_NS);
            }
        if (lane == 0) bulk_wait_group_all();  // shared memory is read until then
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA's memory is still in use by the other
    tc_fence_after();
    if (warp == 0) tmem_dealloc_ct<2>(tmem, TMEM_COLS);
    cluster_sync();
}

// ---------------------------------------------------------------- few rows
// The forward calls for a handful of rows (single tokens of a serving loop): their time is that of
// reading the weights, which 256-column tiles would spread over few SMs (one row, f 1536, k 4096: 7.6 us for a floor of
// 3.7; 1.8 of them are the launch and finding the expert).  A CTA takes
// 16 weight rows (gated: 8 gate rows and the 8 up rows of the same columns) for up to 8 NC
// rows of one expert; its warps share K, each lane loads 16 bytes of a weight row at a time, which are
// the tensor core's operands as they are (mma.sync; what it sees as its K is the lanes'
// order, the same for weights and rows).  The warps' sums meet in shared memory.
constexpr int FEW_THREADS = 256;

__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// grid: blocks of 16 weight rows x chunks of 8 NC rows of an expert (as many as there can be)
template <bool GATED, typename OUT, int NC>
__global__ void __launch_bounds__(FEW_THREADS, 3)
    few_rows_kernel(const uint16_t *__restrict__ x, int64_t ldx, const uint16_t *__restrict__ w, const Args p)
{
    constexpr int WARPS = FEW_THREADS / 32, CHUNK = 8 * NC, FEW_UNROLL = NC > 1 ? 2 : 4;
    __shared__ int s_sum[WARPS], s_found[3];
    __shared__ float s_part[WARPS][16][CHUNK + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, unit = blockIdx.y;
    // the expert whose chunk this is
    if (threadIdx.x == 0) s_found[0] = -1;
    int base = 0;
    bool bad = false;
    for (int g0 = 0; g0 < p.groups; g0 += FEW_THREADS) {
        const int g = g0 + threadIdx.x;
        int lo = 0, hi = 0;
        if (g < p.groups) {
            lo = __ldg(p.offsets + g);
            hi = __ldg(p.offsets + g + 1);
            bad = bad || lo < 0 || hi < lo || hi > p.rows;
        }
        const int n = (hi - lo + CHUNK - 1) / CHUNK;
        int run = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, run, o);
            if (lane >= o) run += v;
        }
        if (lane == 31) s_sum[warp] = run;
        __syncthreads();
        int before = base, all = base;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            if (i < warp) before += s_sum[i];
            all += s_sum[i];
        }
        if (unit >= before + run - n && unit < before + run) {
            s_found[0] = g;
            s_found[1] = lo + CHUNK * (unit - (before + run - n));
            s_found[2] = hi;
        }
        base = all;
        __syncthreads();
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && unit == 0) latch_error(PMN_DEVERR_BAD_OFFSETS);
        return;
    }
    const int g = s_found[0], r0 = s_found[1], m = min(CHUNK, s_found[2] - r0);
    if (g < 0) return;

    const int r = lane >> 2, q = lane & 3;
    const int64_t col = (GATED ? 8 : 16) * (int64_t)blockIdx.x + r, cols = p.n;  // p.n: of the output
    const uint16_t *w0 = w + ((int64_t)g * (GATED ? 2 * cols : cols) + min(col, cols - 1)) * p.k;
    const uint16_t *w1 = w + ((int64_t)g * (GATED ? 2 * cols : cols) + (GATED ? cols + min(col, cols - 1) : min(col + 8, cols - 1))) * p.k;
    const uint16_t *xr[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) xr[j] = x + (r0 + min(8 * j + r, m - 1)) * ldx;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float sum[NC][4] = {};
    // (the same passes for all lanes of a warp, which multiply together; a pass's sums are added to those before
    // it rounded to nearest, where the tensor core would truncate)
    for (int64_t kw = 32 * FEW_UNROLL * warp; kw < p.k; kw += 32 * FEW_UNROLL * WARPS) {
        uint4 a[FEW_UNROLL], b[FEW_UNROLL], c[FEW_UNROLL][NC];
#pragma unroll
        for (int i = 0; i < FEW_UNROLL; ++i) {
            const int64_t k = kw + 32 * i + 8 * q;
            const bool on = k < p.k;
            a[i] = on ? __ldcs(reinterpret_cast<const uint4 *>(w0 + k)) : zero;
            b[i] = on ? __ldcs(reinterpret_cast<const uint4 *>(w1 + k)) : zero;
#pragma unroll
            for (int j = 0; j < NC; ++j)
                c[i][j] = on && 8 * j + r < m ? __ldg(reinterpret_cast<const uint4 *>(xr[j] + k)) : zero;
        }
        __syncwarp();
        float acc[NC][4] = {};
#pragma unroll
        for (int i = 0; i < FEW_UNROLL; ++i)
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                mma_m16n8k16(acc[j], a[i].x, b[i].x, a[i].y, b[i].y, c[i][j].x, c[i][j].y);
                mma_m16n8k16(acc[j], a[i].z, b[i].z, a[i].w, b[i].w, c[i][j].z, c[i][j].w);
            }
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) sum[j][v] = __fadd_rn(sum[j][v], acc[j][v]);
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        s_part[warp][r][8 * j + 2 * q] = sum[j][0];
        s_part[warp][r][8 * j + 2 * q + 1] = sum[j][1];
        s_part[warp][r + 8][8 * j + 2 * q] = sum[j][2];
        s_part[warp][r + 8][8 * j + 2 * q + 1] = sum[j][3];
    }
    __syncthreads();
    constexpr int OUTS = GATED ? 8 : 16;
    for (int i = threadIdx.x; i < OUTS * CHUNK; i += FEW_THREADS) {
        const int c = i % OUTS, n = i / OUTS;
        const int64_t oc = OUTS * (int64_t)blockIdx.x + c;
        if (n >= m || oc >= cols) continue;
        float s = 0.0f, u = 0.0f;
#pragma unroll
        for (int v = 0; v < WARPS; ++v) {
            s = __fadd_rn(s, s_part[v][c][n]);
            if (GATED) u = __fadd_rn(u, s_part[v][c + 8][n]);
        }
        if (GATED) {
            if (p.y) {
                store_one(p.y + (r0 + n) * 2 * cols + oc, s);
                store_one(p.y + (r0 + n) * 2 * cols + cols + oc, u);
            }
            s = __fmul_rn(__fmul_rn(s, sigmoid(s)), u);
        }
        store_one(static_cast<OUT *>(p.out) + (r0 + n) * cols + oc, s);
    }
}

template <bool GATED, typename OUT, int NC>
pmn_status launch_few_of(const void *a, int64_t lda, const void *b, const Args &p, cudaStream_t s)
{
    const dim3 grid((unsigned)((p.n + (GATED ? 7 : 15)) / (GATED ? 8 : 16)),
                    (unsigned)std::min<int64_t>(p.rows, p.rows / (8 * NC) + p.groups));
    few_rows_kernel<GATED, OUT, NC><<<grid, FEW_THREADS, 0, s>>>(static_cast<const uint16_t *>(a), lda,
                                                                  static_cast<const uint16_t *>(b), p);
    return cudaGetLastError() == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

template <bool GATED, typename OUT>
pmn_status launch_few(int chunks, const void *a, int64_t lda, const void *b, const Args &p, cudaStream_t s)
{
    return chunks == 1 ? launch_few_of<GATED, OUT, 1>(a, lda, b, p, s) : launch_few_of<GATED, OUT, 2>(a, lda, b, p, s);
}

// ====================================================================== host
bool make_map(CUtensorMap *m, const void *base, int rank, const uint64_t *dims, const uint64_t *strides, const uint32_t *box,
              CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, bool swizzle = true)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    cuuint64_t d[5], st[4];
    cuuint32_t b[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i + 1 < rank) st[i] = strides[i];
    }
    return fn(m, type, rank, const_cast<void *>(base), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The epilogue's pieces, `box` of [outer, middle, n].
bool piece_map(CUtensorMap *m, const void *base, int64_t outer, int64_t middle, int64_t n, int kind, int b2, int b1, int b0)
{
    const uint64_t b = kind == PMN_OUT_F32 ? 4 : 2;
    const uint64_t dims[3] = {(uint64_t)n, (uint64_t)middle, (uint64_t)outer}, st[2] = {n * b, (uint64_t)middle * n * b};
    const uint32_t box[3] = {(uint32_t)b0, (uint32_t)b1, (uint32_t)b2};
    return make_map(m, base, b2 ? 3 : 2, dims, st, box,
                    kind == PMN_OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, false);
}

// rows [rows, width] of pitch ld, 64 columns (128 bytes) of box_rows rows
bool rows_map(CUtensorMap *m, const void *base, int64_t width, int64_t rows, int64_t ld, int box_rows)
{
    const uint64_t dims[2] = {(uint64_t)width, (uint64_t)rows}, st[1] = {(uint64_t)ld * 2};
    const uint32_t box[2] = {64, (uint32_t)box_rows};
    return make_map(m, base, 2, dims, st, box);
}

template <int FORM, typename OUT, bool LONG>
pmn_status launch_of(const Maps &maps, const Args &args, cudaStream_t s)
{
    auto kern = bf16_kernel<FORM, OUT, LONG>;
    static std::atomic<int> sm_count[MAX_DEVICES];  // of each device this kernel has been set up on
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return PMN_ERR_CUDA;
    int sms = dev < MAX_DEVICES ? sm_count[dev].load(std::memory_order_acquire) : 0;
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 2 ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) != cudaSuccess)
            return PMN_ERR_CUDA;
        if (dev < MAX_DEVICES) sm_count[dev].store(sms, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms / 2 * 2));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, args) == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

template <int FORM, typename OUT>
pmn_status launch(const Maps &maps, const Args &args, cudaStream_t s)
{
    if constexpr (sizeof(OUT) == 2)
        if ((FORM == SUMS ? args.rows : args.k) > LONG_K) return launch_of<FORM, OUT, true>(maps, args, s);
    return launch_of<FORM, OUT, false>(maps, args, s);
}

constexpr int64_t LIMIT = int64_t(1) << 31;

// Sizes that every form asks for: rows in 16-byte pieces, 32-bit coordinates and tile counts.
pmn_status check_sizes(int groups, int64_t rows, int64_t m, int64_t n, int64_t k)
{
    if (groups <= 0 || groups > MAX_GROUPS || rows < 0 || rows >= LIMIT - TILE || m < 0 || m >= LIMIT - TILE || n <= 0 ||
        n >= LIMIT / 2 - TILE || n % 8 != 0 || k < 0 || k >= LIMIT / 2 - TILE)
        return PMN_ERR_INVALID_ARG;
    const int64_t tiles = (m ? groups * (m / TILE + 1) : rows / TILE + groups) * (n / (TILE / 2) + 1);
    return tiles >= LIMIT / 2 ? PMN_ERR_UNSUPPORTED : PMN_OK;
}

// Chunks of eight rows that a CTA of the kernel for a few rows takes, 0 where the tiles serve a call.  f 1536, k 4096,
// gated, us for one chunk, two, and the tiles: one expert, 8 rows 8.0, 10.0, 21; 16 rows 9.1, 10.4, 21; 32 rows 15.3, 11.3,
// 21; 48 rows 21, 20, 21; 64 rows 25, 20, 21.  Eight experts, 32 rows 35, 41, 44; 24 experts, 32 rows 70, 82, 71.
// Smaller weights, f 768, k 2048: one expert, 8 rows 4.7, 5.6, 14; 32 rows 6.2, 6.2, 13; 48 rows 7.8, 7.4, 13; eight experts,
// 32 rows 11.5, 13.0, 14.6, 64 rows 13.2, 12.9, 14.2; 24 experts, 32 rows 21, 24, 26, 64 rows 23, 26, 26: there 64
// rows would still gain.
int few(int64_t rows, int64_t groups) { return rows > 32 ? 0 : rows > 16 && rows > 8 * groups ? 2 : 1; }

// Maps of the token rows [rows, k].
bool token_maps(Maps &maps, const void *a, int64_t rows, int64_t k, int64_t lda)
{
    return rows_map(&maps.x, a, k, rows, lda, 128) && rows_map(&maps.x64, a, k, rows, lda, 64) &&
           rows_map(&maps.x32, a, k, rows, lda, 32) && rows_map(&maps.x16, a, k, rows, lda, 16);
}

// Weights [groups, rows, cols], 64 columns of box_rows rows at a time.
bool weight_map(CUtensorMap *m, const void *b, int groups, int64_t rows, int64_t cols, int box_rows)
{
    const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)groups};
    const uint64_t st[2] = {(uint64_t)cols * 2, (uint64_t)rows * cols * 2};
    const uint32_t box[3] = {64, (uint32_t)box_rows, 1};
    return make_map(m, b, 3, dims, st, box);
}

}  // namespace

pmn_status pmn_bf16_error_word(int **word)
{
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_bf16_error) == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

extern "C" pmn_status pmn_grouped_gemm_bf16(const void *a, int64_t lda, const void *b, int64_t ldb, const int32_t *offsets,
                                            int num_groups, int group_mode, int b_transposed, int64_t m, int64_t n,
                                            int64_t k, int out_kind, void *out, void *stream)
{
    if ((group_mode != PMN_GROUP_M && group_mode != PMN_GROUP_K) || (b_transposed != 0 && b_transposed != 1) ||
        (out_kind != PMN_OUT_BF16 && out_kind != PMN_OUT_F32))
        return PMN_ERR_INVALID_ARG;
    const bool sums = group_mode == PMN_GROUP_K;
    const pmn_status st = check_sizes(num_groups, sums ? k : m, sums ? m : 0, n, sums ? 0 : k);
    if (st != PMN_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(out, 16) || !aligned(offsets, 4) || lda % 8 != 0) return PMN_ERR_INVALID_ARG;
    Maps maps = {};
    if (sums) {
        if (b_transposed || m <= 0 || m % 8 != 0 || lda < m || ldb < n || ldb % 8 != 0) return PMN_ERR_INVALID_ARG;
        if (!out || !offsets) return PMN_ERR_INVALID_ARG;
        if (k == 0)  // sums over no rows
            return cudaMemsetAsync(out, 0, (size_t)num_groups * m * n * (out_kind == PMN_OUT_F32 ? 4 : 2), s) == cudaSuccess
                       ? PMN_OK : PMN_ERR_CUDA;
        if (!a || !b || among(out, {a, b, offsets})) return PMN_ERR_INVALID_ARG;
        if (!rows_map(&maps.w, b, n, k, ldb, 64) || !rows_map(&maps.x, a, m, k, lda, 64) ||
            !piece_map(&maps.out, out, num_groups, m, n, out_kind, 1, 16, 128))
            return PMN_ERR_CUDA;
        const Args args{offsets, num_groups, k, m, n, 0, out, nullptr, pmn_wait_limit_ns()};
        return out_kind == PMN_OUT_F32 ? launch<SUMS, float>(maps, args, s) : launch<SUMS, uint16_t>(maps, args, s);
    }
    if (k <= 0 || k % 8 != 0 || lda < k) return PMN_ERR_INVALID_ARG;
    if (m == 0) return PMN_OK;
    if (!a || !b || !out || !offsets || among(out, {a, b, offsets})) return PMN_ERR_INVALID_ARG;
    const Args args{offsets, num_groups, m, 0, n, k, out, nullptr, pmn_wait_limit_ns()};
    if (const int chunks = b_transposed ? 0 : few(m, num_groups))
        return out_kind == PMN_OUT_F32 ? launch_few<false, float>(chunks, a, lda, b, args, s)
                                       : launch_few<false, uint16_t>(chunks, a, lda, b, args, s);
    if (!token_maps(maps, a, m, k, lda) || !(b_transposed ? weight_map(&maps.w, b, num_groups, k, n, 64)
                                                          : weight_map(&maps.w, b, num_groups, n, k, 128)) ||
        !piece_map(&maps.out, out, 1, m, n, out_kind, 0, 16, 128))
        return PMN_ERR_CUDA;
    if (b_transposed)
        return out_kind == PMN_OUT_F32 ? launch<ROWS_KN, float>(maps, args, s) : launch<ROWS_KN, uint16_t>(maps, args, s);
    return out_kind == PMN_OUT_F32 ? launch<ROWS_NK, float>(maps, args, s) : launch<ROWS_NK, uint16_t>(maps, args, s);
}

extern "C" pmn_status pmn_w1_gemm_swiglu_bf16(const void *a, int64_t lda, const void *b, const int32_t *offsets,
                                              int num_experts, int64_t total_rows, int64_t f, int64_t k, void *out,
                                              void *y_out, void *stream)
{
    const pmn_status st = check_sizes(num_experts, total_rows, 0, f, k);
    if (st != PMN_OK) return st;
    if (f % 16 != 0 || k <= 0 || k % 8 != 0 || lda < k || lda % 8 != 0) return PMN_ERR_INVALID_ARG;
    if (total_rows == 0) return PMN_OK;
    if (!a || !b || !offsets || !out || !aligned(a, 16) || !aligned(b, 16) || !aligned(offsets, 4) || !aligned(out, 16) ||
        !aligned(y_out, 16) || among(out, {a, b, offsets, y_out}) || among(y_out, {a, b, offsets}))
        return PMN_ERR_INVALID_ARG;
    const Args args{offsets, num_experts, total_rows, 0, f, k, out, static_cast<uint16_t *>(y_out),
                    pmn_wait_limit_ns()};
    if (const int chunks = few(total_rows, num_experts))
        return launch_few<true, uint16_t>(chunks, a, lda, b, args, reinterpret_cast<cudaStream_t>(stream));
    // 16 gate rows, the 16 up rows of the same columns, the next 16 gate rows, ..
    const uint64_t dims[5] = {(uint64_t)k, 16, 2, (uint64_t)f / 16, (uint64_t)num_experts};
    const uint64_t str[4] = {(uint64_t)k * 2, (uint64_t)f * k * 2, (uint64_t)k * 32, (uint64_t)f * k * 4};
    const uint32_t box[5] = {64, 16, 2, 4, 1};
    Maps maps = {};
    if (!token_maps(maps, a, total_rows, k, lda) || !make_map(&maps.w, b, 5, dims, str, box) ||
        !piece_map(&maps.out, out, 1, total_rows, f, PMN_OUT_BF16, 0, 16, 64) ||
        (y_out && !piece_map(&maps.y, y_out, total_rows, 2, f, PMN_OUT_BF16, 16, 2, 64)))
        return PMN_ERR_CUDA;
    return launch<GATED, uint16_t>(maps, args, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" pmn_status pmn_dh_gemm_swiglu_backward_bf16(const void *a, int64_t lda, const void *b, const void *y,
                                                       const int32_t *offsets, int num_experts, int64_t total_rows,
                                                       int64_t f, int64_t k, void *out, void *stream)
{
    const pmn_status st = check_sizes(num_experts, total_rows, 0, f, k);
    if (st != PMN_OK) return st;
    if (k <= 0 || k % 8 != 0 || lda < k || lda % 8 != 0) return PMN_ERR_INVALID_ARG;
    if (total_rows == 0) return PMN_OK;
    if (!a || !b || !y || !offsets || !out || !aligned(a, 16) || !aligned(b, 16) || !aligned(y, 16) || !aligned(offsets, 4) ||
        !aligned(out, 16) || among(out, {a, b, y, offsets}))
        return PMN_ERR_INVALID_ARG;
    Maps maps = {};
    if (!token_maps(maps, a, total_rows, k, lda) || !weight_map(&maps.w, b, num_experts, k, f, 64) ||
        !piece_map(&maps.out, out, total_rows, 2, f, PMN_OUT_BF16, 8, 2, 128) ||
        !piece_map(&maps.y, y, total_rows, 2, f, PMN_OUT_BF16, 8, 2, 128))
        return PMN_ERR_CUDA;
    const Args args{offsets, num_experts, total_rows, 0, f, k, out, static_cast<uint16_t *>(const_cast<void *>(y)),
                    pmn_wait_limit_ns()};
    return launch<GATED_BACKWARD, uint16_t>(maps, args, reinterpret_cast<cudaStream_t>(stream));
}
