// matvec.cu -- the few rows of a decode batch times NVFP4 weights, activations in bf16:
//   pmn_matvec_nvfp4   y = W_e x for the rows of each expert, SwiGLU where wanted
// The weights go to the tensor cores as they are stored (tcgen05 kind::mxf4nvf4, their own
// scales), so no instruction is spent on decoding them: on the CUDA cores that alone took
// four times as long as reading them.  What has to be in 4 bits for that is x,
// and it is brought there without loss: a value is a sum of eight E2M1 digits,
//   x = 2^e * scale_block * sum_c 8^-c d_c,   d_c in {0, +-1/2, +-1, +-3/2, +-2}
// (balanced octal digits, halved), each digit a row of the small operand of its own, under a
// scale per 16 values (a power of two, E4M3) and an exponent per row.  A value is exact
// down to 2^-15 of the largest of its 16, and below that within 2^-23 of it; the digits'
// sums are joined in float32.
// Two kernels: the digits of x, then the product, whose 256-deep steps the CTAs share evenly.
// Bound by HBM for a batch (512 rows, 240 experts hit, k 1536, n 4096: 849 MB in 142 us, 6.0 TB/s); for one
// token by latency (57 MB in 18 us: the digits' kernel, 5.6 us until the first scales have arrived,
// 0.3 us a step from L2, 2 us to join the tiles that CTAs share).
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

__device__ int g_matvec_error = 0;

constexpr int MAX_GROUPS = 1024, MAX_DEVICES = 64, MAX_GRID = 256;
constexpr int DIGITS = 8;
constexpr int MAX_CHUNK = 16;                    // most rows of x per pass over the weights
constexpr int BM = 128;                          // weight rows of a tile (gated: 64 gate and the 64 up rows of the same columns)
constexpr int KSTEP = 256;                       // of K per stage: 128 bytes of codes, 16 scales
constexpr int A_BYTES = BM * 128;
// The tensor core truncates each of its additions to float32, an error that grows with their number where terms have one
// sign (one accumulator for K = 262144: 8.8e-5 of such a sum).  RUN stages, 4096 of K, make a sum, and a tile's sums are
// added rounded (512 rows of 384 experts, k 1536: 148.2 -> 148.8 us; runs of 2048: 149.6 to 151.7).  Where signs are
// mixed few bits are lost either way: 3.7e-8 of the norm at k 4096, 5.5e-8 at 16384.
constexpr int RUN = 16;
constexpr int RAW_STEPS = 4, RAW_W = 16 * RAW_STEPS;  // scale rows come 64 bytes (four stages) at a time
constexpr int RAW_A = BM * RAW_W, RAW_BYTES = RAW_A + MAX_CHUNK * RAW_W, RAW_SLOTS = 3;
constexpr uint32_t TMEM_COLS = 512, SF_COLS = 32;

// CHUNK rows of x at a time: the fewer, the more of the weights fits in flight.
template <int CHUNK>
struct Cfg {
    static constexpr int NB = CHUNK * DIGITS;  // rows of the small operand
    static constexpr int B_BYTES = NB * 128, STAGE_BYTES = A_BYTES + B_BYTES;
    // More in flight is not better (512 rows of 384 experts, k 1536 and 4096: 7 stages 191 and 272 us, 6 172 and
    // 274, 5 164 and 278, 4 156 and 285; one token 20.5, 21.5, 20.5, 22.5).
    static constexpr int STAGES = 5;
    static constexpr int RAW_OFF = STAGES * STAGE_BYTES, XCH_OFF = RAW_OFF + RAW_SLOTS * RAW_BYTES;
    static constexpr int BAR_OFF = XCH_OFF + 64 * 20 * 4, CUM_OFF = BAR_OFF + 256;
    static constexpr int SMEM_BYTES = CUM_OFF + (MAX_GROUPS + 1) * 4;
    static constexpr uint32_t SF_COL0 = 2 * NB;
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
    static_assert(SF_COL0 + STAGES * SF_COLS <= TMEM_COLS, "TMEM budget");
    static_assert(8 * (2 * STAGES + 2 * RAW_SLOTS + 5) + 24 <= 256, "barrier space");
};
// warps: 0 weights, 1 MMA, 2 scale rows, 3 digits; 4 .. 7 scale factors; 8 .. 11 epilogue
constexpr int THREADS = 384;
constexpr uint64_t DRAIN_NS = 100000000ull;

struct Args {
    const uint16_t *x;
    int64_t ldx, tokens;
    const uint8_t *codes, *scales;
    const float *outer;
    const int32_t *offsets;
    int experts;
    int64_t rows, n, k;  // n: weight rows of an expert (gated: 2 f)
    const int32_t *row_choice;
    int choices;
    void *out;
    int tiles, nks;      // tiles per expert, stages per tile
    // workspace: digits [rows * 8, k / 2], their scales [rows, k / 16], per row the exponent and
    // whether it holds a value that is not finite, the sums of tiles that CTAs share, and of
    // each such tile's first CTA how many have left theirs
    uint8_t *digits, *digit_scales;
    int2 *meta;
    float *part;
    unsigned *count;
    uint64_t wait_ns;
};

__device__ __forceinline__ void latch_error(int bit) { atomicOr(&g_matvec_error, bit); }

__device__ __forceinline__ float pow2(int e)  // e in [-126, 127]
{
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

__device__ __forceinline__ int64_t token_of(const Args &p, int64_t row)
{
    if (!p.row_choice) return row;
    const int c = __ldg(p.row_choice + row);
    const int64_t t = c < 0 ? -1 : c / p.choices;
    if (t < p.tokens) return t;
    latch_error(PMN_DEVERR_BAD_OFFSETS);
    return -1;
}

// ---------------------------------------------------------------- digits
// One CTA per routed row, eight values per thread at a time: first the row's largest finite
// magnitude (up to 4096 of K stay in registers), then the digits.
constexpr int DIGIT_THREADS = 512;
__global__ void __launch_bounds__(DIGIT_THREADS) digits_kernel(const Args p, int grid)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float s_top[DIGIT_THREADS / 32];
    const int64_t row = blockIdx.x, token = token_of(p, row);
    const uint4 *x = reinterpret_cast<const uint4 *>(p.x + token * p.ldx);
    const int vecs = (int)(p.k / 8);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint4 mine = token >= 0 && (int)threadIdx.x < vecs ? __ldg(x + threadIdx.x) : zero;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < grid; i += DIGIT_THREADS) p.count[i] = 0u;
    float top = 0.0f;
    bool odd = false;
    for (int v = threadIdx.x; v < vecs && token >= 0; v += DIGIT_THREADS) {
        const uint4 q = v < DIGIT_THREADS ? mine : __ldg(x + v);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float a = __uint_as_float((u4_word(q, w) & 0x7FFFu) << 16), b = __uint_as_float(u4_word(q, w) & 0x7FFF0000u);
            odd = odd || !(a < INFINITY) || !(b < INFINITY);
            top = fmaxf(top, fmaxf(a < INFINITY ? a : 0.0f, b < INFINITY ? b : 0.0f));
        }
    }
    const uint32_t warp_top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = __uint_as_float(warp_top);
    odd = __syncthreads_or(odd) != 0;
    top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(s_top[threadIdx.x & (DIGIT_THREADS / 32 - 1)])));
    // top in [2^e, 2^(e+1)); below float32's normal range any larger e will do
    const int e = max((int)(__float_as_uint(top) >> 23) - 127, -126);
    if (threadIdx.x == 0) p.meta[row] = make_int2(e - 8, odd);
    const float down = e == 127 ? __uint_as_float(0x00400000u) : pow2(-e);  // 2^-127 is below the normal range
    for (int v = threadIdx.x; v < vecs; v += DIGIT_THREADS) {  // whole warps: k is a multiple of 256
        const uint4 q = v < DIGIT_THREADS ? mine : token >= 0 ? __ldg(x + v) : zero;
        float f[8], big = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w = u4_word(q, i >> 1);
            float y = __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
            y = fabsf(y) < INFINITY ? y : 0.0f;
            f[i] = __fmul_rn(y, down);
            big = fmaxf(big, fabsf(f[i]));
        }
        big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));  // of the 16
        // the scale 2^s: s = 8 + the exponent of the largest, within E4M3's powers of two
        const int s = max(-9, min(8, (int)(__float_as_uint(big) >> 23) - 119));
        if ((v & 1) == 0) p.digit_scales[row * (p.k / 16) + (v >> 1)] = (uint8_t)(s >= -6 ? (s + 7) << 3 : 1 << (s + 9));
        // 2^22 * 2^8 / 2^s: the value in units of the last digit
        const float up = pow2(30 - s);
        uint32_t d[DIGITS] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // octal digits of the value plus 4 in every place, less 4 each: -4 .. 3, the first -4 .. 4
            const uint32_t u = (uint32_t)(__float2int_rn(__fmul_rn(f[i], up)) + 9586980);
#pragma unroll
            for (int c = 0; c < DIGITS; ++c) {
                const uint32_t o = c == 0 ? u >> 21 : (u >> (3 * (7 - c))) & 7u;
                // E2M1 code of (o - 4) / 2: the magnitude |o - 4| itself, sign in bit 3
                const uint32_t code = c == 0 && o == 8 ? 4u : (0x32109ABCu >> (4 * o)) & 15u;
                d[c] |= code << (4 * i);
            }
        }
#pragma unroll
        for (int c = 0; c < DIGITS; ++c)
            *reinterpret_cast<uint32_t *>(p.digits + (row * DIGITS + c) * (p.k / 2) + 4 * v) = d[c];
    }
}

// ---------------------------------------------------------------- product
// Steps (256 of K of a tile of a chunk of rows) in one line, an even share of it for each
// CTA: a piece is what a CTA has of one tile.
struct Piece {
    int e, line, tile, k0, k1;  // expert, tile of all chunks, tile, stages of K
    int r0, m;                  // first routed row of the chunk, rows of it
};

template <int CHUNK>
struct Walk {
    uint32_t at, end;
    int e;
    __device__ __forceinline__ bool next(const Args &p, const int *s_cum, Piece &q)
    {
        if (at >= end) return false;
        q.line = (int)(at / (uint32_t)p.nks);
        q.k0 = (int)(at - (uint32_t)q.line * p.nks);
        q.k1 = (int)min((uint32_t)p.nks, q.k0 + (end - at));
        at += q.k1 - q.k0;
        const int unit = q.line / p.tiles;
        q.tile = q.line - unit * p.tiles;
        while (e + 1 < p.experts && s_cum[e + 1] <= unit) ++e;
        q.e = e;
        q.r0 = __ldg(p.offsets + e) + (unit - s_cum[e]) * CHUNK;
        q.m = min(CHUNK, __ldg(p.offsets + e + 1) - q.r0);
        return true;
    }
};

__device__ __forceinline__ int digit_rows(const Piece &q) { return (q.m + 1) / 2 * 2 * DIGITS; }  // a multiple of 16

__device__ __forceinline__ void mma_nvfp4_by(uint32_t el, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate), "r"(el)
        : "memory");
}

__device__ __forceinline__ void store_one(uint16_t *p, float v)
{
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    *p = *reinterpret_cast<const uint16_t *>(&b);
}
__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }

// The row's product by plain float32 sums: for rows with values that no digit stands for.
__device__ __noinline__ float plain_dot(const Args &p, int64_t wrow, int64_t token)
{
    const uint8_t *c = p.codes + wrow * (p.k / 2), *s = p.scales + wrow * (p.k / 16);
    const uint16_t *x = p.x + token * p.ldx;
    float acc = 0.0f;
    for (int64_t i = 0; i < p.k; ++i) {
        const uint32_t b = __ldg(s + (i >> 4)), code = __ldg(c + (i >> 1)) >> (4 * (i & 1));
        const float w = __fmul_rn(e2m1_to_f32(code & 15u), (b & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : e4m3_to_f32(b));
        acc = fmaf(w, __uint_as_float((uint32_t)__ldg(x + i) << 16), acc);
    }
    return acc;
}

template <int CHUNK, bool GATED, typename OUT>
__global__ void __launch_bounds__(THREADS, 1)
    matvec_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS,
                  const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmDS, const Args p)
{
    using C = Cfg<CHUNK>;
    constexpr int STAGES = C::STAGES, STAGE_BYTES = C::STAGE_BYTES, NB = C::NB, RAW_OFF = C::RAW_OFF;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw;
    asm volatile("" : "+l"(smem));
    const uint32_t stages = smem_u32(smem);
    const uint32_t bar_full = stages + C::BAR_OFF, bar_empty = bar_full + 8 * STAGES;
    const uint32_t bar_raw = bar_empty + 8 * STAGES, bar_raw_empty = bar_raw + 8 * RAW_SLOTS;
    const uint32_t bar_acc_full = bar_raw_empty + 8 * RAW_SLOTS, bar_acc_empty = bar_acc_full + 16, bar_drain = bar_acc_empty + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::BAR_OFF + 8 * (2 * STAGES + 2 * RAW_SLOTS + 5));
    int *s_abort = reinterpret_cast<int *>(tmem_slot + 1), *s_units = s_abort + 1, *s_last = s_abort + 2;
    int *s_cum = reinterpret_cast<int *>(smem + C::CUM_OFF);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 6);  // weights, digits, four scale-factor warps
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int s = 0; s < RAW_SLOTS; ++s) {
            mbar_init(bar_raw + 8 * s, 1);
            mbar_init(bar_raw_empty + 8 * s, 4);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_acc_full + 8 * b, 1);
            mbar_init(bar_acc_empty + 8 * b, 4);
        }
        mbar_init(bar_drain, 1);
        *s_abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmS);
        tma_prefetch_desc(&tmD);
        tma_prefetch_desc(&tmDS);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc_ct<1>(smem_u32(tmem_slot), TMEM_COLS);
    }
    // chunks of each expert, then their running sum
    bool bad = false;
    for (int e = threadIdx.x; e < p.experts; e += THREADS) {
        const int lo = __ldg(p.offsets + e), hi = __ldg(p.offsets + e + 1);
        if (lo < 0 || hi < lo || hi > p.rows) bad = true;
        s_cum[e] = (hi - lo + CHUNK - 1) / CHUNK;
    }
    bad = __syncthreads_or(bad) != 0;
    if (warp == 0) {
        int sum = 0;
        for (int g0 = 0; g0 < p.experts; g0 += 32) {
            const int n = g0 + lane < p.experts ? s_cum[g0 + lane] : 0;
            int run = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, run, o);
                if (lane >= o) run += v;
            }
            if (g0 + lane < p.experts) s_cum[g0 + lane] = sum + run - n;
            sum += __shfl_sync(0xFFFFFFFFu, run, 31);
        }
        if (lane == 0) {
            s_cum[p.experts] = sum;
            *s_units = bad ? 0 : sum;
            if (bad && blockIdx.x == 0) latch_error(PMN_DEVERR_BAD_OFFSETS);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // (fewer than 2^31 steps: the host's checks)
    const uint32_t total = (uint32_t)*s_units * p.tiles * p.nks, ctas = max(1u, min(gridDim.x, total));  // with a share
    const uint32_t each = total / ctas, more = total - each * ctas;
    auto share = [&](uint32_t b) { return each * b + min(b, more); };  // first step of CTA b
    Walk<CHUNK> walk{0, 0, 0};
    if (blockIdx.x < ctas) walk = Walk<CHUNK>{share(blockIdx.x), share(blockIdx.x + 1), 0};
    const int half = GATED ? BM / 2 : BM;
    bool dead = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {  // false: a wait ran out, here or in another warp
        dead = dead || __any_sync(0xFFFFFFFFu, *(volatile int *)s_abort != 0);
        if (!dead && !warp_wait(bar, parity, p.wait_ns)) {
            dead = true;
            if (lane == 0) {
                *(volatile int *)s_abort = 1;
                latch_error(PMN_DEVERR_WAIT_TIMEOUT);
            }
        }
        return !dead;
    };
    uint32_t stage = 0, phase = 0;
    auto next_stage = [&]() {
        if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
        }
    };
    Piece q;

    if (warp == 0) {
        // ---------------------------------------------------- weights, 64 rows a box
        while (!dead && walk.next(p, s_cum, q)) {
            const int64_t row = (int64_t)q.e * p.n + q.tile * half;
            const int32_t ra = (int32_t)row, rb = (int32_t)(row + (GATED ? p.n / 2 : 64));
            for (int k = q.k0; k < q.k1; ++k) {
                if (!wait(bar_empty + 8 * stage, phase ^ 1)) break;
                if (elect_one()) {
                    const uint32_t st = stages + stage * STAGE_BYTES, fb = bar_full + 8 * stage;
                    mbar_arrive_expect_tx(fb, A_BYTES);
                    tma_load_2d(st, &tmW, fb, 128 * k, ra);
                    tma_load_2d(st + A_BYTES / 2, &tmW, fb, 128 * k, rb);
                }
                __syncwarp();
                next_stage();
            }
        }
    } else if (warp == 3) {
        // ---------------------------------------------------- digits, 16 rows a box
        asm volatile("griddepcontrol.wait;" ::: "memory");
        while (!dead && walk.next(p, s_cum, q)) {
            const int nb = digit_rows(q);
            for (int k = q.k0; k < q.k1; ++k) {
                if (!wait(bar_empty + 8 * stage, phase ^ 1)) break;
                if (elect_one()) {
                    const uint32_t st = stages + stage * STAGE_BYTES + A_BYTES, fb = bar_full + 8 * stage;
                    mbar_arrive_expect_tx(fb, nb * 128);
                    for (int r = 0; r < nb; r += 16) tma_load_2d(st + 128 * r, &tmD, fb, 128 * k, q.r0 * DIGITS + r);
                }
                __syncwarp();
                next_stage();
            }
        }
    } else if (warp == 2) {
        // ---------------------------------------------------- scale rows, four stages at a time
        uint32_t slot = 0, sphase = 0;
        bool waited = false;
        int pending = 0;  // slots whose digits' scales are still to be asked for
        int32_t px[RAW_SLOTS], pr[RAW_SLOTS];
        auto ask_digits = [&](int s, int32_t x, int32_t r) {
            if (elect_one()) tma_load_2d(stages + RAW_OFF + s * RAW_BYTES + RAW_A, &tmDS, bar_raw + 8 * s, x, r);
            __syncwarp();
        };
        auto flush = [&]() {  // the digits have been written
            asm volatile("griddepcontrol.wait;" ::: "memory");
            waited = true;
#pragma unroll
            for (int s = 0; s < RAW_SLOTS; ++s)
                if (s < pending) ask_digits(s, px[s], pr[s]);
        };
        while (!dead && walk.next(p, s_cum, q)) {
            const int64_t row = (int64_t)q.e * p.n + q.tile * half;
            const int32_t ra = (int32_t)row, rb = (int32_t)(row + (GATED ? p.n / 2 : 64));
            for (int k = q.k0; k < q.k1; k += RAW_STEPS) {
                if (!waited && pending == RAW_SLOTS) flush();
                if (!wait(bar_raw_empty + 8 * slot, sphase ^ 1)) break;
                if (elect_one()) {
                    const uint32_t st = stages + RAW_OFF + slot * RAW_BYTES, fb = bar_raw + 8 * slot;
                    mbar_arrive_expect_tx(fb, RAW_A + CHUNK * RAW_W);
                    tma_load_2d(st, &tmS, fb, 16 * k, ra);
                    tma_load_2d(st + RAW_A / 2, &tmS, fb, 16 * k, rb);
                }
                __syncwarp();
                if (waited) ask_digits(slot, 16 * k, q.r0);
                else {
#pragma unroll
                    for (int s = 0; s < RAW_SLOTS; ++s)
                        if (s == pending) px[s] = 16 * k, pr[s] = q.r0;
                    ++pending;
                }
                if (++slot == RAW_SLOTS) {
                    slot = 0;
                    sphase ^= 1;
                }
            }
        }
        if (!waited) flush();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0), el = elect_one();
        uint32_t abuf = 0, aphase = 0;
        while (!dead && walk.next(p, s_cum, q)) {
            const uint32_t idesc = (1u << 7) | (1u << 10) | ((uint32_t)(digit_rows(q) >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
            for (int run = q.k0; run < q.k1 && !dead; run += RUN) {
                if (!wait(bar_acc_empty + 8 * abuf, aphase ^ 1)) break;
                const uint32_t d = tm + abuf * NB;
                const int end = min(q.k1, run + RUN);
                for (int k = run; k < end; ++k) {
                    if (!wait(bar_full + 8 * stage, phase)) break;
                    tc_fence_after();
                    const uint32_t a = stages + stage * STAGE_BYTES, b = a + A_BYTES;
                    const uint32_t sfa = tm + C::SF_COL0 + stage * SF_COLS, sfb = sfa + 16;
#pragma unroll
                    for (int s = 0; s < 4; ++s)  // 64 of K: 32 bytes of the swizzled rows
                        mma_nvfp4_by(el, d, smem_desc(a + 32 * s, 16, 1024, 2), smem_desc(b + 32 * s, 16, 1024, 2), idesc, sfa + 4 * s,
                                     sfb + 4 * s, k > run || s > 0);
                    tc_commit_ct<1>(el, bar_empty + 8 * stage);
                    next_stage();
                }
                if (dead) break;
                tc_commit_ct<1>(el, bar_acc_full + 8 * abuf);
                if (++abuf == 2) {
                    abuf = 0;
                    aphase ^= 1;
                }
            }
        }
        if (elect_one()) tc_commit(bar_drain);  // every tcgen05 operation of this warp has completed
        __syncwarp();
        (void)warp_wait(bar_drain, 0, DRAIN_NS);
    } else if (warp < 8) {
        // ---------------------------------------------------- scale factors
        // For 64 of K (s) the tensor core finds the four scale bytes of row 32 j + r in column
        // 4 s + j of lane r, in each of TMEM's four groups of 32 lanes: one group per warp, which
        // writes all rows' there.  The eight digits of a value share a scale.  (By way of shared memory,
        // eight tcgen05.cp a stage, one token takes 22.5 us for 20.5;
        // a wait for every stage's store: 512 rows of 384 experts, k 1536, 164 to 182 us for 148.)
        const int quad = warp & 3;
        uint32_t slot = 0, sphase = 0;
        while (!dead && walk.next(p, s_cum, q)) {
            for (int k = q.k0; k < q.k1 && !dead; k += RAW_STEPS) {
                if (!wait(bar_raw + 8 * slot, sphase)) break;
                const uint8_t *raw = smem + RAW_OFF + slot * RAW_BYTES;
                // two stages at a time: the store's completion is waited for once
#pragma unroll
                for (int c = 0; c < RAW_STEPS; c += 2) {
                    if (k + c >= q.k1 || dead) break;
                    const bool two = k + c + 1 < q.k1;
                    uint32_t sa[2][16], sb[2][16];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int row = 32 * j + lane, piece = c + h;
                            // (64-byte swizzle: eight lanes meet all banks)
                            const uint4 va = *reinterpret_cast<const uint4 *>(raw + RAW_W * row + 16 * (piece ^ ((row >> 1) & 3)));
                            const uint4 vb = 32 * j < NB ? *reinterpret_cast<const uint4 *>(raw + RAW_A + RAW_W * (row >> 3) + 16 * piece)
                                                         : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                            for (int s = 0; s < 4; ++s) {
                                sa[h][4 * s + j] = u4_word(va, s);
                                sb[h][4 * s + j] = u4_word(vb, s);
                            }
                        }
                    const uint32_t to = tmem + ((uint32_t)(32 * quad) << 16) + C::SF_COL0, first = stage;
                    if (!wait(bar_empty + 8 * stage, phase ^ 1)) break;
                    tc_fence_after();
                    tmem_st_32x32b_x16(to + stage * SF_COLS, sa[0]);
                    tmem_st_32x32b_x16(to + stage * SF_COLS + 16, sb[0]);
                    next_stage();
                    if (two) {
                        if (!wait(bar_empty + 8 * stage, phase ^ 1)) break;
                        tc_fence_after();
                        tmem_st_32x32b_x16(to + stage * SF_COLS, sa[1]);
                        tmem_st_32x32b_x16(to + stage * SF_COLS + 16, sb[1]);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        // The slot's rows may be overwritten once they are in registers, which only the stores that
                        // have used them show: an arrival does not wait for loads before it.
                        if (c == RAW_STEPS - 2 || k + c + 2 >= q.k1) mbar_arrive(bar_raw_empty + 8 * slot);
                        mbar_arrive(bar_full + 8 * first);
                        if (two) mbar_arrive(bar_full + 8 * stage);
                    }
                    if (two) next_stage();
                }
                if (++slot == RAW_SLOTS) {
                    slot = 0;
                    sphase ^= 1;
                }
            }
        }
    } else {
        // ---------------------------------------------------- epilogue: a weight row per thread
        const int quad = warp & 3, i = threadIdx.x - 256;
        uint32_t abuf = 0, aphase = 0;
        asm volatile("griddepcontrol.wait;" ::: "memory");
        while (walk.next(p, s_cum, q)) {  // to the end, also after a timeout: the four warps meet at barriers
            const int m = q.m;
            float y[CHUNK];
            const float outer = __ldg(p.outer + q.e);
            int exponent[CHUNK], odd = 0;  // bit t: row t holds a value that is not finite
#pragma unroll
            for (int t = 0; t < CHUNK; ++t) {
                const int2 meta = t < m ? __ldcg(p.meta + q.r0 + t) : make_int2(0, 0);
                exponent[t] = meta.x;
                odd |= meta.y << t;
            }
            auto take = [&](bool more) {  // the next accumulator's sums, added to those before it
                if (wait(bar_acc_full + 8 * abuf, aphase)) {
                    tc_fence_after();
                    const uint32_t acc = tmem + ((uint32_t)(32 * quad) << 16) + abuf * NB;
#pragma unroll
                    for (int t = 0; t < CHUNK; t += 2) {
                        if (t >= m) break;
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(acc + DIGITS * t, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float sum = __uint_as_float(v[8 * u + 7]);
#pragma unroll
                            for (int c = 6; c >= 0; --c) sum = fmaf(sum, 0.125f, __uint_as_float(v[8 * u + c]));
                            y[t + u] = more ? __fadd_rn(y[t + u], sum) : sum;
                        }
                    }
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_acc_empty + 8 * abuf);
                if (++abuf == 2) {
                    abuf = 0;
                    aphase ^= 1;
                }
            };
            take(false);
            for (int k = q.k0 + RUN; k < q.k1; k += RUN) take(true);
            if (q.k1 - q.k0 < p.nks) {
                // A tile that CTAs first .. last share: each leaves its sums, and the one that
                // comes last adds them up in the order of K.  A CTA's slot 0 is for a tile that began
                // before its share, slot 1 for one that begins in it.
                const uint32_t s0 = (uint32_t)q.line * p.nks, s1 = s0 + p.nks;
                int first = blockIdx.x, last = blockIdx.x;
                while (share(first) > s0) --first;
                while (share(last + 1) < s1) ++last;
                float *mine = p.part + ((int64_t)blockIdx.x * 2 + (q.k0 == 0)) * MAX_CHUNK * BM;
#pragma unroll
                for (int t = 0; t < CHUNK; ++t)
                    if (t < m) __stcg(mine + t * BM + i, y[t]);
                __threadfence();
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (i == 0) *s_last = atomicAdd(p.count + first, 1u) == (unsigned)(last - first);
                asm volatile("bar.sync 1, 128;" ::: "memory");
                const bool finish = *(volatile int *)s_last;
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (!finish) continue;
                __threadfence();
#pragma unroll
                for (int t = 0; t < CHUNK; ++t) y[t] = 0.0f;
                for (int b = first; b <= last; ++b) {
                    const float *from = p.part + ((int64_t)b * 2 + (b == first)) * MAX_CHUNK * BM + i;
#pragma unroll
                    for (int t = 0; t < CHUNK; ++t)
                        if (t < m) y[t] = __fadd_rn(y[t], __ldcg(from + t * BM));
                }
            }
            const int half_n = (int)(GATED ? p.n / 2 : p.n), c = GATED ? i & 63 : i, col = q.tile * half + c;
            const int64_t wrow = (int64_t)q.e * p.n + col + (GATED && i >= 64 ? half_n : 0);
            const bool on = col < half_n && !dead;
#pragma unroll
            for (int t = 0; t < CHUNK; ++t) {
                if (t >= m) break;
                const int e1 = max(exponent[t], -126);
                y[t] = __fmul_rn(__fmul_rn(__fmul_rn(y[t], outer), pow2(e1)), pow2(exponent[t] - e1));
                if (((odd >> t) & 1) && on) {
                    const int64_t token = token_of(p, q.r0 + t);
                    y[t] = __fmul_rn(plain_dot(p, wrow, token), outer);
                }
            }
            OUT *o = static_cast<OUT *>(p.out) + (int64_t)q.r0 * half_n + col;
            if (!GATED) {
#pragma unroll
                for (int t = 0; t < CHUNK; ++t)
                    if (t < m && on) store_one(o + (int64_t)t * half_n, y[t]);
            } else {
                // the up rows' threads hand theirs to the gate rows'
                float *xch = reinterpret_cast<float *>(smem + C::XCH_OFF) + c * 20;
                if (i >= 64) {
#pragma unroll
                    for (int t = 0; t < CHUNK; t += 4)
                        *reinterpret_cast<float4 *>(xch + t) = make_float4(y[t], y[t + 1], y[t + 2], y[t + 3]);
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (i < 64) {
#pragma unroll
                    for (int t = 0; t < CHUNK; ++t) {
                        if (t >= m) break;
                        if (on) store_one(o + (int64_t)t * half_n, __fmul_rn(__fmul_rn(y[t], sigmoid(y[t])), xch[t]));
                    }
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*(volatile int *)s_abort) {  // copies that nobody waited for may still be landing
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 10000000ull) {
        }
    }
    __syncthreads();
    if (warp == 1) tmem_dealloc_ct<1>(tmem, TMEM_COLS);
}

// ====================================================================== host
// Bytes [rows, width] in boxes of box_w x box_rows.
bool make_map(CUtensorMap *m, const void *base, int64_t width, int64_t rows, uint32_t box_w, uint32_t box_rows,
              CUtensorMapSwizzle swizzle)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)width};
    const cuuint32_t box[2] = {box_w, box_rows}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              box_w == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int64_t up128(int64_t n) { return (n + 127) / 128 * 128; }

// The workspace's parts, each on a 128-byte boundary.
struct Parts {
    int64_t digits, scales, meta, part, count, end;
    Parts(int64_t rows, int64_t k)
    {
        digits = 0;
        scales = digits + up128(rows * DIGITS * (k / 2));
        meta = scales + up128(rows * (k / 16));
        part = meta + up128(rows * 8);
        count = part + (int64_t)MAX_GRID * 2 * MAX_CHUNK * BM * 4;
        end = count + MAX_GRID * 4;
    }
};

constexpr int64_t LIMIT = int64_t(1) << 31;

bool good_sizes(int64_t rows, int64_t k)
{
    return rows >= 0 && rows < LIMIT / DIGITS - 256 && k > 0 && k % KSTEP == 0 && k < LIMIT / 4;
}

template <int CHUNK, bool GATED, typename OUT>
pmn_status launch_chunk(const Args &args, int64_t n, cudaStream_t s)
{
    CUtensorMap maps[4];
    if (!make_map(&maps[0], args.codes, args.k / 2, n, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&maps[1], args.scales, args.k / 16, n, RAW_W, 64, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !make_map(&maps[2], args.digits, args.k / 2, args.rows * DIGITS, 128, 16, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&maps[3], args.digit_scales, args.k / 16, args.rows, RAW_W, CHUNK, CU_TENSOR_MAP_SWIZZLE_NONE))
        return PMN_ERR_CUDA;
    auto kern = matvec_kernel<CHUNK, GATED, OUT>;
    static std::atomic<int> sm_count[MAX_DEVICES];  // of each device this kernel has been set up on
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return PMN_ERR_CUDA;
    int sms = dev < MAX_DEVICES ? sm_count[dev].load(std::memory_order_acquire) : 0;
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1 ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<CHUNK>::SMEM_BYTES) != cudaSuccess)
            return PMN_ERR_CUDA;
        sms = std::min(sms, MAX_GRID);
        if (dev < MAX_DEVICES) sm_count[dev].store(sms, std::memory_order_release);
    }
    digits_kernel<<<(unsigned)args.rows, DIGIT_THREADS, 0, s>>>(args, sms);
    if (cudaGetLastError() != cudaSuccess) return PMN_ERR_CUDA;
    // launched while the digits are made: the weights need not wait for them
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sms);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Cfg<CHUNK>::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], maps[3], args) == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

template <bool GATED, typename OUT>
pmn_status launch(const Args &args, int64_t n, cudaStream_t s)
{
    if (args.rows <= 8 * (int64_t)args.experts) return launch_chunk<8, GATED, OUT>(args, n, s);
    return launch_chunk<16, GATED, OUT>(args, n, s);
}

}  // namespace

pmn_status pmn_matvec_error_word(int **word)
{
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_matvec_error) == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

extern "C" int64_t pmn_matvec_nvfp4_workspace_bytes(int64_t total_rows, int64_t k)
{
    return !good_sizes(total_rows, k) ? -1 : total_rows == 0 ? 0 : Parts(total_rows, k).end;
}

extern "C" pmn_status pmn_matvec_nvfp4(const void *x, int64_t ldx, int64_t tokens, const uint8_t *codes,
                                       const uint8_t *scales, const float *outer, const int32_t *offsets,
                                       int num_experts, int64_t total_rows, int64_t n, int64_t k,
                                       const int32_t *row_choice, int choices, int swiglu, int out_kind, void *out,
                                       void *workspace, int64_t workspace_bytes, void *stream)
{
    if (num_experts <= 0 || num_experts > MAX_GROUPS || !good_sizes(total_rows, k) || tokens < 0 || tokens >= LIMIT || n <= 0 ||
        n % 16 != 0 || n >= LIMIT / 2 || num_experts * n >= LIMIT - 256 || ldx < k || ldx % 8 != 0 || (swiglu != 0 && swiglu != 1) ||
        choices < 1 || (out_kind != PMN_OUT_BF16 && out_kind != PMN_OUT_F32) || (!row_choice && tokens != total_rows))
        return PMN_ERR_INVALID_ARG;
    if (total_rows == 0) return PMN_OK;
    const Parts w(total_rows, k);
    if ((!x && tokens > 0) || !codes || !scales || !outer || !offsets || !out || !workspace || workspace_bytes < w.end ||
        !aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(outer, 4) || !aligned(offsets, 4) ||
        !aligned(row_choice, 4) || !aligned(out, 16) || !aligned(workspace, 16))
        return PMN_ERR_INVALID_ARG;
    // steps are counted in 32 bits
    if ((total_rows / 8 + num_experts) * (n / 64 + 1) * (k / KSTEP) >= LIMIT) return PMN_ERR_UNSUPPORTED;
    if (among(out, {x, codes, scales, outer, offsets, row_choice, workspace}) ||
        among(workspace, {x, codes, scales, outer, offsets, row_choice}))
        return PMN_ERR_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const int64_t half_n = swiglu ? n / 2 : n, half = swiglu ? BM / 2 : BM;
    const Args a{static_cast<const uint16_t *>(x), ldx, tokens, codes, scales, outer, offsets, num_experts, total_rows, n, k,
                 row_choice, choices, out, (int)((half_n + half - 1) / half), (int)(k / KSTEP), ws + w.digits, ws + w.scales,
                 reinterpret_cast<int2 *>(ws + w.meta), reinterpret_cast<float *>(ws + w.part),
                 reinterpret_cast<unsigned *>(ws + w.count), pmn_wait_limit_ns()};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (swiglu) return out_kind == PMN_OUT_F32 ? launch<true, float>(a, num_experts * n, s) : launch<true, uint16_t>(a, num_experts * n, s);
    return out_kind == PMN_OUT_F32 ? launch<false, float>(a, num_experts * n, s) : launch<false, uint16_t>(a, num_experts * n, s);
}
