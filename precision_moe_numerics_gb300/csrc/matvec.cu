// matvec.cu -- the few rows of a decode batch times NVFP4 weights, activations in bf16:
//   pmn_matvec_nvfp4   y = W_e x for the rows of each expert, SwiGLU where wanted
// A weight is code * scale (E2M1 times E4M3: at most 6 significant bits, exact in f16) times
// the expert's float32 scale.  x is brought into f16's range by a power of two per 256
// of K and row, chosen from the largest magnitude there: what that loses lies 2^-40
// below the largest element.  f16 products of the tensor cores (mma.sync) add up in
// float32; a share of K per warp, joined in float32 in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "../../include/pmn.h"
#include "numerics.cuh"
#include "sm100.cuh"

using namespace pmn;
using namespace pmn::sm100;

uint64_t pmn_wait_limit_ns();  // gemm.cu: the limit of every bounded device wait

namespace {

__device__ int g_matvec_error = 0;

constexpr int MAX_GROUPS = 1024, MAX_DEVICES = 64;
constexpr int WARPS = 16, THREADS = 32 * WARPS;
constexpr int SLICE = 256;                       // of K, for one warp
constexpr int CODE_BYTES = WARPS * 16 * SLICE / 2, SCALE_BYTES = WARPS * 16 * SLICE / 16;
constexpr int STAGES = 5, STAGE_BYTES = CODE_BYTES + SCALE_BYTES;
constexpr int PITCH = 20, PART = 8 * PITCH;      // floats of a warp's 8 x 16 sums: both accesses free of conflicts
constexpr uint64_t DRAIN_NS = 100000000ull;

template <int NT>
struct Smem {
    static constexpr int PART_OFF = STAGES * STAGE_BYTES, PART_BYTES = WARPS * NT * PART * 4;
    static constexpr int BAR_OFF = PART_OFF + 2 * PART_BYTES, CUM_OFF = BAR_OFF + 8 * STAGES + 24;
    static constexpr int BYTES = CUM_OFF + (MAX_GROUPS + 1) * 4;
    static_assert(BYTES <= 232448, "shared memory budget");
};

// An item is 16 rows of the weights (gated: 8 gate and the 8 up rows of the same
// columns) times `groups`, as many as keep the warps busy when K is short; K is taken in
// `passes` of up to `slices` warps' shares.
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
    int all_slices, slices, passes, groups, items;  // items per expert
    uint64_t wait_ns;
};

__device__ __forceinline__ void latch_error(int bit) { atomicOr(&g_matvec_error, bit); }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// D (16 x 8, float32) += A (16 x 16) B (16 x 8), f16
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

struct Item {
    int e, tile;       // expert; 16 * groups weight rows
    int r0, m;         // first routed row of the chunk, rows left in the segment
};

template <int NT>
__device__ __forceinline__ Item get_item(int64_t i, const Args &p, const int *s_cum, int &gc)
{
    const int unit = (int)(i / p.items);  // a chunk of 8 NT rows of an expert
    while (gc + 1 < p.experts && s_cum[gc + 1] <= unit) ++gc;
    Item it;
    it.e = gc;
    it.tile = (int)(i - (int64_t)unit * p.items);
    it.r0 = __ldg(p.offsets + gc) + (unit - s_cum[gc]) * 8 * NT;
    it.m = __ldg(p.offsets + gc + 1) - it.r0;
    return it;
}

__device__ __forceinline__ void store_one(uint16_t *p, float v)
{
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    *p = *reinterpret_cast<const uint16_t *>(&b);
}
__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }

template <int NT, bool GATED, typename OUT>
__global__ void __launch_bounds__(THREADS, 1) matvec_kernel(const Args p)
{
    using S = Smem<NT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem), bar_full = base + S::BAR_OFF;
    int *s_abort = reinterpret_cast<int *>(smem + S::BAR_OFF + 8 * STAGES), *s_total = s_abort + 1, *s_bad = s_abort + 2;
    int *s_cum = reinterpret_cast<int *>(smem + S::CUM_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(bar_full + 8 * s, 1);
        *s_abort = 0;
        *s_bad = 0;
        fence_barrier_init();
    }
    __syncthreads();
    // chunks of 8 NT rows of each expert, then their running sum
    for (int e = threadIdx.x; e < p.experts; e += THREADS) {
        const int lo = __ldg(p.offsets + e), hi = __ldg(p.offsets + e + 1);
        if (lo < 0 || hi < lo || hi > p.rows) *s_bad = 1;
        s_cum[e] = (hi - lo + 8 * NT - 1) / (8 * NT);
    }
    __syncthreads();
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
            *s_total = *s_bad ? 0 : sum;
            if (*s_bad && blockIdx.x == 0) latch_error(PMN_DEVERR_BAD_OFFSETS);
        }
    }
    __syncthreads();
    const int64_t total = (int64_t)*s_total * p.items;
    const int64_t first = total * blockIdx.x / gridDim.x, last = total * (blockIdx.x + 1) / gridDim.x;
    const int tile_rows = 16 * p.groups, half_rows = GATED ? tile_rows / 2 : tile_rows;  // gated: gate rows, up rows
    const int64_t half_n = GATED ? p.n / 2 : p.n;

    // Weights come by bulk copies, STAGES passes ahead.  One warp asks for the next pass
    // whenever the barrier that ends one has freed its stage.
    const int64_t all_passes = (last - first) * p.passes;
    int64_t asked = 0;
    int ask_gc = 0;
    auto ask = [&]() {
        if (asked >= all_passes || __any_sync(0xFFFFFFFFu, *(volatile int *)s_abort != 0)) return;
        const int64_t ahead = asked / p.passes;
        const int pass = (int)(asked - ahead * p.passes), stage = (int)(asked % STAGES);
        const Item it = get_item<NT>(first + ahead, p, s_cum, ask_gc);
        const int row0 = it.tile * half_rows, rows = (int)min((int64_t)half_rows, half_n - row0);
        const int64_t cp = p.k / 2, sp = p.k / 16;  // row pitches
        const uint32_t st = base + stage * STAGE_BYTES, fb = bar_full + 8 * stage;
        const int s0 = pass * p.slices, ns = min(p.slices, p.all_slices - s0);
        const int halves = GATED ? 2 : 1;
        if (lane == 0) mbar_arrive_expect_tx(fb, halves * rows * ns * (SLICE / 2 + SLICE / 16));
        __syncwarp();
        for (int h = 0; h < halves; ++h) {
            const int64_t row = (int64_t)it.e * p.n + h * half_n + row0;
            const uint32_t cd = st + h * half_rows * ns * (SLICE / 2), sd = st + CODE_BYTES + h * half_rows * ns * (SLICE / 16);
            const uint8_t *c = p.codes + row * cp + s0 * (SLICE / 2), *sc = p.scales + row * sp + s0 * (SLICE / 16);
            if (p.passes == 1) {  // the rows lie end to end
                if (lane == 0) bulk_load(cd, c, rows * cp, fb);
                if (lane == 1) bulk_load(sd, sc, rows * sp, fb);
            } else {
                for (int r = lane; r < rows; r += 32) {
                    bulk_load(cd + r * ns * (SLICE / 2), c + r * cp, ns * (SLICE / 2), fb);
                    bulk_load(sd + r * ns * (SLICE / 16), sc + r * sp, ns * (SLICE / 16), fb);
                }
            }
        }
        __syncwarp();
        ++asked;
    };
    if (warp == WARPS - 1)
        for (int s = 0; s < STAGES; ++s) ask();

    // Lane 4 r + q holds, of weight rows r and r + 8 and of row r of x, 32 of every 128 of
    // the warp's slice of K: what mma.sync sees as its K is this order, the same on both sides.
    const int r = lane >> 2, q = lane & 3;
    const int group = warp / p.slices, slice = warp - group * p.slices;
    uint32_t xf[NT][32];
    float unscale[NT][2];  // of columns 2 q and 2 q + 1 of the sums
    int have_unit = -1, have_pass = -1;
    uint32_t stage = 0, phase = 0;
    int gc = 0, buf = 0;
    bool dead = false;
    for (int64_t i = first; i < last; ++i, buf ^= 1) {
        const Item it = get_item<NT>(i, p, s_cum, gc);
        const int unit = (int)(i / p.items);
        const float outer = __ldg(p.outer + it.e);
        float sum[NT][4] = {};
        for (int pass = 0; pass < p.passes; ++pass) {
            const int s0 = pass * p.slices, ns = min(p.slices, p.all_slices - s0);
            const bool active = group < p.groups && slice < ns;
            if (active && (unit != have_unit || pass != have_pass)) {
                have_unit = unit;
                have_pass = pass;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int row = 8 * t + r;
                    int64_t token = -1;
                    if (row < it.m) {
                        token = it.r0 + row;
                        if (p.row_choice) {
                            const int c = __ldg(p.row_choice + token);
                            token = c < 0 ? -1 : c / p.choices;
                            if (token >= p.tokens) {
                                latch_error(PMN_DEVERR_BAD_OFFSETS);
                                token = -1;
                            }
                        }
                    }
                    uint4 raw[8];
                    const uint16_t *xp = p.x + token * p.ldx + (s0 + slice) * SLICE + 32 * q;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        raw[j] = token >= 0 ? __ldg(reinterpret_cast<const uint4 *>(xp + 128 * (j >> 2) + 8 * (j & 3)))
                                            : make_uint4(0u, 0u, 0u, 0u);
                    float top = 0.0f;  // the largest finite magnitude
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t v = u4_word(raw[j], w);
                            const float a = __uint_as_float((v & 0x7FFFu) << 16), b = __uint_as_float(v & 0x7FFF0000u);
                            top = fmaxf(top, fmaxf(a < INFINITY ? a : 0.0f, b < INFINITY ? b : 0.0f));
                        }
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    // top * 2^e in [2^14, 2^15)
                    const int e = max(-126, min(126, 141 - (int)(__float_as_uint(top) >> 23)));
                    const float f = __uint_as_float((uint32_t)(127 + e) << 23), back = __uint_as_float((uint32_t)(127 - e) << 23);
                    unscale[t][0] = __shfl_sync(0xFFFFFFFFu, back, 8 * q);      // lane 4 (2 q)
                    unscale[t][1] = __shfl_sync(0xFFFFFFFFu, back, 8 * q + 4);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t v = u4_word(raw[j], w);
                            xf[t][4 * j + w] = f16x2(__fmul_rn(__uint_as_float(v << 16), f),
                                                     __fmul_rn(__uint_as_float(v & 0xFFFF0000u), f));
                        }
                }
            }
            dead = dead || *(volatile int *)s_abort != 0;
            if (!dead && !warp_wait(bar_full + 8 * stage, phase, p.wait_ns)) {
                dead = true;
                if (lane == 0) {
                    *(volatile int *)s_abort = 1;
                    latch_error(PMN_DEVERR_WAIT_TIMEOUT);
                }
            }
            dead = __any_sync(0xFFFFFFFFu, dead);
            if (active && !dead) {
                const int ra = GATED ? 8 * group + r : 16 * group + r, rb = GATED ? half_rows + ra : ra + 8;
                const uint32_t st = base + stage * STAGE_BYTES, code = st + slice * (SLICE / 2) + 16 * q;
                const uint32_t scale = st + CODE_BYTES + slice * (SLICE / 16);
                // even rows take the first 64 bytes first, odd rows the last: 8 lanes meet all banks
                const uint32_t ca = code + ra * ns * (SLICE / 2), cb = code + rb * ns * (SLICE / 2), odd = (r & 1) * 64;
                uint4 wa[2], wb[2];
                const uint4 a0 = lds128(ca + odd), a1 = lds128(ca + (odd ^ 64)), b0 = lds128(cb + odd), b1 = lds128(cb + (odd ^ 64));
                const uint4 sa = lds128(scale + ra * ns * (SLICE / 16)), sb = lds128(scale + rb * ns * (SLICE / 16));
                wa[0] = odd ? a1 : a0, wa[1] = odd ? a0 : a1, wb[0] = odd ? b1 : b0, wb[1] = odd ? b0 : b1;
                float acc[NT][4] = {};
                const bool second = NT > 1 && it.m > 8;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    // the two scales of these 32 weights: bytes 8 c + 2 q, + 1
                    const uint32_t a2 = (q & 2 ? (c ? sa.w : sa.y) : (c ? sa.z : sa.x)) >> (16 * (q & 1));
                    const uint32_t b2 = (q & 2 ? (c ? sb.w : sb.y) : (c ? sb.z : sb.x)) >> (16 * (q & 1));
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t va[4], vb[4];
                        e2m1x8_mul_h2(u4_word(wa[c], w), e4m3_to_h2(a2 >> (8 * (w >> 1))), va);
                        e2m1x8_mul_h2(u4_word(wb[c], w), e4m3_to_h2(b2 >> (8 * (w >> 1))), vb);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int x = 16 * c + 4 * w + 2 * h;
                            mma_f16(acc[0], va[2 * h], vb[2 * h], va[2 * h + 1], vb[2 * h + 1], xf[0][x], xf[0][x + 1]);
                            if (NT > 1 && second)
                                mma_f16(acc[NT - 1], va[2 * h], vb[2 * h], va[2 * h + 1], vb[2 * h + 1], xf[NT - 1][x], xf[NT - 1][x + 1]);
                        }
                    }
                }
                // the expert's scale first: the sums are within f16's range times 2^20 here
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sum[t][j] = fmaf(__fmul_rn(acc[t][j], outer), unscale[t][j & 1], sum[t][j]);
            }
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1;
            }
            if (pass + 1 < p.passes) {
                __syncthreads();  // the pass has been read
                if (warp == WARPS - 1) ask();
            }
        }
        // join the warps' shares of K
        float *part = reinterpret_cast<float *>(smem + S::PART_OFF + buf * S::PART_BYTES);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float *o = part + (warp * NT + t) * PART + r;
            o[(2 * q) * PITCH] = sum[t][0];
            o[(2 * q + 1) * PITCH] = sum[t][1];
            o[(2 * q) * PITCH + 8] = sum[t][2];
            o[(2 * q + 1) * PITCH + 8] = sum[t][3];
        }
        __syncthreads();
        if (warp == WARPS - 1) ask();
        if (*(volatile int *)s_abort) continue;
        const int m = min(8 * NT, it.m), row0 = it.tile * half_rows, cols = (int)min((int64_t)half_rows, half_n - row0);
        for (int o = threadIdx.x; o < m * half_rows; o += THREADS) {
            const int n = o / half_rows, c = o - n * half_rows;
            if (c >= cols) continue;
            const int g = GATED ? c >> 3 : c >> 4, rr = GATED ? c & 7 : c & 15;
            const float *v = part + (g * p.slices * NT + (n >> 3)) * PART + (n & 7) * PITCH + rr;
            float a = 0.0f, b = 0.0f;
            for (int w = 0; w < p.slices; ++w) {
                a = __fadd_rn(a, v[w * NT * PART]);
                if (GATED) b = __fadd_rn(b, v[w * NT * PART + 8]);
            }
            if (GATED) a = __fmul_rn(__fmul_rn(a, __fdividef(1.0f, __fadd_rn(1.0f, __expf(-a)))), b);
            store_one(static_cast<OUT *>(p.out) + (it.r0 + n) * half_n + row0 + c, a);
        }
    }
    // after a timeout copies that nobody waited for may still be landing
    if (warp == WARPS - 1 && dead)
        for (int64_t a = max((int64_t)0, asked - STAGES); a < asked; ++a)
            (void)warp_wait(bar_full + 8 * (uint32_t)(a % STAGES), (uint32_t)(a / STAGES) & 1u, DRAIN_NS);
}

inline bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int NT, bool GATED, typename OUT>
pmn_status launch(const Args &args, cudaStream_t s)
{
    auto kern = matvec_kernel<NT, GATED, OUT>;
    static std::atomic<int> sm_count[MAX_DEVICES];  // of each device this kernel has been set up on
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return PMN_ERR_CUDA;
    int sms = dev < MAX_DEVICES ? sm_count[dev].load(std::memory_order_acquire) : 0;
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1 ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<NT>::BYTES) != cudaSuccess)
            return PMN_ERR_CUDA;
        if (dev < MAX_DEVICES) sm_count[dev].store(sms, std::memory_order_release);
    }
    kern<<<sms, THREADS, Smem<NT>::BYTES, s>>>(args);
    return cudaGetLastError() == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

template <bool GATED, typename OUT>
pmn_status launch_by_rows(const Args &args, cudaStream_t s)
{
    return args.rows <= 8 ? launch<1, GATED, OUT>(args, s) : launch<2, GATED, OUT>(args, s);
}

}  // namespace

pmn_status pmn_take_matvec_device_error(cudaStream_t s, int *bits)
{
    int host = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbolAsync(&host, g_matvec_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return PMN_ERR_CUDA;
    if (host != 0 &&
        (cudaMemcpyToSymbolAsync(g_matvec_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
         cudaStreamSynchronize(s) != cudaSuccess))
        return PMN_ERR_CUDA;
    *bits = host;
    return PMN_OK;
}

extern "C" pmn_status pmn_matvec_nvfp4(const void *x, int64_t ldx, int64_t tokens, const uint8_t *codes,
                                       const uint8_t *scales, const float *outer, const int32_t *offsets,
                                       int num_experts, int64_t total_rows, int64_t n, int64_t k,
                                       const int32_t *row_choice, int choices, int swiglu, int out_kind, void *out,
                                       void *stream)
{
    if (num_experts <= 0 || num_experts > MAX_GROUPS || total_rows < 0 || total_rows >= (int64_t(1) << 31) - 64 || tokens < 0 ||
        tokens >= (int64_t(1) << 31) || n <= 0 || n % 16 != 0 || n >= (int64_t(1) << 28) || k <= 0 || k % 256 != 0 ||
        k >= (int64_t(1) << 28) || ldx < k || ldx % 8 != 0 || (swiglu != 0 && swiglu != 1) || choices < 1 ||
        (out_kind != PMN_OUT_BF16 && out_kind != PMN_OUT_F32) || (!row_choice && tokens != total_rows))
        return PMN_ERR_INVALID_ARG;
    if (total_rows == 0) return PMN_OK;
    if ((!x && tokens > 0) || !codes || !scales || !outer || !offsets || !out || !aligned(x, 16) || !aligned(codes, 16) ||
        !aligned(scales, 16) || !aligned(outer, 4) || !aligned(offsets, 4) || !aligned(row_choice, 4) || !aligned(out, 16))
        return PMN_ERR_INVALID_ARG;
    const int all = (int)(k / SLICE), passes = (all + WARPS - 1) / WARPS, slices = (all + passes - 1) / passes;
    const int groups = WARPS / slices, per_half = (swiglu ? 8 : 16) * groups;
    const int64_t half_n = swiglu ? n / 2 : n;
    const Args a{static_cast<const uint16_t *>(x), ldx, tokens, codes, scales, outer, offsets, num_experts, total_rows, n, k,
                 row_choice, choices, out, all, slices, passes, groups, (int)((half_n + per_half - 1) / per_half),
                 pmn_wait_limit_ns()};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (swiglu) return out_kind == PMN_OUT_F32 ? launch_by_rows<true, float>(a, s) : launch_by_rows<true, uint16_t>(a, s);
    return out_kind == PMN_OUT_F32 ? launch_by_rows<false, float>(a, s) : launch_by_rows<false, uint16_t>(a, s);
}
