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
//
// Measured on one GB300 (d_model 4096, d_ff 1536; device time, operands larger than L2
// or streaming through it), and what bounds it:
//   forward, training, 8192 rows of 24 experts    97 us   2.1 PFLOP/s   8.2 rounds of 256-row tiles
//                                                (6.7 without the segments' ends) take 9;
//                                                the bytes alone 62 us
//   forward, serving, 16384 rows of one expert   120 us   3.4 PFLOP/s   the tensor pipe: 430 clocks a stage,
//                                                of which 384 are MMAs, plus the ends of 14 rounds
//   backward, 8192 rows of 24 experts             68 us   1.5 PFLOP/s   4.1 rounds take 5; as the next
//   backward, 16384 rows of one expert            92 us   2.2 PFLOP/s   the operand copies beside the
//                                                epilogue's requests: 18 to 22 thousand clocks a
//                                                tile, forward 15 to 16, the MMAs alone 13.8
//   forward, serving, 512 rows of 24 experts      52 us   6.0 TB/s      HBM (46 us)
//   forward, serving, one row                    4.4 us   3.0 TB/s      latency: a launch, two
//                                                dependent reads, a cluster barrier
//   148096 rows of 384 experts: training 2.00 ms   1.9 PFLOP/s   the segments' ends: 386 rows each
//     backward 1.22 ms, serving 1.51 ms                          take two 256-row tiles
// What the tiles and roles are for: 192 weight rows per tile leave TMEM room for two
// accumulators beside the scale factors, so the epilogue of one tile runs while the
// next is multiplied; two CTAs per 256-row tile load 28 KB per stage and SM where one
// loads 40 KB.  (When both were chosen, for 8192 rows forward, 8192 and 16384 rows
// backward: tiles of 256 with one accumulator 143, 112, 206 us, of 128 165, 112, 195,
// of 192 132, 100, 163; backward of 16384 rows by single CTAs 119, by pairs 101.)
// All of these are of f = 1536, which 96 and 192 columns of h divide; for other f the
// last column tile is part empty (forward 12 % more products at f = 256 and 512, half as
// many again at 128; backward 12 % at 512 and 1024, 20 % at 640, half at 128 and 256).
// Accuracy: the tensor core truncates its float32 sums, and the sigmoid comes from the
// hardware's exponential, so 2 to 2.6 times as many E4M3 codes fall on the other side of
// a rounding boundary as after a float32 product (5 to 11 in 10^6, off by one step).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/pmn.h"
#include "numerics.cuh"
#include "sm100.cuh"
#include "tensormap.cuh"

using namespace pmn;
using namespace pmn::sm100;

uint64_t pmn_wait_limit_ns();  // gemm.cu: the limit of every bounded device wait

namespace {

__device__ int g_gated_error = 0;

template <int CT>
__device__ __forceinline__ void mma_mxfp8_ct(uint32_t el, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate)
{
    if (CT == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate), "r"(el)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate), "r"(el)
            : "memory");
}

constexpr int BM = 128;  // rows per CTA
constexpr int MAX_GROUPS = 1024;
constexpr int MAX_DEVICES = 64;
constexpr uint32_t TMEM_COLS = 512;
// An epilogue warp's shared memory.  Backward: 32 rows x 32 columns of bf16 gate and
// up (2 x 2 KB), and, once those are in registers, two blocks that are being
// transposed (32 rows of 36 bytes each).  Forward for training: one such block.
constexpr int WARP_BUF = 4096, COL_BYTES = 32 * 36;

// Forward for serving (h alone), forward for training (h^T and y where wanted),
// backward.
constexpr int SERVE = 0, TRAIN = 1, BACKWARD = 2;

// One tile: 128 routed rows of an expert (CT = 2: 256 on a pair of CTAs) times TBN
// rows of its weight.  Forward: TBN / 2 gate rows and the TBN / 2 up rows of the same
// columns of h; backward: TBN columns of dH.  A stage holds 128 bytes of K of both
// operands (TMA, 128-byte swizzle) and their scale factors in the 32 x 128-bit form
// that tcgen05.cp copies into TMEM.
template <int MODE, int TBN, int CT>
struct Cfg {
    static constexpr bool BWD = MODE == BACKWARD;
    static constexpr int HB = BWD ? TBN : TBN / 2;  // columns of h (dH) per tile
    // Epilogue warps: GR per quarter of the rows.  No more than keep up with the main
    // loop, whose loads their stores get in the way of (training forward of 8192 rows:
    // 12 warps 101.5 us, 4 warps 100.4; backward of 8192 and 16384 rows: 12 warps 77.3
    // and 99.4, 8 warps 74.8 and 95.6).  Serving stores little, and with few tiles the
    // epilogue's latency counts.
    static constexpr int EW = BWD ? 8 : MODE == TRAIN ? 4 : 12, GR = EW / 4, THREADS = 128 + 32 * EW;
    static constexpr int NCH = HB / 32;              // 32-column chunks (MX blocks) of the epilogue
    static constexpr int CPW = NCH / GR;             // consecutive chunks per epilogue warp
    static constexpr int RB = (TBN + 127) / 128;    // 128-row scale blocks of B
    static constexpr int A_BYTES = BM * 128, B_BYTES = TBN / CT * 128;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES, SF_BYTES = 512 * (1 + RB);
    // Stages in flight, as many as fit (training forward of 8192 rows: 4 stages 115 us,
    // 5 101.5, 6 99.7; a seventh and sixth at the price of RAW_W = 16 lose more).
    static constexpr int STAGES = CT == 2 && !BWD ? 6 : 5;
    static constexpr uint32_t SF_COLS = 4 * (1 + RB);
    static constexpr int ACC = 2 * TBN + STAGES * (int)SF_COLS <= (int)TMEM_COLS ? 2 : 1;  // accumulators
    static constexpr uint32_t SF_COL0 = ACC * TBN;
    // Scale-factor warp w has the boxes of 32 scale rows at words 2 w, 2 w + 1 of each
    // block; a box holds RAW_W bytes of each row, a quarter as many stages' worth.
    // A row of a box costs TMA about as much as 128 bytes of a tile, so the boxes are as
    // wide as fits (training forward of 8192 rows: 16 bytes 103 us, 32 98.0, 64 96.5;
    // copied by the lanes with cp.async instead 101; with 512 rows 63 for 52).
    static constexpr int NR = 2 * (1 + RB);
    static constexpr bool in_tile(int j, int w) { return j < 2 || 128 * (j / 2 - 1) + 32 * (2 * w + (j & 1)) < TBN; }
    static constexpr int boxes(int w)
    {
        int n = 0;
        for (int j = 0; j < NR; ++j) n += in_tile(j, w);
        return n;
    }
    static constexpr int RAW_W = CT == 2 ? 64 : 16, RAW_SLOTS = 2, RAW_BOX = 32 * RAW_W;
    static constexpr int WARP_BYTES = BWD ? WARP_BUF : MODE == TRAIN ? COL_BYTES : 0;
    // column scales that a group of four warps collects: two buffers of 128 bytes per
    // block and chunk
    static constexpr int GROUP_BYTES = MODE == SERVE ? 0 : 2 * 128 * CPW * (BWD ? 2 : 1);
    static constexpr int SF_OFF = STAGES * STAGE_BYTES, WARP_OFF = SF_OFF + STAGES * SF_BYTES,
                         RAW_OFF = WARP_OFF + EW * WARP_BYTES, BAR_OFF = RAW_OFF + RAW_SLOTS * RAW_BOX * (boxes(0) + boxes(1)),
                         SCALE_OFF = BAR_OFF + 224, CUM_OFF = SCALE_OFF + GR * GROUP_BYTES;
    static constexpr int SMEM_BYTES = CUM_OFF + (MAX_GROUPS + 1) * 4;
    static_assert(NCH % GR == 0 && HB % 32 == 0 && (MODE == SERVE || CPW >= 3), "chunks per warp");
    static_assert(STAGE_BYTES % 1024 == 0 && SF_BYTES % 512 == 0, "TMA and descriptor alignment");
    static_assert(8 * (2 * STAGES + 8 + 2 * RAW_SLOTS) + 16 <= 224, "barrier space");
    static_assert(SF_COL0 + STAGES * SF_COLS <= TMEM_COLS, "TMEM budget");
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

struct Args {
    const int32_t *offsets;
    int groups;
    int64_t m, f, k;         // routed rows, columns of h, contraction length
    int64_t b_rows;          // rows of B of all experts
    uint8_t *out, *out_sc, *out_t, *out_t_sc;
    uint16_t *y;             // forward: written (or NULL); backward: read
    bool wide, wide_y;       // out, y are 32-byte aligned
    bool words;              // alignment lets four column scales be stored at once
    uint64_t wait_ns;
};

struct Tile {
    int g;
    int64_t m0, row_end;
    int h0;  // first column of h
};

template <int MODE, int TBN, int CT>
__device__ __forceinline__ Tile get_tile(int t, const Args &p, const int *s_cum, int &gc)
{
    while (gc + 1 < p.groups && s_cum[gc + 1] <= t) ++gc;  // every role walks its tiles upwards
    constexpr int HB = Cfg<MODE, TBN, CT>::HB;
    const int nt = (int)((p.f + HB - 1) / HB);
    const int local = t - s_cum[gc], mi = local / nt;
    Tile ti;
    ti.g = gc;
    ti.m0 = __ldg(p.offsets + gc) + (int64_t)mi * (CT * BM);  // of the tile
    ti.row_end = __ldg(p.offsets + gc + 1);
    ti.h0 = (local - mi * nt) * HB;
    return ti;
}

__device__ __forceinline__ void latch_error(int bit) { atomicOr(&g_gated_error, bit); }

// After a timeout a role still waits for its own copies and tensor operations in
// flight, this long for each: they need microseconds, but a barrier that counts
// another role's arrivals too may never complete.
constexpr uint64_t DRAIN_NS = 100000000ull;

// Instruction descriptor of the block-scaled MMA: E4M3 operands, E8M0 scales,
// M = 128 per CTA, N = TBN; sf_id selects the scale byte of the 32-deep K step.
template <int TBN, int CT>
__device__ __forceinline__ uint32_t make_idesc(uint32_t sf_id)
{
    return (sf_id << 4) | ((uint32_t)(TBN >> 3) << 17) | (1u << 23) | ((uint32_t)(CT * BM >> 4) << 24) | (sf_id << 29);
}

// 1 / (1 + e^-g) on two lanes, from the hardware's exponential and reciprocal: a
// relative error of a few 2^-23 and (the argument's rounding) |g| 2^-23; 0 and 1
// where e^-g leaves float32's normal range.
__device__ __forceinline__ void sigmoid2(float g0, float g1, float &s0, float &s1)
{
    float a0, a1, b0, b1;
    mul2(g0, g1, -1.44269504f, -1.44269504f, a0, a1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b0) : "f"(a0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b1) : "f"(a1));
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\t"
        "add.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}" : "=f"(a0), "=f"(a1) : "f"(b0), "f"(b1), "f"(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s0) : "f"(a0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s1) : "f"(a1));
}

// a * b + c on two lanes, each rounded once.
__device__ __forceinline__ void fma2v(float a0, float a1, float b0, float b1, float c0, float c1, float &r0, float &r1)
{
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r0), "=f"(r1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

// Four values times their scales -> four E4M3 bytes, nearest even.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float sa, float sb, float sc, float sd)
{
    float x[4];
    mul2(a, b, sa, sb, x[0], x[1]);
    mul2(c, d, sc, sd, x[2], x[3]);
    return cvt_e4m3x2_rn(x[0], x[1]) | (cvt_e4m3x2_rn(x[2], x[3]) << 16);
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
    for (int j = 0; j < 8; ++j) w[j] = e4m3x4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], s, s, s, s);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// 16-byte piece i of row r in 32 rows of 64 bytes: eight lanes that access one
// piece of eight consecutive rows, or the four pieces of two rows, meet eight
// different bank groups.
__device__ __forceinline__ int piece64(int r, int i) { return 64 * r + 16 * (i ^ ((r >> 1) & 3)); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 32 bytes of one row: a whole sector in one store where the tensor is 32-byte aligned.
__device__ __forceinline__ void store32(uint8_t *o, const uint4 (&q)[2], bool wide)
{
    if (wide)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(q[0].x), "r"(q[0].y),
                     "r"(q[0].z), "r"(q[0].w), "r"(q[1].x), "r"(q[1].y), "r"(q[1].z), "r"(q[1].w)
                     : "memory");
    else {
        reinterpret_cast<uint4 *>(o)[0] = q[0];
        reinterpret_cast<uint4 *>(o)[1] = q[1];
    }
}

__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Largest magnitude over the warp's lanes (NaN ignored, as fmaxf does).
__device__ __forceinline__ uint32_t warp_absmax(float v)
{
    float m;
    asm volatile("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return __float_as_uint(m);
}

// MXFP8 along the rows of a warp's 32 x 32 block (lane = row, v[j] = column j).
// A column's maximum is one reduction over the lanes, so the values are scaled
// and converted where they are and only bytes are transposed: through shared
// memory (rows 36 bytes apart: conflict-free both ways), lane 4 k + r then holds
// columns 4 k .. 4 k + 3, rows 8 r .. 8 r + 7.
// The exponent rule of mx_exponent_448 on the bits M of the maximum: with
// t = (max(M, 8 << 23) + 0x1FFFFF) >> 23 (a carry where M's fraction is above 1.75),
// e = t - 135, so the scale byte is t - 8 and 2^-e has the exponent field 262 - t.
// q: the block's first column at its first row; pitch: bytes between columns.
// NB blocks are worked on side by side, as each step waits on the one before.
template <int NB>
__device__ __forceinline__ void col_blocks(const float (*const (&v)[NB])[32], uint8_t *buf, uint8_t *const (&q)[NB],
                                           int64_t pitch, uint8_t (&sc)[NB], int lane)
{
    uint32_t sb[NB][8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            float x[4], m[4];
            uint32_t t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = (*v[n])[4 * k + i];
                t[i] = max(warp_absmax(x[i]), 0x04000000u) - (0x04000000u - 0x1FFFFFu);  // byte in bits 23 .. 30
                m[i] = __uint_as_float(0x7F000000u - (t[i] & 0x7F800000u));
            }
            *reinterpret_cast<uint32_t *>(buf + n * COL_BYTES + 36 * lane + 4 * k) =
                e4m3x4(x[0], x[1], x[2], x[3], m[0], m[1], m[2], m[3]);
            sb[n][k] = __byte_perm(__byte_perm(t[0] << 1, t[1] << 1, 0x0073), __byte_perm(t[2] << 1, t[3] << 1, 0x0073),
                                   0x5410);
        }
    __syncwarp();
    const int k = lane >> 2, r = lane & 3;
    uint32_t w[NB][8];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[n][i] = *reinterpret_cast<const uint32_t *>(buf + n * COL_BYTES + 36 * (8 * r + i) + 4 * k);
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        uint2 o[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 4 x 4 bytes each
            const uint32_t w0 = w[n][4 * h], w1 = w[n][4 * h + 1], w2 = w[n][4 * h + 2], w3 = w[n][4 * h + 3];
            const uint32_t a = __byte_perm(w0, w1, 0x5140), b = __byte_perm(w2, w3, 0x5140);
            const uint32_t c = __byte_perm(w0, w1, 0x7362), d = __byte_perm(w2, w3, 0x7362);
            (h ? o[0].y : o[0].x) = __byte_perm(a, b, 0x5410);
            (h ? o[1].y : o[1].x) = __byte_perm(a, b, 0x7632);
            (h ? o[2].y : o[2].x) = __byte_perm(c, d, 0x5410);
            (h ? o[3].y : o[3].x) = __byte_perm(c, d, 0x7632);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint2 *>(q[n] + (4 * k + i) * pitch + 8 * r) = o[i];
        const uint32_t s01 = k & 1 ? sb[n][1] : sb[n][0], s23 = k & 1 ? sb[n][3] : sb[n][2],
                       s45 = k & 1 ? sb[n][5] : sb[n][4], s67 = k & 1 ? sb[n][7] : sb[n][6];
        const uint32_t lo = k & 2 ? s23 : s01, hi = k & 2 ? s67 : s45;
        sc[n] = (uint8_t)((k & 4 ? hi : lo) >> (8 * r));
    }
}

// One persistent kernel per call, one CTA per SM (CT = 2: a pair per two SMs, whose
// leader issues the MMAs of both):
//   warp 0      loads the operands' code tiles by TMA
//   warp 1      copies a stage's scale factors into TMEM and issues its MMAs (copies
//               and MMAs of one lane execute in order)
//   warps 2, 3  put the scale rows into the form that tcgen05.cp expects
//   warps 4..   epilogue: a row per thread, 32 columns at a time
// Every wait is bounded: on a timeout an error bit is latched and the CTA winds
// down.
template <int MODE, int TBN, int CT>
__global__ void __launch_bounds__(Cfg<MODE, TBN, CT>::THREADS, 1)
    gated_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB, const Args p)
{
    using C = Cfg<MODE, TBN, CT>;
    constexpr bool BWD = MODE == BACKWARD;
    constexpr int STAGES = C::STAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];  // TMA and descriptors: 1024-byte swizzle atoms
    // the compiler is kept from knowing the address: with it the MMA loop's operands are
    // formed by a longer chain (forward of 16384 rows 123 -> 132 us)
    uint8_t *smem = smem_raw;
    asm volatile("" : "+l"(smem));
    const uint32_t stages = smem_u32(smem);
    const uint32_t bar_full = stages + C::BAR_OFF, bar_empty = bar_full + 8 * STAGES;
    const uint32_t bar_acc_full = bar_empty + 8 * STAGES, bar_acc_empty = bar_acc_full + 16;
    const uint32_t bar_drain = bar_acc_empty + 16, bar_group = bar_drain + 8, bar_raw = bar_group + 24;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::BAR_OFF + 8 * (2 * STAGES + 8 + 2 * C::RAW_SLOTS));
    int *s_abort = reinterpret_cast<int *>(tmem_slot + 1);
    int *s_total = s_abort + 1;
    int *s_cum = reinterpret_cast<int *>(smem + C::CUM_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CT == 2 ? (int)cluster_rank() : 0;
    const int tile0 = blockIdx.x / CT, tstep = gridDim.x / CT;  // tiles of this CTA (pair)

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1 + 2 * CT);  // the code tiles' bytes, each CTA's two scale-factor warps
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_acc_full + 8 * b, 1);
            mbar_init(bar_acc_empty + 8 * b, CT * C::EW);
        }
        mbar_init(bar_drain, 1);
        for (int g = 0; g < 3; ++g) mbar_init(bar_group + 8 * g, 4);
        for (int g = 0; g < 2 * C::RAW_SLOTS; ++g) mbar_init(bar_raw + 8 * g, 1);
        *s_abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmSA);
        tma_prefetch_desc(&tmSB);
    }
    if (warp == 0) {
        __syncwarp();
        tmem_alloc_ct<CT>(smem_u32(tmem_slot), TMEM_COLS);
    }
    if (warp == 1) {
        // tiles of each group and their running sum, 32 groups at a time; offsets
        // that are not monotone, in range and (with column blocks) multiples of
        // 32 run no tile
        const int nt = (int)((p.f + C::HB - 1) / C::HB);
        const bool cols = MODE != SERVE && p.out_t != nullptr;
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
            int n = (hi - lo + CT * BM - 1) / (CT * BM) * nt, sum = n;
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
    if (CT == 2) cluster_sync();  // the pair's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // A last round of few tiles: two or three pairs multiply each of them and each
    // stores a share of its columns, so that the epilogue that nothing overlaps is short
    // (backward of 8192 rows of 24 experts 73.5 -> 68.3 us, of 256 rows of one 18.6 -> 14.5).
    const int all = __shfl_sync(0xFFFFFFFFu, *s_total, 0), tail = all % tstep, full = all - tail;
    const int shares = MODE == SERVE ? 1 : 3 * tail <= tstep ? 3 : 2 * tail <= tstep ? 2 : 1;
    const int total = full + shares * tail;
    auto tile_at = [&](int t) { return t < full ? t : full + (t - full) / shares; };
    const int nks = (int)(p.k / 128);
    auto give_up = [&]() {  // a wait ran out: every role winds down
        if (lane == 0) {
            *(volatile int *)s_abort = 1;
            latch_error(PMN_DEVERR_WAIT_TIMEOUT);
        }
    };

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        uint32_t stage = 0, phase = 0, issued = 0, last = 0;
        int gc = 0;
        bool ok = true;
        // first row of B that this CTA loads for a tile (single CTA: of the gate half)
        auto b_row = [&](const Tile &ti) {
            const int64_t br = (int64_t)ti.g * (BWD ? p.f : 2 * p.f) + ti.h0;
            return CT == 1 || rank == 0 ? br : BWD ? br + TBN / 2 : br + p.f;
        };
        for (int t = tile0; t < total && ok; t += tstep) {
            const Tile ti = get_tile<MODE, TBN, CT>(tile_at(t), p, s_cum, gc);
            const int32_t arow = (int32_t)ti.m0 + BM * rank, brow = (int32_t)b_row(ti);
            for (int ks = 0; ks < nks; ++ks) {
                ok = warp_wait(bar_empty + 8 * stage, phase ^ 1, p.wait_ns);
                if (!ok || __any_sync(0xFFFFFFFFu, *(volatile int *)s_abort != 0)) {
                    if (!ok) give_up();
                    ok = false;
                    break;
                }
                const uint32_t st = stages + stage * C::STAGE_BYTES, fb = bar_full + 8 * stage;
                const int32_t x = ks * 128;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(fb, CT * (C::A_BYTES + C::B_BYTES));
                    if constexpr (CT == 2) {
                        // forward: the leader holds the gate rows, its peer the up rows
                        tma_load_2d_pair(st, &tmA, leader_addr(fb), x, arow);
                        tma_load_2d_pair(st + C::A_BYTES, &tmB, leader_addr(fb), x, brow);
                    } else {
                        tma_load_2d(st, &tmA, fb, x, arow);
                        tma_load_2d(st + C::A_BYTES, &tmB, fb, x, brow);
                        if (!BWD) tma_load_2d(st + C::A_BYTES + C::B_BYTES / 2, &tmB, fb, x, (int32_t)(brow + p.f));
                    }
                }
                __syncwarp();
                issued |= 1u << stage;
                last = (last & ~(1u << stage)) | (phase << stage);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // no copy may still be landing when the CTA ends; a pair's copies are
        // counted by its leader, and both CTAs end together
        for (int s = 0; s < STAGES; ++s)
            if (rank == 0 && (issued & (1u << s))) (void)warp_wait(bar_full + 8 * s, (last >> s) & 1u, DRAIN_NS);
        if (CT == 2 && *(volatile int *)s_abort) {  // one side may have given up before the other: let copies land
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 10000000ull) {
            }
        }
        __syncwarp();
    } else if (warp == 2 || warp == 3) {
        // ---------------------------------------------------- scale factors
        // Block b (A, then the 128-row blocks of B), lane r, word j: the four
        // scale bytes of row 32 j + r of the stage's 128-deep K range.  Words 0, 1
        // are warp 2's, words 2, 3 warp 3's; both take part in every stage, as a
        // wait tells one phase of a barrier from the next alone.  The rows come by TMA,
        // two groups of RAW_W / 4 stages ahead, in boxes of 32 rows.  (Plain loads from
        // 32 rows each queue behind the epilogue's stores and held the MMAs up.)
        const int per_tile = (nks + C::RAW_W / 4 - 1) / (C::RAW_W / 4);
        const int wr = __shfl_sync(0xFFFFFFFFu, warp, 0) - 2;
        const int boxes = wr ? C::boxes(1) : C::boxes(0), slot_bytes = boxes * C::RAW_BOX;
        const int raw0 = C::RAW_OFF + wr * C::RAW_SLOTS * C::RAW_BOX * C::boxes(0);
        const uint32_t bar = bar_raw + 8 * C::RAW_SLOTS * wr;
        const int64_t tiles = tile0 < total ? (total - 1 - tile0) / tstep + 1 : 0, groups = tiles * per_tile;
        int64_t asked = 0;  // groups whose scales have been asked for
        int t = tile0, q = 0, gc = 0;
        Tile ti;
        if (t < total) ti = get_tile<MODE, TBN, CT>(tile_at(t), p, s_cum, gc);
        auto fetch = [&]() {
            if (asked >= groups) return;
            const int slot = (int)(asked % C::RAW_SLOTS);
            const int32_t arow = (int32_t)ti.m0 + BM * rank;
            const int64_t brow = (int64_t)ti.g * (BWD ? p.f : 2 * p.f) + ti.h0;
            uint32_t d = stages + raw0 + slot * slot_bytes;
            if (elect_one()) {
                mbar_arrive_expect_tx(bar + 8 * slot, slot_bytes);
#pragma unroll
                for (int j = 0; j < C::NR; ++j) {
                    const int n = 128 * (j / 2 - 1) + 32 * (2 * wr + (j & 1));  // row of B within the tile (j >= 2)
                    if (j >= 2 && n >= TBN) continue;
                    if (j < 2) tma_load_2d(d, &tmSA, bar + 8 * slot, C::RAW_W * q, arow + 32 * (2 * wr + j));
                    else
                        tma_load_2d(d, &tmSB, bar + 8 * slot, C::RAW_W * q,
                                    (int32_t)(brow + n + (!BWD && n >= C::HB ? p.f - C::HB : 0)));
                    d += C::RAW_BOX;
                }
            }
            __syncwarp();
            ++asked;
            if (++q == per_tile) {
                q = 0;
                t += tstep;
                if (t < total) ti = get_tile<MODE, TBN, CT>(tile_at(t), p, s_cum, gc);
            }
        };
        for (int i = 0; i < C::RAW_SLOTS; ++i) fetch();
        uint32_t stage = 0, phase = 0, rslot = 0, rphase = 0;
        bool ok = true;
        int64_t g = 0;
        int gq = 0;  // the group within its tile
        for (; g < groups && ok; ++g) {
            ok = warp_wait(bar + 8 * rslot, rphase, p.wait_ns);
            if (!ok) {
                give_up();
                break;
            }
            const uint8_t *raw = smem + raw0 + rslot * slot_bytes + C::RAW_W * lane;
            if (++rslot == C::RAW_SLOTS) {
                rslot = 0;
                rphase ^= 1;
            }
            const int parts = min(C::RAW_W / 16, nks / 4 - C::RAW_W / 16 * gq);  // k is a multiple of 512
            if (++gq == per_tile) gq = 0;
            for (int part = 0; part < parts && ok; ++part) {
                uint4 v[C::NR];
                int box = 0;
#pragma unroll
                for (int j = 0; j < C::NR; ++j) {
                    v[j] = make_uint4(0u, 0u, 0u, 0u);
                    if (j >= 2 && 128 * (j / 2 - 1) + 32 * (2 * wr + (j & 1)) >= TBN) continue;
                    v[j] = *reinterpret_cast<const uint4 *>(raw + box * C::RAW_BOX + 16 * part);
                    ++box;
                }
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    ok = ok && warp_wait(bar_empty + 8 * stage, phase ^ 1, p.wait_ns);
                    if (!ok || __any_sync(0xFFFFFFFFu, *(volatile int *)s_abort != 0)) {
                        if (!ok) give_up();
                        ok = false;
                        break;
                    }
                    uint2 *sf = reinterpret_cast<uint2 *>(smem + C::SF_OFF + stage * C::SF_BYTES) + 2 * lane + wr;
#pragma unroll
                    for (int b = 0; b < 1 + C::RB; ++b) sf[64 * b] = make_uint2(u4_word(v[2 * b], s), u4_word(v[2 * b + 1], s));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (CT == 2) mbar_arrive_leader(bar_full + 8 * stage);
                        else mbar_arrive(bar_full + 8 * stage);
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // the slot may be refilled: what was read from it has been written on
            if (ok) fetch();
        }
        // copies that nobody will wait for may still be landing
        for (; !ok && g < asked; ++g)
            (void)warp_wait(bar + 8 * (uint32_t)(g % C::RAW_SLOTS), (uint32_t)(g / C::RAW_SLOTS) & 1u, DRAIN_NS);
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        // The whole warp walks the loop, so that the operands of the tensor
        // instructions are warp-uniform values; one elected lane issues.
        if (rank == 0) {
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0), el = elect_one();
            uint32_t stage = 0, phase = 0, abuf = 0, aphase = 0;
            bool ok = true, ready = false;
            for (int t = tile0; t < total && ok; t += tstep) {
                ok = warp_wait(bar_acc_empty + 8 * abuf, aphase ^ 1, p.wait_ns);
                if (!ok || __any_sync(0xFFFFFFFFu, *(volatile int *)s_abort != 0)) {
                    if (!ok) give_up();
                    break;
                }
                const uint32_t d = tm + abuf * TBN;
                for (int ks = 0; ks < nks; ++ks) {
                    // asked for a stage ahead, the answer is there when it is needed
                    if (__all_sync(0xFFFFFFFFu, ready) == 0) {
                        ok = warp_wait(bar_full + 8 * stage, phase, p.wait_ns);
                        if (!ok) {
                            give_up();
                            break;
                        }
                    }
                    tc_fence_after();
                    const uint32_t a = stages + stage * C::STAGE_BYTES, b = a + C::A_BYTES;
                    const uint32_t sf = stages + C::SF_OFF + stage * C::SF_BYTES;
                    const uint32_t sfa = tm + C::SF_COL0 + stage * C::SF_COLS, sfb = sfa + 4, done = bar_empty + 8 * stage;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                    ready = mbar_test(bar_full + 8 * stage, phase);
#pragma unroll
                    for (int i = 0; i < 1 + C::RB; ++i)
                        tc_cp_ct<CT>(el, sfa + 4 * i, smem_desc(sf + 512 * i, 0, 128, 0));
#pragma unroll
                    for (int s = 0; s < 4; ++s)  // 32 of K per MMA inside the 128-byte swizzled rows
                        mma_mxfp8_ct<CT>(el, d, smem_desc(a + 32 * s, 16, 1024, 2), smem_desc(b + 32 * s, 16, 1024, 2),
                                         make_idesc<TBN, CT>((uint32_t)s), sfa, sfb, (ks > 0 || s > 0) ? 1u : 0u);
                    tc_commit_ct<CT>(el, done);
                }
                if (!ok) break;
                tc_commit_ct<CT>(el, bar_acc_full + 8 * abuf);
                if (++abuf == C::ACC) {
                    abuf = 0;
                    aphase ^= 1;
                }
            }
            if (elect_one()) tc_commit_own<CT>(bar_drain);  // every tcgen05 operation of this warp has completed
            __syncwarp();
            (void)warp_wait(bar_drain, 0, DRAIN_NS);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------- epilogue
        // Warp w reads accumulator lanes (rows) 32 (w % 4) .. + 31 of CPW chunks of
        // 32 columns in a row (of its share in a shared tile).
        const int wu = __shfl_sync(0xFFFFFFFFu, warp, 0);  // warp-uniform, and known to be
        const int quad = wu & 3, cw = ((wu - 4) >> 2) * C::CPW;
        const int per_share = (C::CPW + shares - 1) / shares;
        auto first_chunk = [&](int t) { return cw + (t < full ? 0 : (t - full) % shares * per_share); };
        uint8_t *buf = smem + C::WARP_OFF + (wu - 4) * C::WARP_BYTES;
        const uint32_t bufs = stages + C::WARP_OFF + (wu - 4) * C::WARP_BYTES;
        const int pr = lane >> 2, pi = lane & 3;  // four lanes cover a row's 64 bytes of y
        // The four warps that hold a chunk's 128 rows collect its column scales, so
        // that a column's four bytes leave in one store: two buffers in turn, one
        // barrier per tile.
        const int group = (wu - 4) >> 2;
        uint8_t *const sscale0 = smem + C::SCALE_OFF + group * C::GROUP_BYTES;
        uint32_t collected = 0;
        uint32_t abuf = 0, aphase = 0;
        int gc = 0;
        bool ok = true, have = false;  // have: the tile's first gate and up values have been asked for
        // backward: copies gate and up of 32 rows x 32 columns into the buffer
        auto fetch_y = [&](int64_t row0, int64_t col) {
            const uint16_t *g = p.y + (row0 + pr) * 2 * p.f + col + 8 * pi;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t d = bufs + piece64(pr + 8 * i, pi);
                cp_async16(d, g + 16 * i * p.f);
                cp_async16(d + WARP_BUF / 2, g + 16 * i * p.f + p.f);
            }
        };
        for (int t = tile0; t < total && ok; t += tstep) {
            const Tile ti = get_tile<MODE, TBN, CT>(tile_at(t), p, s_cum, gc);
            const int c0 = first_chunk(t), c1 = min(t < full ? c0 + C::CPW : c0 + per_share, cw + C::CPW);
            const int64_t row0 = ti.m0 + BM * rank + 32 * quad, row = row0 + lane;
            const bool valid = row < ti.row_end, any = row0 < ti.row_end;
            const int64_t tile_row = ti.m0 + BM * rank;
            const bool words = MODE != SERVE && p.words && tile_row % 128 == 0 && tile_row + BM <= ti.row_end;
            uint8_t *const sscale = sscale0 + C::GROUP_BYTES / 2 * (collected & 1u);
            // The next tile's first gate and up values are asked for once this tile's
            // last ones have been used.
            bool has_next = false;
            int64_t next_row0 = 0, next_col = 0;
            if (BWD) {
                if (!have && any && ti.h0 + 32 * c0 < p.f) fetch_y(row0, ti.h0 + 32 * c0);
                have = false;
                if (t + tstep < total) {
                    int g2 = gc;
                    const Tile tn = get_tile<MODE, TBN, CT>(tile_at(t + tstep), p, s_cum, g2);
                    next_row0 = tn.m0 + BM * rank + 32 * quad;
                    next_col = tn.h0 + 32 * first_chunk(t + tstep);
                    has_next = next_row0 < tn.row_end && next_col < p.f;
                    have = has_next && any && ti.h0 + 32 * c0 < p.f;
                }
            }
            ok = warp_wait(bar_acc_full + 8 * abuf, aphase, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(32 * quad) << 16) + abuf * TBN;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CT == 2) mbar_arrive_leader(bar_acc_empty + 8 * abuf);
                    else mbar_arrive(bar_acc_empty + 8 * abuf);
                }
            };
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
                const int64_t col = ti.h0 + 32 * c;
                const bool on = any && col < p.f;  // (with column blocks: all 32 rows are valid)
                float v[32], u[32];
                uint4 q[2];
                uint8_t sc;
                if constexpr (!BWD) {
                    tmem_ld_32x32b_x32(acc + 32 * c, reinterpret_cast<uint32_t(&)[32]>(v));
                    tmem_ld_32x32b_x32(acc + C::HB + 32 * c, reinterpret_cast<uint32_t(&)[32]>(u));
                    tmem_ld_wait();
                    if (c == c1 - 1) release();
                    if (!on) continue;
                    if (MODE == TRAIN && p.y && valid) {
                        // y in bf16 for the backward pass, whole sectors straight from
                        // the row's thread (through shared memory, four lanes to a row's
                        // 64 bytes: the same time, and a stage's worth of memory)
                        uint16_t *o = p.y + row * 2 * p.f + col;
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const float *x = (h & 2 ? u : v) + 16 * (h & 1);
                            uint32_t w[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                                w[i] = *reinterpret_cast<const uint32_t *>(&b2);
                            }
                            const uint4 y2[2] = {make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
                            store32(reinterpret_cast<uint8_t *>(o + (h & 2 ? p.f : 0) + 16 * (h & 1)), y2, p.wide_y);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float s0, s1;
                        sigmoid2(v[j], v[j + 1], s0, s1);
                        mul2(v[j], v[j + 1], s0, s1, s0, s1);
                        mul2(s0, s1, u[j], u[j + 1], v[j], v[j + 1]);
                    }
                    row_block(v, q, sc);
                    if (valid) {
                        store32(p.out + row * p.f + col, q, p.wide);
                        p.out_sc[row * (p.f / 32) + col / 32] = sc;
                    }
                    if (MODE == TRAIN && p.out_t) {
                        uint8_t st[1];
                        col_blocks<1>({&v}, buf, {p.out_t + col * p.m + row0}, p.m, st, lane);
                        if (words) sscale[128 * (c - c0) + 4 * lane + quad] = st[0];
                        else p.out_t_sc[(col + lane) * (p.m / 32) + row0 / 32] = st[0];
                    }
                } else {
                    tmem_ld_32x32b_x32(acc + 32 * c, reinterpret_cast<uint32_t(&)[32]>(v));
                    cp_async_wait();
                    __syncwarp();
                    tmem_ld_wait();
                    if (c == c1 - 1) release();
                    if (!on) continue;
                    // The gate and up values leave the buffer before it is written again:
                    // they are in the codes stored below.  (Copies by TMA overtook reads
                    // that were still outstanding behind a warp barrier and even a
                    // barrier's arrival; these copies are the lanes' own, in order.)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 gw = *reinterpret_cast<const uint4 *>(buf + piece64(lane, i));
                        const uint4 uw = *reinterpret_cast<const uint4 *>(buf + WARP_BUF / 2 + piece64(lane, i));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int j = 8 * i + 2 * k;
                            const uint32_t a = u4_word(gw, k), b = u4_word(uw, k);
                            const float g0 = __uint_as_float(a << 16), g1 = __uint_as_float(a & 0xFFFF0000u);
                            const float u0 = __uint_as_float(b << 16), u1 = __uint_as_float(b & 0xFFFF0000u);
                            float s0, s1, d0, d1, k0, k1;
                            sigmoid2(g0, g1, s0, s1);
                            mul2(v[j], v[j + 1], s0, s1, d0, d1);             // dh s
                            mul2(d0, d1, g0, g1, u[j], u[j + 1]);             // dup
                            fma2v(s0, s1, -1.0f, -1.0f, 1.0f, 1.0f, k0, k1);  // 1 - s
                            fma2v(g0, g1, k0, k1, 1.0f, 1.0f, k0, k1);        // 1 + gate (1 - s)
                            mul2(d0, d1, u0, u1, d0, d1);
                            mul2(d0, d1, k0, k1, v[j], v[j + 1]);             // dgate
                        }
                    }
                    const int64_t f2 = 2 * p.f;
                    uint8_t *os = p.out_sc + row * (f2 / 32) + col / 32;
                    row_block(v, q, sc);
                    store32(p.out + row * f2 + col, q, p.wide);
                    os[0] = sc;
                    row_block(u, q, sc);
                    store32(p.out + row * f2 + p.f + col, q, p.wide);
                    os[p.f / 32] = sc;
                    __syncwarp();
                    uint8_t st[2];
                    uint8_t *qt = p.out_t + col * p.m + row0;
                    col_blocks<2>({&v, &u}, buf, {qt, qt + p.f * p.m}, p.m, st, lane);
                    if (words) {
                        sscale[256 * (c - c0) + 4 * lane + quad] = st[0];
                        sscale[256 * (c - c0) + 128 + 4 * lane + quad] = st[1];
                    } else {
                        uint8_t *ot = p.out_t_sc + (col + lane) * (p.m / 32) + row0 / 32;
                        ot[0] = st[0];
                        ot[p.f * (p.m / 32)] = st[1];
                    }
                    if (c + 1 < c1 && col + 32 < p.f) fetch_y(row0, col + 32);  // the blocks above have been read
                    else if (has_next) fetch_y(next_row0, next_col);
                }
            }
            if (words) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_group + 8 * group);
                ok = warp_wait(bar_group + 8 * group, collected & 1u, p.wait_ns);
                if (!ok) break;
                ++collected;
                constexpr int NOUT = BWD ? 2 : 1;  // slot: chunk and (backward) gate or up
                for (int s = quad; s < (c1 - c0) * NOUT; s += 4) {
                    const int64_t col = ti.h0 + 32 * (c0 + s / NOUT) + lane;
                    if (col < p.f)
                        *reinterpret_cast<uint32_t *>(p.out_t_sc + (col + (s % NOUT) * p.f) * (p.m / 32) + tile_row / 32) =
                            *reinterpret_cast<const uint32_t *>(sscale + 128 * s + 4 * lane);
                }
            }
            if (++abuf == C::ACC) {
                abuf = 0;
                aphase ^= 1;
            }
        }
        if (!ok) give_up();
        if (BWD) cp_async_wait();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (CT == 2) cluster_sync();  // neither CTA's memory is still in use by the other
    tc_fence_after();
    if (warp == 0) tmem_dealloc_ct<CT>(tmem, TMEM_COLS);
    if (CT == 2) cluster_sync();
}

// ---------------------------------------------------------------- few rows
// The forward for a handful of rows (single tokens of a serving loop): its time is
// that of reading the weights, which 128-row tiles would spread over a dozen SMs.
// A cluster of 1 to 8 CTAs takes 32 columns of h for one row, each CTA a share of K
// in units of 512; a warp holds 8 of the 64 weight rows, a lane 16 consecutive codes
// of each (512 bytes per warp load), multiplied in float32 and scaled once per half
// block.  The partial sums meet in the leader's shared memory.  Rows of one expert
// share its weights through L2 only.  Bound by latency for one row, by the decoding
// and multiplying for more (three CTAs per SM: 80 registers; two with more loads in
// flight are slower).
constexpr int FEW_CTAS = 8;  // at most

// 16 E4M3 codes -> float32
__device__ __forceinline__ void decode16(const uint4 &q, float (&v)[16])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t h2;
        const uint16_t b16 = (uint16_t)(u4_word(q, i >> 1) >> (16 * (i & 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(b16));
        v[2 * i] = h2_lo_to_f32(h2);
        v[2 * i + 1] = h2_hi_to_f32(h2);
    }
}

__global__ void __launch_bounds__(256, 3) gated_rows_kernel(const uint8_t *__restrict__ a, const uint8_t *__restrict__ sa, const uint8_t *__restrict__ b,
                      const uint8_t *__restrict__ sb, const Args p)
{
    __shared__ float part[FEW_CTAS][64];  // the leader's: gate sums 0 .. 31, up sums 32 .. 63
    __shared__ int s_expert;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank(), ctas = (int)cluster_ctas();
    const int64_t t = blockIdx.y;
    const int64_t col = 32 * (int64_t)(blockIdx.x / ctas);
    if (threadIdx.x == 0) s_expert = -1;
    __syncthreads();
    bool good = true;
    for (int e = threadIdx.x; e < p.groups; e += 256) {
        const int lo = __ldg(p.offsets + e), hi = __ldg(p.offsets + e + 1);
        if (lo < 0 || hi < lo || hi > p.m) good = false;
        if (lo <= t && t < hi) s_expert = e;
    }
    good = __syncthreads_and(good) != 0;
    if (!good) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) latch_error(PMN_DEVERR_BAD_OFFSETS);
        return;  // alike in every CTA
    }
    if (s_expert < 0) return;  // a row outside the segments: alike in the cluster
    // the leader's memory is written below: every CTA of the cluster has to have begun
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int64_t wrow = (int64_t)s_expert * 2 * p.f + (warp >= 4 ? p.f : 0) + col + 8 * (warp & 3);
    const int64_t pitch = p.k / 32;
    const uint8_t *wp = b + wrow * p.k + 16 * lane, *wsp = sb + wrow * pitch + lane / 2;
    const uint8_t *xp = a + t * p.k + 16 * lane, *xsp = sa + t * pitch + lane / 2;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    const int units = (int)(p.k / 512);
#pragma unroll 2
    for (int u = rank; u < units; u += ctas) {
        uint4 w[8];
        uint32_t ws[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = __ldcs(reinterpret_cast<const uint4 *>(wp + j * p.k + 512 * u));
            ws[j] = __ldg(wsp + j * pitch + 16 * u);
        }
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(xp + 512 * u));
        const float s = e8m0_to_f32(__ldg(xsp + 16 * u));
        float xv[16];
        decode16(x, xv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float wv[16];
            decode16(w[j], wv);
            float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; i += 2) fma2v(wv[i], wv[i + 1], xv[i], xv[i + 1], d0, d1, d0, d1);
            // the scales first: one of them alone may take the sum out of float32's range
            acc[j] = fmaf(__fadd_rn(d0, d1), e8m0_to_f32(ws[j]) * s, acc[j]);
        }
    }
    // A sum that is not finite is formed again: the product of the scales may have passed
    // float32's range on its own, beside codes whose sum is 0, and a byte of 255 is NaN,
    // where the factor above is infinite.
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) odd |= !(fabsf(acc[j]) <= 3.402823466e38f);
    if (odd) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
#pragma unroll 1
        for (int u = rank; u < units; u += ctas) {
            const uint32_t xs = __ldg(xsp + 16 * u);
            float xv[16];
            decode16(__ldg(reinterpret_cast<const uint4 *>(xp + 512 * u)), xv);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t ws = __ldg(wsp + j * pitch + 16 * u);
                float wv[16], d = 0.0f;
                decode16(__ldg(reinterpret_cast<const uint4 *>(wp + j * p.k + 512 * u)), wv);
#pragma unroll
                for (int i = 0; i < 16; ++i) d = fmaf(wv[i], xv[i], d);
                const uint32_t lo = (xs + ws) >> 1, hi = xs + ws - lo;  // 2^(xs + ws - 254) in two factors
                acc[j] = xs == 255u || ws == 255u ? __uint_as_float(0x7FC00000u)
                                                  : fmaf(__fmul_rn(d, e8m0_to_f32(lo)), e8m0_to_f32(hi), acc[j]);
            }
        }
    }
    // The lanes' sums of the 8 rows: the first three steps halve the rows a lane holds.
    float mine;
    {
        float a4[4], a2[2];
        const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float give = h16 ? acc[j] : acc[j + 4];
            a4[j] = (h16 ? acc[j + 4] : acc[j]) + __shfl_xor_sync(0xFFFFFFFFu, give, 16);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float give = h8 ? a4[j] : a4[j + 2];
            a2[j] = (h8 ? a4[j + 2] : a4[j]) + __shfl_xor_sync(0xFFFFFFFFu, give, 8);
        }
        const float give = h4 ? a2[0] : a2[1];
        mine = (h4 ? a2[1] : a2[0]) + __shfl_xor_sync(0xFFFFFFFFu, give, 4);
        mine += __shfl_xor_sync(0xFFFFFFFFu, mine, 2);
        mine += __shfl_xor_sync(0xFFFFFFFFu, mine, 1);
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if ((lane & 3) == 0)  // lane 4 j holds row j's sum
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(leader_addr(smem_u32(&part[rank][8 * warp + lane / 4]))),
                     "f"(mine)
                     : "memory");
    __syncwarp();
    cluster_sync();
    if (rank != 0 || warp != 0) return;
    float g = 0.0f, v = 0.0f, s0, s1;
    for (int c = 0; c < ctas; ++c) {
        g += part[c][lane];
        v += part[c][32 + lane];
    }
    sigmoid2(g, 0.0f, s0, s1);
    const float h = __fmul_rn(__fmul_rn(g, s0), v);
    const int e = mx_exponent_448(__uint_as_float(warp_absmax(h)));
    p.out[t * p.f + col + lane] = (uint8_t)cvt_e4m3x2_rn(__fmul_rn(h, exp2_neg(e)), 0.0f);
    if (lane == 0) p.out_sc[t * (p.f / 32) + col / 32] = (uint8_t)(e + 127);
}

// ====================================================================== host
// Bytes [rows, width] in boxes of box_w (128: with the 128-byte swizzle) x
// box_rows; rows past the end read as zeros.
bool make_map(CUtensorMap *m, const void *base, uint64_t width, uint64_t rows, uint32_t box_w, uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {width, rows}, strides[1] = {width};
    cuuint32_t box[2] = {box_w, box_rows}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, box_w == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              box_w == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void *p) { return aligned(p, 16); }

template <int MODE, int TBN, int CT>
pmn_status launch(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b, const uint8_t *b_scales,
                  const Args &args, cudaStream_t s)
{
    using C = Cfg<MODE, TBN, CT>;
    constexpr bool BWD = MODE == BACKWARD;
    const uint64_t k = (uint64_t)args.k, m = (uint64_t)args.m, n = (uint64_t)args.b_rows;
    CUtensorMap ma, mb, msa, msb;
    if (!make_map(&ma, a, k, m, 128, BM) || !make_map(&mb, b, k, n, 128, BWD ? TBN / CT : TBN / 2) ||
        !make_map(&msa, a_scales, k / 32, m, C::RAW_W, 32) || !make_map(&msb, b_scales, k / 32, n, C::RAW_W, 32))
        return PMN_ERR_CUDA;
    auto kern = gated_kernel<MODE, TBN, CT>;
    static std::atomic<int> sm_count[MAX_DEVICES];  // of each device this kernel has been set up on
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return PMN_ERR_CUDA;
    int sms = dev < MAX_DEVICES ? sm_count[dev].load(std::memory_order_acquire) : 0;
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < CT ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
            return PMN_ERR_CUDA;
        if (dev < MAX_DEVICES) sm_count[dev].store(sms, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms / CT * CT));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CT;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CT > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, ma, mb, msa, msb, args) == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

// The kernel for a few rows: as many CTAs share K as one wave of three CTAs per SM
// allows (one, two, four rows of f 1536: 8 CTAs 4.3, 7.6, 13.4 us; 4 CTAs 5.0, 6.3, 10.9;
// 2 CTAs 5.4, 7.3, 9.6; eight rows: one CTA 20.0, two 21.2, four 23.9).
pmn_status launch_rows(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b, const uint8_t *b_scales,
                       const Args &args, cudaStream_t s)
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PMN_ERR_CUDA;
    unsigned ctas = FEW_CTAS;
    while (ctas > 1 && (args.f / 32 * args.m * ctas > 3 * (int64_t)sms || ctas > args.k / 512)) ctas /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(args.f / 32) * ctas, (unsigned)args.m);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gated_rows_kernel, a, a_scales, b, b_scales, args) == cudaSuccess ? PMN_OK
                                                                                                      : PMN_ERR_CUDA;
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
// collects each translation unit's word: this is where this file's is.
pmn_status pmn_gated_error_word(int **word)
{
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_gated_error) == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
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
    const Args args{offsets, num_experts, total_rows, f, k, (int64_t)num_experts * 2 * f,
                    out, out_scales, out_t, out_t_scales, static_cast<uint16_t *>(y_out), aligned(out, 32),
                    aligned(y_out, 32), out_t && total_rows % 128 == 0 && aligned(out_t_scales, 4),
                    pmn_wait_limit_ns()};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (out_t || y_out) return launch<TRAIN, 192, 2>(a, a_scales, b, b_scales, args, s);
    // Serving.  A few rows, each its own cluster and its own read of the weights, against
    // tiles (f 1536, k 4096, us): one expert, one row 4.3 and 12.2, four 9.5 and 12.0, six
    // 12.4 and 12.2, eight 16.7 and 12.2; 8 experts, 8 rows 19.3 and 26.2, 12 rows 26.4 and
    // 25.1; 24 experts, 8 rows 19.9 and 28.1, 24 rows 45 and 55.
    if (total_rows <= 4 || (total_rows <= 24 && total_rows <= num_experts))
        return launch_rows(a, a_scales, b, b_scales, args, s);
    // 256-row tiles on CTA pairs load less per product, 128-row tiles waste less at
    // the segments' ends.  Paired and single, us: one expert 64 rows 12.2 and 13.0, 16384
    // rows 119 and 141; 8 experts 8192 rows 73.5 and 83.6, 3000 rows 40.4 and 36.7; 24
    // experts 32768 rows 267 and 308, 8192 rows 96.2 and 96.8, 512 rows 61 and 52.5.
    if (num_experts == 1 || total_rows >= 1024 * (int64_t)num_experts)
        return launch<SERVE, 192, 2>(a, a_scales, b, b_scales, args, s);
    return launch<SERVE, 192, 1>(a, a_scales, b, b_scales, args, s);
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
    const Args args{offsets, num_experts, total_rows, f, k, (int64_t)num_experts * f,
                    out, out_scales, out_t, out_t_scales, static_cast<uint16_t *>(const_cast<void *>(y)), aligned(out, 32),
                    aligned(y, 32), total_rows % 128 == 0 && aligned(out_t_scales, 4), pmn_wait_limit_ns()};
    return launch<BACKWARD, 192, 2>(a, a_scales, b, b_scales, args, reinterpret_cast<cudaStream_t>(stream));
}
