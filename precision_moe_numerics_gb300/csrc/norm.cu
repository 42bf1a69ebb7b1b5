// norm.cu -- the residual stream's side of the MXFP8 layers:
//   pmn_add_rmsnorm_mxfp8     residual addition, root-mean-square norm, MXFP8 rows
//   pmn_add_rmsnorm_backward  its gradients (row gradients and the weight's)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/pmn.h"
#include "numerics.cuh"

using namespace pmn;

namespace {

constexpr int RES_NONE = 0, RES_BF16 = 1, RES_F32 = 2;
constexpr int CTA = 256;
constexpr int WARP_COLS = 1024;     // rows up to here: one warp each; longer ones: one CTA each
constexpr int BWD_WARP_COLS = 512;  // the same in the backward pass, which holds more per column
constexpr int MAX_COLS = 16384;

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

__device__ __forceinline__ void unpack8(const uint4 &q, float (&v)[8])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t w = u4_word(q, k);
        v[2 * k] = __uint_as_float(w << 16);
        v[2 * k + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight consecutive values of a row in the residual's type.
template <int RK>
struct Piece {
    uint4 a, b;  // bf16: a; f32: a, b
    __device__ __forceinline__ void load(const void *p, int64_t i)
    {
        if (RK == RES_F32) {
            const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i);
            a = __ldcs(q);
            b = __ldcs(q + 1);
        } else {
            a = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i));
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        if (RK == RES_F32) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = __uint_as_float(u4_word(a, k));
                v[4 + k] = __uint_as_float(u4_word(b, k));
            }
        } else {
            unpack8(a, v);
        }
    }
    __device__ __forceinline__ static void store(void *p, int64_t i, const float (&v)[8])
    {
        if (RK == RES_F32) {
            float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = pack8(v);
        }
    }
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the threads of one row: a warp (T = 32) or the whole CTA (one
// barrier; `slot` alternates between calls so that a slot's readers are done
// before its next writer: a barrier of the other slot lies between them).
template <int T>
__device__ __forceinline__ float row_sum(float v, float (*red)[T / 32], int slot)
{
    v = warp_sum(v);
    if (T == 32) return v;
    if ((threadIdx.x & 31) == 0) red[slot][threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) s += red[slot][w];
    return s;
}

// r = round(x + residual), rstd = 1 / sqrt(mean r^2 + eps), y = r rstd w, MXFP8
// of y.  Memory-bound: every value is read and written once, so a row stays in
// its threads' registers between the two uses.  A thread holds 8 consecutive
// columns (16 bytes of bf16) per piece; four adjacent lanes hold one 32-column
// block and take its maximum with two shuffles.
// Measured on one GB300: 16384 x 4096 in bf16 with y written, 89 us, 6.85 TB/s, all
// that HBM gives, in float32 127 us, 6.9 TB/s; one row 1.8 us, the latency of a launch
// and two dependent steps.
template <int T, int NP, int RK>
__global__ void __launch_bounds__(CTA) add_rmsnorm_kernel(const uint16_t *__restrict__ x, int64_t ldx,
                                                          const void *res, int64_t ldr,
                                                          const uint16_t *__restrict__ weight, int64_t rows, int cols,
                                                          float eps, void *res_out,
                                                          uint8_t *__restrict__ out, uint8_t *__restrict__ out_sc,
                                                          uint16_t *__restrict__ y_out, float *__restrict__ rstd_out)
{
    __shared__ float red[2][T / 32];
    const int t = threadIdx.x & (T - 1);
    const int64_t row = T == 32 ? (int64_t)blockIdx.x * (CTA / 32) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    if (T == 32 && row >= rows) return;  // whole warps
    uint4 xv[NP], wv[NP];
    Piece<RK> rv[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = 8 * (t + T * i);
        if (c < cols) {
            xv[i] = __ldcs(reinterpret_cast<const uint4 *>(x + row * ldx + c));
            if (RK != RES_NONE) rv[i].load(res, row * ldr + c);
        }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = 8 * (t + T * i);
        if (c < cols) wv[i] = __ldg(reinterpret_cast<const uint4 *>(weight + c));
    }
    float v[NP][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = 8 * (t + T * i);
        if (c < cols) {
            unpack8(xv[i], v[i]);
            if (RK != RES_NONE) {
                float r8[8];
                rv[i].values(r8);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[i][k] = __fadd_rn(v[i][k], r8[k]);
                // the stream is carried in its own type, and the norm reads what is
                // carried, so the backward pass can start from the stored r
                if (RK == RES_BF16) {
                    const uint4 q = pack8(v[i]);
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(res_out) + row * cols + c) = q;
                    unpack8(q, v[i]);
                } else {
                    Piece<RK>::store(res_out, row * cols + c, v[i]);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(v[i][k], v[i][k], ss);
        }
    }
    ss = row_sum<T>(ss, red, 0);
    const float rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)cols), eps)));
    if (rstd_out && t == 0) rstd_out[row] = rstd;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = 8 * (t + T * i);
        const bool on = c < cols;  // alike in the four lanes of a block (cols % 32 == 0)
        float w8[8], y[8];
        unpack8(on ? wv[i] : make_uint4(0u, 0u, 0u, 0u), w8);
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            y[k] = on ? __fmul_rn(__fmul_rn(v[i][k], rstd), w8[k]) : 0.0f;
            amax = fmaxf(amax, fabsf(y[k]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        if (!on) continue;
        const int e = mx_exponent_448(amax);
        const float sc = exp2_neg(e);
        uint32_t q[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            q[k] = cvt_e4m3x2_rn(__fmul_rn(y[4 * k], sc), __fmul_rn(y[4 * k + 1], sc)) |
                   (cvt_e4m3x2_rn(__fmul_rn(y[4 * k + 2], sc), __fmul_rn(y[4 * k + 3], sc)) << 16);
        *reinterpret_cast<uint2 *>(out + row * cols + c) = make_uint2(q[0], q[1]);
        if ((threadIdx.x & 3) == 0) out_sc[row * (cols / 32) + c / 32] = (uint8_t)(e + 127);
        if (y_out) *reinterpret_cast<uint4 *>(y_out + row * cols + c) = pack8(y);
    }
}

// Gradients of y = r rstd w.  With xh = r rstd, g = dy w, c = mean(g xh):
//   dr = rstd (g - xh c) + dres,   dw = sum over rows of dy xh.
// Memory-bound: dy, r and dres are read once and dr is written once.  The
// threads walk the rows with the grid's stride; each keeps the dw sums of its
// own columns in registers and writes them once, and a second kernel adds the
// CTAs' partial sums in a fixed order (no atomics: the same bits every run).
// dr may be dres, and in the forward res_out the residual: none of these is __restrict__,
// and a thread reads its own columns of a row before it writes them.
// AHEAD: the next row's loads are on their way while this one is reduced and
// written; rows of more than 8192 columns have no registers for that.
// Measured on one GB300: 16384 x 4096 in bf16 92.6 us, 5.8 TB/s (79 us at HBM's rate:
// one wave of CTAs has fewer loads in flight than a copy, and the partial sums are 5 MB
// and a second kernel); 1021 x 1536 in float32 7.0 us (3.7), latency of the two
// launches.  16384 rows between the thread counts' steps, where threads hold nothing:
// 1056 columns 38 us, 3.7 TB/s (132 of 256 threads at work), 2560 72 us, 4.7 TB/s, 5120
// 140 us, 4.8 TB/s (62 %).  Spills: float32 rows of 257 to 512, 2049 to 4096 and 4097 to
// 8192 columns 88, 36 and 36 bytes (5.0, 6.1, 6.2 TB/s), more than 8192 columns 508
// (bf16) and 936 (2.9 and 2.6 TB/s).
template <int T, int NP, int RK, int PER_SM>
__global__ void __launch_bounds__(T == 32 ? CTA : T, PER_SM) add_rmsnorm_backward_kernel(
    const uint16_t *__restrict__ dy, const void *__restrict__ r, const float *__restrict__ rstd,
    const uint16_t *__restrict__ weight, const void *dres, int64_t rows, int cols, void *dr,
    uint16_t *__restrict__ dx, float *__restrict__ partial)
{
    __shared__ float red[2][T / 32];
    constexpr int RPC = T == 32 ? CTA / T : 1;  // rows of a CTA at a time
    constexpr bool AHEAD = T * NP <= 1024;
    const int t = threadIdx.x & (T - 1);
    uint4 wv[NP];
    float acc[NP][8];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = 8 * (t + T * i);
        wv[i] = make_uint4(0u, 0u, 0u, 0u);
        if (c < cols) wv[i] = __ldg(reinterpret_cast<const uint4 *>(weight + c));
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[i][k] = 0.0f;
    }
    int slot = 0;
    uint4 dv[NP];
    Piece<RK> rv[NP], sv[NP];
    float rs = 0.0f;
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = 8 * (t + T * i);
            if (c < cols) {
                dv[i] = __ldcs(reinterpret_cast<const uint4 *>(dy + row * cols + c));
                rv[i].load(r, row * cols + c);
                if (dres) sv[i].load(dres, row * cols + c);
            }
        }
        rs = __ldg(rstd + row);
    };
    const int64_t step = (int64_t)gridDim.x * RPC;
    int64_t row = (int64_t)blockIdx.x * RPC + (T == 32 ? threadIdx.x >> 5 : 0);
    if (AHEAD && row < rows) load(row);
    for (; row < rows; row += step, slot ^= 1) {
        if (!AHEAD) load(row);
        // g = dy w and xh = r rstd take the loads' place
        float g[NP][8], xh[NP][8], s8[NP][8];
        const float rstd_row = rs;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if (8 * (t + T * i) < cols) {
                float d8[8], w8[8];
                unpack8(dv[i], d8);
                rv[i].values(xh[i]);
                unpack8(wv[i], w8);
                if (dres) sv[i].values(s8[i]);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    xh[i][k] = __fmul_rn(xh[i][k], rstd_row);
                    g[i][k] = __fmul_rn(d8[k], w8[k]);
                    acc[i][k] = fmaf(d8[k], xh[i][k], acc[i][k]);
                    s = fmaf(g[i][k], xh[i][k], s);
                }
            }
        }
        if (AHEAD && row + step < rows) load(row + step);
        const float c1 = __fdiv_rn(row_sum<T>(s, red, slot), (float)cols);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = 8 * (t + T * i);
            if (c < cols) {
                float o[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    o[k] = __fmul_rn(rstd_row, fmaf(-xh[i][k], c1, g[i][k]));
                    if (dres) o[k] = __fadd_rn(o[k], s8[i][k]);
                }
                Piece<RK>::store(dr, row * cols + c, o);
                if (dx) *reinterpret_cast<uint4 *>(dx + row * cols + c) = pack8(o);
            }
        }
    }
    if constexpr (T == 32) {
        // the CTA's eight warps hold sums of the same columns
        __shared__ float sums[CTA / 32][BWD_WARP_COLS];
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = 8 * (t + T * i) + k;
                if (c < cols) sums[threadIdx.x >> 5][c] = acc[i][k];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += CTA) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < CTA / 32; ++w) v += sums[w][c];
            partial[(int64_t)blockIdx.x * cols + c] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = 8 * (t + T * i);
            if (c < cols) {
                float4 *p = reinterpret_cast<float4 *>(partial + (int64_t)blockIdx.x * cols + c);
                p[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                p[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
            }
        }
    }
}

// dw[c] = sum of the CTAs' partial sums: 32 columns per CTA, each of its 32 warps
// takes every 32nd partial row, then the warps' sums are added in order.
constexpr int DW_WARPS = 32;
__global__ void __launch_bounds__(32 * DW_WARPS) add_rmsnorm_dw_kernel(const float *__restrict__ partial, int parts,
                                                                       int cols, float *__restrict__ dw)
{
    __shared__ float sums[DW_WARPS][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // cols % 32 == 0
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the backward kernel still runs
    float v = 0.0f;
#pragma unroll 8
    for (int p = w; p < parts; p += DW_WARPS) v += partial[(int64_t)p * cols + c];
    sums[w][lane] = v;
    __syncthreads();
    if (w == 0) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < DW_WARPS; ++k) s += sums[k][lane];
        dw[c] = s;
    }
}

// CTAs of the backward kernel per SM: as many as the SMs hold at once.  More are slower:
// they run in turn, and each adds a row of partial sums (16384 x 4096: 304 CTAs 93 us,
// 456 110 us, 608 97 us; 304 of 512 threads, half of them waiting, 111 us).  With one
// piece per thread and many rows, half as many again at 80 registers keep more loads in
// flight (16384 x 1056 47 -> 37 us, x 2048 56 -> 49); few rows are better off with fewer
// partial sums and uneven shares (1021 x 1536 in float32 7.0 us, 8.4 with 456 CTAs).
bool many_rows(int64_t rows) { return rows >= 4096; }
int backward_per_sm(int64_t rows, int64_t cols)
{
    if (cols > 4096) return 1;                             // 512 threads
    if (cols > 2048 || cols <= BWD_WARP_COLS) return 2;    // 256 threads
    if (cols > 1024) return many_rows(rows) ? 3 : 2;       // 256 threads
    return many_rows(rows) ? 6 : 4;                        // 128 threads
}

// CTAs in all: rows of partial sums.  From constants, so that the workspace's size and
// the sums' order depend on the sizes alone.
int64_t backward_parts(int64_t rows, int64_t cols)
{
    const int64_t per = cols <= BWD_WARP_COLS ? CTA / 32 : 1;
    return std::min<int64_t>(152 * backward_per_sm(rows, cols), (rows + per - 1) / per);
}

struct NormArgs {
    const uint16_t *x;
    int64_t ldx;
    const void *res;
    int64_t ldr;
    const uint16_t *weight;
    int64_t rows;
    int cols;
    float eps;
    void *res_out;
    uint8_t *out, *out_sc;
    uint16_t *y;
    float *rstd;
};

template <int T, int NP>
void launch_norm(int rk, const NormArgs &a, cudaStream_t s)
{
    const unsigned grid = (unsigned)(T == 32 ? (a.rows + CTA / 32 - 1) / (CTA / 32) : a.rows);
#define PMN_NORM(RK)                                                                                                  \
    add_rmsnorm_kernel<T, NP, RK><<<grid, CTA, 0, s>>>(a.x, a.ldx, a.res, a.ldr, a.weight, a.rows, a.cols, a.eps,     \
                                                       a.res_out, a.out, a.out_sc, a.y, a.rstd)
    if (rk == RES_NONE) PMN_NORM(RES_NONE);
    else if (rk == RES_BF16) PMN_NORM(RES_BF16);
    else PMN_NORM(RES_F32);
#undef PMN_NORM
}

struct NormBwdArgs {
    const uint16_t *dy;
    const void *r;
    const float *rstd;
    const uint16_t *weight;
    const void *dres;
    int64_t rows;
    int cols;
    void *dr;
    uint16_t *dx;
    float *partial;
};

template <int T, int NP, int PER_SM>
void launch_norm_bwd(int rk, int parts, const NormBwdArgs &a, cudaStream_t s)
{
#define PMN_NORM_BWD(RK)                                                                                              \
    add_rmsnorm_backward_kernel<T, NP, RK, PER_SM><<<parts, T == 32 ? CTA : T, 0, s>>>(                               \
        a.dy, a.r, a.rstd, a.weight, a.dres, a.rows, a.cols, a.dr, a.dx, a.partial)
    if (rk == RES_BF16) PMN_NORM_BWD(RES_BF16);
    else PMN_NORM_BWD(RES_F32);
#undef PMN_NORM_BWD
}

// Pieces of 8 columns per thread, rounded up to a compiled count.
#define PMN_BY_COLS(cols, CALL)                           \
    do {                                                  \
        if ((cols) <= 256) CALL(32, 1);                   \
        else if ((cols) <= 512) CALL(32, 2);              \
        else if ((cols) <= WARP_COLS) CALL(32, 4);        \
        else if ((cols) <= 2048) CALL(256, 1);            \
        else if ((cols) <= 4096) CALL(256, 2);            \
        else if ((cols) <= 8192) CALL(256, 4);            \
        else CALL(256, 8);                                \
    } while (0)

bool good_sizes(int64_t rows, int64_t cols)
{
    return rows >= 0 && rows < (int64_t(1) << 31) && cols > 0 && cols <= MAX_COLS && cols % 32 == 0;
}

int res_kind(int kind)
{
    return kind == PMN_OUT_BF16 ? RES_BF16 : kind == PMN_OUT_F32 ? RES_F32 : -1;
}

}  // namespace

extern "C" pmn_status pmn_add_rmsnorm_mxfp8(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                                            int residual_kind, const void *weight, int64_t rows, int64_t cols, float eps,
                                            void *res_out, uint8_t *out, uint8_t *out_scales, void *y_out, float *rstd,
                                            void *stream)
{
    if (!good_sizes(rows, cols) || !(eps > 0.0f) || ldx < cols || ldx % 8 != 0) return PMN_ERR_INVALID_ARG;
    const int rk = residual ? res_kind(residual_kind) : RES_NONE;
    if (rk < 0 || (residual != nullptr) != (res_out != nullptr)) return PMN_ERR_INVALID_ARG;
    if (residual && (ldr < cols || ldr % (rk == RES_F32 ? 4 : 8) != 0)) return PMN_ERR_INVALID_ARG;
    if (rows == 0) return PMN_OK;
    if (!x || !weight || !out || !out_scales) return PMN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(res_out) || !aligned16(out) ||
        !aligned16(y_out) || ((uintptr_t)rstd & 3u))
        return PMN_ERR_INVALID_ARG;
    const NormArgs a{static_cast<const uint16_t *>(x), ldx, residual, ldr, static_cast<const uint16_t *>(weight), rows,
                     (int)cols, eps, res_out, out, out_scales, static_cast<uint16_t *>(y_out), rstd};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define PMN_CALL(T, NP) launch_norm<T, NP>(rk, a, s)
    PMN_BY_COLS(cols, PMN_CALL);
#undef PMN_CALL
    return cudaGetLastError() == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

extern "C" int64_t pmn_add_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols)
{
    if (!good_sizes(rows, cols)) return -1;
    return backward_parts(rows, cols) * cols * 4;
}

extern "C" pmn_status pmn_add_rmsnorm_backward(const void *dy, const void *r, int residual_kind, const float *rstd,
                                               const void *weight, const void *dres, int64_t rows, int64_t cols,
                                               void *dr, void *dx, float *dw, void *workspace, int64_t workspace_bytes,
                                               void *stream)
{
    const int rk = res_kind(residual_kind);
    if (!good_sizes(rows, cols) || rk < 0 || !dw || ((uintptr_t)dw & 3u)) return PMN_ERR_INVALID_ARG;
    if (dx && rk != RES_F32) return PMN_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0)  // the sum over no rows
        return cudaMemsetAsync(dw, 0, (size_t)cols * 4, s) == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
    const int parts = (int)backward_parts(rows, cols);
    if (!dy || !r || !rstd || !weight || !dr || !workspace || workspace_bytes < (int64_t)parts * cols * 4)
        return PMN_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(r) || !aligned16(weight) || !aligned16(dres) || !aligned16(dr) || !aligned16(dx) ||
        !aligned16(workspace) || ((uintptr_t)rstd & 3u))
        return PMN_ERR_INVALID_ARG;
    float *partial = static_cast<float *>(workspace);
    const NormBwdArgs a{static_cast<const uint16_t *>(dy), r, rstd, static_cast<const uint16_t *>(weight), dres, rows,
                        (int)cols, dr, static_cast<uint16_t *>(dx), partial};
    const bool many = many_rows(rows);
    if (cols <= 256) launch_norm_bwd<32, 1, 2>(rk, parts, a, s);
    else if (cols <= BWD_WARP_COLS) launch_norm_bwd<32, 2, 2>(rk, parts, a, s);
    else if (cols <= 1024 && many) launch_norm_bwd<128, 1, 6>(rk, parts, a, s);
    else if (cols <= 1024) launch_norm_bwd<128, 1, 4>(rk, parts, a, s);
    else if (cols <= 2048 && many) launch_norm_bwd<256, 1, 3>(rk, parts, a, s);
    else if (cols <= 2048) launch_norm_bwd<256, 1, 2>(rk, parts, a, s);
    else if (cols <= 4096) launch_norm_bwd<256, 2, 2>(rk, parts, a, s);
    else if (cols <= 8192) launch_norm_bwd<512, 2, 1>(rk, parts, a, s);
    else launch_norm_bwd<512, 4, 1>(rk, parts, a, s);
    if (cudaGetLastError() != cudaSuccess) return PMN_ERR_CUDA;
    // the second kernel's launch overlaps the first one's end; it waits for its writes
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(cols / 32));
    cfg.blockDim = dim3(32 * DW_WARPS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, add_rmsnorm_dw_kernel, (const float *)partial, parts, (int)cols, dw) == cudaSuccess
               ? PMN_OK : PMN_ERR_CUDA;
}
