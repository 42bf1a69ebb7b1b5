// optim.cu -- pmn_adamw_step: one AdamW step over many tensors, with float32
// or MXFP8 states.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/pmn.h"
#include "numerics.cuh"

using namespace pmn;

namespace {

constexpr int CTA = 256;
constexpr int WARP_ELEMS = 512;                    // 2 groups of 8 elements per thread
constexpr int CHUNK = CTA / 32 * WARP_ELEMS;       // elements of one CTA

// The tensors travel as a kernel argument (no table in device memory that a
// caller would have to keep alive): up to MAXT per launch.
template <int MAXT>
struct Table {
    pmn_adamw_tensor t[MAXT];
    int first[MAXT + 1];  // first chunk (CTA) of each tensor
    int count;
    uint32_t base;        // index of t[0] among the call's tensors
};

struct Hyper {
    float beta1, omb1, beta2, omb2;  // omb: 1 - beta
    float decay;                     // 1 - lr * weight_decay
    float lr1;                       // lr / (1 - beta1^step)
    float rbc2;                      // 1 / sqrt(1 - beta2^step)
    float eps;
    int v_top;                       // v below these bits and |m| up to this: root2 and
    float m_top;                     // quotient2 hold (0 and 0: never)
    uint32_t step;
    uint64_t seed;
    const float *grad_scale;
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Eight consecutive elements of an array of B-byte elements as they lie in memory.
// Loads and decoding are apart, so that all of a thread's loads are in flight
// together; `left` counts the elements from i to the array's end.
template <int B>
struct Raw {
    uint32_t w[2 * B];
    __device__ __forceinline__ void load(const void *p, int64_t i)
    {
        const uint8_t *b = static_cast<const uint8_t *>(p) + i * B;
        if (B == 1) {
            const uint2 q = __ldcs(reinterpret_cast<const uint2 *>(b));
            w[0] = q.x;
            w[1] = q.y;
        } else {
#pragma unroll
            for (int j = 0; j < B / 2; ++j) {
                const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(b) + j);
                w[4 * j] = q.x;
                w[4 * j + 1] = q.y;
                w[4 * j + 2] = q.z;
                w[4 * j + 3] = q.w;
            }
        }
    }
    __device__ __forceinline__ void load_some(const void *p, int64_t i, int64_t left)
    {
#pragma unroll
        for (int j = 0; j < 2 * B; ++j) w[j] = 0u;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < left) {
                if (B == 4) w[k] = static_cast<const uint32_t *>(p)[i + k];
                else if (B == 2) w[k >> 1] |= (uint32_t) static_cast<const uint16_t *>(p)[i + k] << (16 * (k & 1));
                else w[k >> 2] |= (uint32_t) static_cast<const uint8_t *>(p)[i + k] << (8 * (k & 3));
            }
    }
    // float32, bf16, or E4M3 codes times `scale`
    __device__ __forceinline__ void values(float (&v)[8], float scale = 1.0f) const
    {
        if constexpr (B == 4) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
        } else if constexpr (B == 2) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = __uint_as_float(w[k] << 16);
                v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t h2;  // two codes as f16x2 (exact)
                const uint16_t b16 = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(b16));
                mul2(h2_lo_to_f32(h2), h2_hi_to_f32(h2), scale, scale, v[2 * k], v[2 * k + 1]);
            }
        }
    }
};

__device__ __forceinline__ void store8_f32(void *p, int64_t i, int64_t left, const float (&v)[8])
{
    float *o = static_cast<float *>(p) + i;
    if (left >= 8) {
        reinterpret_cast<float4 *>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < left) o[k] = v[k];
    }
}

__device__ __forceinline__ void store8_b16(void *p, int64_t i, int64_t left, const uint32_t (&w)[4])
{
    uint16_t *o = static_cast<uint16_t *>(p) + i;
    if (left >= 8) {
        *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < left) o[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
    }
}

// MXFP8 of the thread's eight values, its block being the 32 values of four
// adjacent lanes, rounded stochastically with the words r0 (values 0..3) and r1
// (4..7).  keep: a nonzero value takes the smallest code instead of 0.
// (A value below the smallest code 2^-9 of its block becomes that code exactly,
// whose rounding is certain; larger ones never round to 0.  Blocks that have such
// a value are rare, so one comparison of the thread's minimum guards the work.)
// An infinite value takes the NaN code and has no part in the block's scale: its
// 31 neighbours would otherwise become 0 or, kept, codes whose squares overflow.
template <bool KEEP>
__device__ __forceinline__ void store8_mx(uint8_t *q, uint8_t *sc, int64_t i, int64_t left, float (&v)[8], uint32_t r0,
                                          uint32_t r1)
{
    float amax = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(v[k]));
    if (__float_as_uint(amax) == 0x7F800000u) {
        amax = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (fabsf(v[k]) > 3.402823466e38f) v[k] = __uint_as_float(0x7FC00000u);
            amax = fmaxf(amax, fabsf(v[k]));
        }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    const int e = mx_exponent_448(amax);
    const float s = exp2_neg(e);
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; k += 2) mul2(v[k], v[k + 1], s, s, y[k], y[k + 1]);
    if (KEEP) {
        float least = y[0];
#pragma unroll
        for (int k = 1; k < 8; ++k) least = fminf(least, y[k]);
        if (least < 0.001953125f) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (y[k] > 0.0f) y[k] = fmaxf(y[k], 0.001953125f);
        }
    }
    const uint32_t w[2] = {cvt_e4m3x4_rs(y[0], y[1], y[2], y[3], r0), cvt_e4m3x4_rs(y[4], y[5], y[6], y[7], r1)};
    if (left >= 8) {
        *reinterpret_cast<uint2 *>(q + i) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < left) q[i + k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
    }
    if (left > 0 && (threadIdx.x & 3) == 0) sc[i / 32] = (uint8_t)(e + 127);
}

// The random words of the thread's two groups of 8 elements, at elements
// i and i + 256 of the tensor.  One Philox call serves 16 elements: the call of
// the even lane covers the first group of a lane pair, the odd lane's the second
// one, and the pair exchanges the halves (words 0, 1 go to the even lane).
__device__ __forceinline__ void pair_words(uint64_t seed, uint32_t tag, uint32_t step, int64_t i, uint32_t (&r)[2][2])
{
    const bool odd = threadIdx.x & 1;
    const uint64_t j = (uint64_t)(odd ? i + 256 : i) >> 4;
    const uint4 c = philox4x32_10(make_uint4((uint32_t)j, (uint32_t)(j >> 32), tag, step), (uint32_t)seed,
                                  (uint32_t)(seed >> 32));
    const uint32_t a = __shfl_xor_sync(0xFFFFFFFFu, odd ? c.x : c.z, 1);
    const uint32_t b = __shfl_xor_sync(0xFFFFFFFFu, odd ? c.y : c.w, 1);
    r[0][0] = odd ? a : c.x;
    r[0][1] = odd ? b : c.y;
    r[1][0] = odd ? c.z : a;
    r[1][1] = odd ? c.w : b;
}

// The 16 random bits of element k (0..3) of a word, as the hardware's
// stochastic conversion takes them: low half, low half reversed, high half,
// high half reversed.
__device__ __forceinline__ uint32_t bits16(uint32_t w, int k)
{
    if (k == 0) return w & 0xFFFFu;
    if (k == 1) return __brev(w) >> 16;
    if (k == 2) return w >> 16;
    return __brev(w) & 0xFFFFu;
}

// a * b + c on two lanes, each rounded once.
__device__ __forceinline__ void fma2v(float a0, float a1, float b0, float b1, float c0, float c1, float &r0, float &r1)
{
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r0), "=f"(r1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ float rsqrt_approx(float x)
{
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Square roots and quotients of two pairs from the hardware's approximations and one
// step of Newton's method on the residual, which a fused multiply-add gives (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990):
// x - r^2 and n - q d are exact up to one rounding of a small number, so the results
// are within one place of the correctly rounded values (3 2^-24 for a subnormal n).
// x is 0 or a normal number (the root of 0 comes out as 0); d is normal and below
// 2^126, so that its reciprocal is normal too; n is finite and n / d does not overflow.
__device__ __forceinline__ void root2(float x0, float x1, float &r0, float &r1)
{
    const float least = 1.17549435e-38f;
    const float y0 = rsqrt_approx(fmaxf(x0, least)), y1 = rsqrt_approx(fmaxf(x1, least));
    float a0, a1, e0, e1, h0, h1;
    mul2(x0, x1, y0, y1, a0, a1);
    fma2v(-a0, -a1, a0, a1, x0, x1, e0, e1);
    mul2(y0, y1, 0.5f, 0.5f, h0, h1);
    fma2v(e0, e1, h0, h1, a0, a1, r0, r1);
}

__device__ __forceinline__ void quotient2(float n0, float n1, float d0, float d1, float &q0, float &q1)
{
    const float y0 = rcp_approx(d0), y1 = rcp_approx(d1);
    float a0, a1, e0, e1;
    mul2(n0, n1, y0, y1, a0, a1);
    fma2v(-a0, -a1, d0, d1, n0, n1, e0, e1);
    fma2v(e0, e1, y0, y1, a0, a1, q0, q1);
}

// One AdamW step.  Memory-bound: each value is read and written once, 16 elements
// a thread in two groups of 8 so that both groups' loads are in flight together.
//   g = grad_scale grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// MXFP8 states hold m and sqrt(v): the root halves the range of exponents that
// one block's scale has to serve.  Both are rounded stochastically: a step moves
// v by about 1 - b2 of itself, far less than half a step of E4M3, and rounding to
// nearest would never move it.  p is updated from the unrounded m and v.
// Measured on one GB300, 75.5 million elements in eight tensors: float32 parameters and
// states 331 us, 6.8 TB/s, all that HBM gives; bf16 parameters and MXFP8 states 163 us,
// 4.7 TB/s (113 us at HBM's rate): bound by issue, 63 instructions per element with the
// issue slots 75 % busy (one of them, and 2 us, is the largest |m|).  With two groups a thread a pair of lanes shares two Philox
// calls per state, and no random word is thrown away.
template <bool PF32, bool GF32, bool MX, int MAXT>
__global__ void __launch_bounds__(CTA, MX ? 4 : 3) adamw_kernel(const __grid_constant__ Table<MAXT> tab, const Hyper h)
{
    // With float32 parameters and MXFP8 states the products and sums of m and v are rounded
    // one by one: the same states, code for code, as from the formulas in plain float32.  A
    // fused sum differs in its last place, which turns a stochastic rounding now and then (7
    // of 10^5 codes of m), and the next step moves the parameter by a few per cent more or
    // less.  (Parameters in bf16 are rounded themselves, by far more than that, and their
    // kernel is bound by issue: fused, 165 us for 75 million elements; one by one 168.)
    constexpr bool APART = PF32 && MX;
    int lo = 0, hi = tab.count - 1;
    while (lo < hi) {  // the last tensor whose first chunk is at or before this one
        const int mid = (lo + hi + 1) >> 1;
        if (tab.first[mid] <= (int)blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const pmn_adamw_tensor &t = tab.t[lo];
    const int64_t n = t.n;
    const int64_t i0 = (int64_t)((int)blockIdx.x - tab.first[lo]) * CHUNK + (threadIdx.x >> 5) * WARP_ELEMS +
                       8 * (threadIdx.x & 31);
    const uint32_t tag = 4u * (tab.base + (uint32_t)lo);
    Raw<PF32 ? 4 : 2> rp[2];
    Raw<GF32 ? 4 : 2> rg[2];
    Raw<MX ? 1 : 4> rm[2], rv[2];
    uint32_t ms[2] = {0u, 0u}, vs[2] = {0u, 0u};
    if (i0 - 8 * (threadIdx.x & 31) + WARP_ELEMS <= n) {  // the whole warp's elements lie inside
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t i = i0 + 256 * u;
            rp[u].load(t.param, i);
            rg[u].load(t.grad, i);
            rm[u].load(t.m, i);
            rv[u].load(t.v, i);
            if (MX) {
                ms[u] = t.m_scales[i / 32];
                vs[u] = t.v_scales[i / 32];
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t i = i0 + 256 * u, left = n - i;
            rp[u].load_some(t.param, i, left);
            rg[u].load_some(t.grad, i, left);
            rm[u].load_some(t.m, i, left);
            rv[u].load_some(t.v, i, left);
            if (MX && left > 0) {
                ms[u] = t.m_scales[i / 32];
                vs[u] = t.v_scales[i / 32];
            }
        }
    }
    const float gs = h.grad_scale ? __ldg(h.grad_scale) : 1.0f;
    float p[2][8], g[2][8], m[2][8], v[2][8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        rp[u].values(p[u]);
        rg[u].values(g[u]);
        const float m_scale = MX ? e8m0_to_f32(ms[u]) : 1.0f;
        rm[u].values(m[u], APART ? __fmul_rn(m_scale, h.beta1) : m_scale);  // APART: beta1 m, rounded once
        rv[u].values(v[u], MX ? e8m0_to_f32(vs[u]) : 1.0f);
        int top = 0;                    // largest v's bits: infinity
        uint32_t odd = 0xFFFFFFFFu;     // smallest v's bits - 1, 0 not counted: subnormal
        float m_max = 0.0f;             // largest |m|
#pragma unroll
        for (int k = 0; k < 8; k += 2) {  // two elements at a time
            float g0, g1, t0, t1, s0, s1;
            mul2(g[u][k], g[u][k + 1], gs, gs, g0, g1);
            mul2(g0, g1, h.omb1, h.omb1, t0, t1);
            if (APART) {
                m[u][k] = __fadd_rn(m[u][k], t0);
                m[u][k + 1] = __fadd_rn(m[u][k + 1], t1);
            } else {
                fma2v(h.beta1, h.beta1, m[u][k], m[u][k + 1], t0, t1, m[u][k], m[u][k + 1]);
            }
            m_max = fmaxf(fmaxf(m_max, fabsf(m[u][k])), fabsf(m[u][k + 1]));
            if (MX) mul2(v[u][k], v[u][k + 1], v[u][k], v[u][k + 1], v[u][k], v[u][k + 1]);
            mul2(g0, g1, g0, g1, t0, t1);
            mul2(t0, t1, h.omb2, h.omb2, t0, t1);
            if (APART) {
                mul2(v[u][k], v[u][k + 1], h.beta2, h.beta2, s0, s1);
                v[u][k] = __fadd_rn(s0, t0);
                v[u][k + 1] = __fadd_rn(s1, t1);
            } else {
                fma2v(h.beta2, h.beta2, v[u][k], v[u][k + 1], t0, t1, v[u][k], v[u][k + 1]);
            }
            top = max(max(top, __float_as_int(v[u][k])), __float_as_int(v[u][k + 1]));
            odd = min(min(odd, __float_as_uint(v[u][k]) - 1u), __float_as_uint(v[u][k + 1]) - 1u);
        }
        // every v is 0 or normal, and no quotient leaves the range
        const bool plain = top < h.v_top && odd >= 0x007FFFFFu && m_max <= h.m_top;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            float r0, r1, d0, d1, t0, t1;
            if (plain) {
                root2(v[u][k], v[u][k + 1], r0, r1);
            } else {
                r0 = __fsqrt_rn(v[u][k]);
                r1 = __fsqrt_rn(v[u][k + 1]);
            }
            fma2v(r0, r1, h.rbc2, h.rbc2, h.eps, h.eps, d0, d1);
            if (plain) {
                quotient2(m[u][k], m[u][k + 1], d0, d1, d0, d1);
            } else {
                d0 = __fdiv_rn(m[u][k], d0);
                d1 = __fdiv_rn(m[u][k + 1], d1);
            }
            mul2(p[u][k], p[u][k + 1], h.decay, h.decay, t0, t1);
            fma2v(-h.lr1, -h.lr1, d0, d1, t0, t1, p[u][k], p[u][k + 1]);
            if (MX) v[u][k] = r0, v[u][k + 1] = r1;
        }
    }
    uint32_t r[2][2];
    if (!PF32) pair_words(h.seed, tag, h.step, i0, r);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int64_t i = i0 + 256 * u, left = n - i;
        uint32_t w[4];
        if (PF32) {
            store8_f32(t.param, i, left, p[u]);
            if (t.copy) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(p[u][2 * k], p[u][2 * k + 1]);
                    w[k] = *reinterpret_cast<const uint32_t *>(&b);
                }
                store8_b16(t.copy, i, left, w);
            }
        } else {
            // bf16 without a master: the step is often below half a place, so the
            // rounding is stochastic (16 bits added below the last place)
            uint32_t b[8];
            float any = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                b[k] = __float_as_uint(p[u][k]) + bits16(r[u][k >> 2], k & 3);
                any += p[u][k];
            }
            if (any != any) {  // the addition may carry a NaN's bits into the sign
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (p[u][k] != p[u][k]) b[k] = 0x7FC00000u;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __byte_perm(b[2 * k], b[2 * k + 1], 0x7632);
            store8_b16(t.param, i, left, w);
        }
        if (!MX) {
            store8_f32(t.m, i, left, m[u]);
            store8_f32(t.v, i, left, v[u]);
        }
    }
    if (MX) {
        pair_words(h.seed, tag + 1u, h.step, i0, r);
#pragma unroll
        for (int u = 0; u < 2; ++u)
            store8_mx<false>(static_cast<uint8_t *>(t.m), t.m_scales, i0 + 256 * u, n - i0 - 256 * u, m[u], r[u][0],
                             r[u][1]);
        pair_words(h.seed, tag + 2u, h.step, i0, r);
#pragma unroll
        for (int u = 0; u < 2; ++u)
            store8_mx<true>(static_cast<uint8_t *>(t.v), t.v_scales, i0 + 256 * u, n - i0 - 256 * u, v[u], r[u][0],
                            r[u][1]);
    }
}

int64_t chunks_of(int64_t n) { return n / CHUNK + (n % CHUNK != 0); }

template <int MAXT>
pmn_status launch_adamw(const pmn_adamw_tensor *t, int count, uint32_t base, int kinds, const Hyper &h, cudaStream_t s)
{
    static thread_local Table<MAXT> tab;
    int64_t chunks = 0;
    for (int i = 0; i < count; ++i) {
        tab.t[i] = t[i];
        tab.first[i] = (int)chunks;
        chunks += chunks_of(t[i].n);
    }
    tab.first[count] = (int)chunks;
    tab.count = count;
    tab.base = base;
    if (chunks == 0) return PMN_OK;
    const unsigned grid = (unsigned)chunks;
#define PMN_ADAMW(P, G, M) adamw_kernel<P, G, M, MAXT><<<grid, CTA, 0, s>>>(tab, h)
    switch (kinds) {
        case 0: PMN_ADAMW(false, false, false); break;
        case 1: PMN_ADAMW(true, false, false); break;
        case 2: PMN_ADAMW(false, true, false); break;
        case 3: PMN_ADAMW(true, true, false); break;
        case 4: PMN_ADAMW(false, false, true); break;
        case 5: PMN_ADAMW(true, false, true); break;
        case 6: PMN_ADAMW(false, true, true); break;
        default: PMN_ADAMW(true, true, true); break;
    }
#undef PMN_ADAMW
    return cudaGetLastError() == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

constexpr int SMALL_TABLE = 48, LARGE_TABLE = 440;  // 3.3 KB and 30 KB of kernel arguments (limit 32 764 bytes)

}  // namespace

extern "C" pmn_status pmn_adamw_step(const pmn_adamw_tensor *tensors, int num_tensors, int param_kind, int grad_kind,
                                     int state_kind, double lr, double beta1, double beta2, double eps,
                                     double weight_decay, int64_t step, const float *grad_scale, uint64_t seed,
                                     void *stream)
{
    if (num_tensors < 0 || num_tensors > (1 << 28) || (num_tensors > 0 && !tensors)) return PMN_ERR_INVALID_ARG;
    const auto two = [](int k) { return k == PMN_OUT_BF16 || k == PMN_OUT_F32; };
    if (!two(param_kind) || !two(grad_kind) || (state_kind != PMN_STATE_F32 && state_kind != PMN_STATE_MXFP8))
        return PMN_ERR_INVALID_ARG;
    // NaN fails every comparison
    if (!(std::isfinite(lr) && beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0 && eps > 0.0 &&
          std::isfinite(weight_decay)) || !std::isfinite((float)eps) || (float)eps < 1.17549435e-38f || step < 1 ||
        ((uintptr_t)grad_scale & 3u))
        return PMN_ERR_INVALID_ARG;
    int64_t chunks = 0;  // of a launch
    for (int i = 0; i < num_tensors; ++i) {
        const pmn_adamw_tensor &t = tensors[i];
        if (i % LARGE_TABLE == 0) chunks = 0;
        if (t.n < 0 || (t.copy && param_kind != PMN_OUT_F32)) return PMN_ERR_INVALID_ARG;
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v) return PMN_ERR_INVALID_ARG;
        if (!aligned16(t.param) || !aligned16(t.copy) || !aligned16(t.grad) || !aligned16(t.m) || !aligned16(t.v))
            return PMN_ERR_INVALID_ARG;
        if (state_kind == PMN_STATE_MXFP8 && (!t.m_scales || !t.v_scales)) return PMN_ERR_INVALID_ARG;
        // before the first launch: a refused step has updated nothing
        if ((chunks += chunks_of(t.n)) >= (int64_t(1) << 31)) return PMN_ERR_UNSUPPORTED;
    }
    Hyper h;
    h.beta1 = (float)beta1;
    h.omb1 = (float)(1.0 - beta1);
    h.beta2 = (float)beta2;
    h.omb2 = (float)(1.0 - beta2);
    h.decay = (float)(1.0 - lr * weight_decay);
    h.lr1 = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
    h.rbc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
    h.eps = (float)eps;
    // the denominator is at least eps, and at most eps + 2^91 (v's root is below 2^64, rbc2
    // below 2^27: beta2 is at most 1 - 2^-53)
    const bool usual = h.eps <= 0x1p100f;
    h.v_top = usual ? 0x7F800000 : 0;
    h.m_top = usual ? (float)std::fmin(3.402823466e38, (double)h.eps * 0x1p126) : 0.0f;
    h.step = (uint32_t)step;
    h.seed = seed;
    h.grad_scale = grad_scale;
    const int kinds = (param_kind == PMN_OUT_F32 ? 1 : 0) | (grad_kind == PMN_OUT_F32 ? 2 : 0) |
                      (state_kind == PMN_STATE_MXFP8 ? 4 : 0);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (int at = 0; at < num_tensors; at += LARGE_TABLE) {
        const int count = num_tensors - at < LARGE_TABLE ? num_tensors - at : LARGE_TABLE;
        const pmn_status st = count <= SMALL_TABLE ? launch_adamw<SMALL_TABLE>(tensors + at, count, at, kinds, h, s)
                                                   : launch_adamw<LARGE_TABLE>(tensors + at, count, at, kinds, h, s);
        if (st != PMN_OK) return st;
    }
    return PMN_OK;
}
