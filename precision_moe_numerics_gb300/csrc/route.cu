// route.cu -- from router logits to rows in expert order and back:
//   pmn_route_topk             chosen experts, gates, and the routed rows' layout
//   pmn_route_topk_backward    the logits' gradient
//   pmn_dispatch_rows          token rows -> routed rows
//   pmn_combine_rows           the weighted sum of each token's routed rows
//   pmn_combine_rows_backward  its gradients
// The router is bound by latency (16384 tokens of 384 experts: choosing 16 us, of which its 8.7 M warp instructions
// fill the issue slots for 7; placing 15 for 4, half of it behind the choosing; the gradient 7 to 10 for 3; up to 256
// tokens 6 to 8 in all; 512 and 1024 experts 27 and 45, k 16 and 32 of 384 31 and 93, where the lanes no longer bound
// the choice), the rows by HBM (16384 x 4096 bf16, top-8: 215 us out, 6.2 TB/s, and 190 us back).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/pmn.h"
#include "args.cuh"
#include "numerics.cuh"

using namespace pmn;

namespace {

__device__ int g_route_error = 0;

constexpr int MAX_EXPERTS = 1024, MAX_K = 32, MAX_CHOICES = 64;
constexpr unsigned FULL = 0xFFFFFFFFu;

// ====================================================================== router
// Tokens are counted and laid out in chunks, one CTA each: at most MAX_CHUNKS, so that
// every CTA of the second kernel can add up the counts of all of them by itself.
constexpr int MAX_CHUNKS = 152, MIN_CHUNK = 64, SUB = 128;
constexpr int64_t MAX_TOKENS = 8384512;
static_assert((MAX_TOKENS + MAX_CHUNKS - 1) / MAX_CHUNKS <= 65535, "a chunk's counts are 16 bits wide");
constexpr int CLUSTER = 8, FEW_TOKENS = 32 * CLUSTER;  // so few are routed by one cluster, a token per warp

inline int64_t chunk_tokens(int64_t tokens) { return std::max<int64_t>(MIN_CHUNK, (tokens + MAX_CHUNKS - 1) / MAX_CHUNKS); }

inline int64_t chunk_count(int64_t tokens) { return (tokens + chunk_tokens(tokens) - 1) / chunk_tokens(tokens); }

struct RouteArgs {
    const void *logits;
    int64_t ldl;
    const float *bias;
    int64_t tokens, chunk, rows;
    int experts, k, half, score, normalize, pad;  // half: half the power of two that holds k
    float scale;
    int32_t *chosen;
    float *gates;
    int32_t *row_index, *row_choice, *offsets;
    uint16_t *counts;  // [chunks][experts, rounded up to an even number]
};

template <int KIND>
__device__ __forceinline__ float load_logit(const void *p, int64_t i)
{
    if (KIND == PMN_OUT_F32) return __ldg(static_cast<const float *>(p) + i);
    return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(p) + i) << 16);
}

// Larger value, larger key; NaN above everything; NONE (-inf) below every other value.  The sum
// makes +0 of -0 (equal values, equal keys) and a positive NaN of any.
constexpr uint32_t NONE = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

// The largest of the lanes' values, NaN left out.
__device__ __forceinline__ float warp_max(float v)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(FULL, v, o));
    return v;
}

// log(1 / (1 + e^-x)), which keeps its relative precision where the sigmoid vanishes
__device__ __forceinline__ float log_sigmoid(float x) { return __fsub_rn(fminf(x, 0.0f), log1pf(expf(-fabsf(x)))); }

// 1 / (1 + e^-x); far below zero it is e^x, also where e^-x leaves float32's range.
__device__ __forceinline__ float score_sigmoid(float x) { return x < -80.0f ? expf(x) : 1.0f / (1.0f + expf(-x)); }

// k experts by k rounds over all keys: many equals, or a large k.
template <int NV>
__device__ __noinline__ int choose_slowly(const uint32_t (&given)[NV], int k, int lane)
{
    uint32_t key[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) key[j] = given[j];
    int expert = -1;
    for (int i = 0; i < k; ++i) {
        uint32_t best = NONE;
        int which = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (key[j] > best) {
                best = key[j];
                which = j;
            }
        const uint32_t m = __reduce_max_sync(FULL, best);
        if (m == NONE) break;
        const int win = __reduce_min_sync(FULL, best == m ? 32 * which + lane : 0x7FFFFFFF);
        if (lane == i) expert = win;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (32 * j + lane == win) key[j] = NONE;
    }
    return expert;
}

// T tokens (token, token + step, ..) by one warp, side by side: lane i < k gets each one's i-th expert (-1:
// none is left) and its gate.  Lane l holds experts l, l + 32, ..  The k-th largest of the lanes' own largest
// keys bounds the token's k-th largest from below, so what is not less than it -- little more
// than k keys -- holds the choice; those few are packed, one to a lane, in the experts' order,
// and ordered by comparing them all.  (16384 tokens of 384 experts: k rounds over all keys 27 us, k rounds over the
// few 18, this 17; 530 instructions a token, which seven warps a scheduler issue less than half of the time: they wait
// for the k maxima, each behind the one before.)
template <int T, int NV, int KIND>
__device__ __forceinline__ void choose(const RouteArgs &p, int64_t token, int64_t step, int lane, uint2 (*few)[32],
                                       int (&expert)[T], float (&gate)[T])
{
    uint32_t key[T][NV], best[T], bound[T];
    float top[T], total[T];
    const bool every = p.score == PMN_SCORE_SOFTMAX && !p.normalize;
    {
        float v[T][NV];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                v[t][j] = lane + 32 * j < p.experts && token + t * step < p.tokens
                              ? load_logit<KIND>(p.logits, (token + t * step) * p.ldl + lane + 32 * j) : -INFINITY;
        if (every) {  // the denominator runs over all experts
#pragma unroll
            for (int t = 0; t < T; ++t) {
                top[t] = -INFINITY;
                total[t] = 0.0f;
#pragma unroll
                for (int j = 0; j < NV; ++j) top[t] = fmaxf(top[t], v[t][j]);
                top[t] = warp_max(top[t]);
                if (top[t] == -INFINITY) top[t] = 0.0f;
#pragma unroll
                for (int j = 0; j < NV; ++j) total[t] += expf(v[t][j] - top[t]);
                total[t] = warp_sum(total[t]);
            }
        }
        if (p.bias) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const float b = lane + 32 * j < p.experts ? __ldg(p.bias + lane + 32 * j) : 0.0f;
#pragma unroll
                for (int t = 0; t < T; ++t)  // (a token behind the last has no logits to be chosen by: -inf plus inf is a NaN)
                    if (t == 0 || token + t * step < p.tokens) v[t][j] = __fadd_rn(v[t][j], b);
            }
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
            best[t] = NONE;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                key[t][j] = order_key(v[t][j]);
                best[t] = max(best[t], key[t][j]);
            }
            bound[t] = NONE + 1;  // every expert above -inf, where fewer than k lanes have one
        }
    }
    for (int i = 0; i < p.k; ++i) {
        uint32_t m[T];
#pragma unroll
        for (int t = 0; t < T; ++t) m[t] = __reduce_max_sync(FULL, best[t]);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            bound[t] = max(m[t], NONE + 1);
            if (best[t] == m[t]) best[t] = NONE;
        }
    }
    int count[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        expert[t] = -1;
        count[t] = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t in = __ballot_sync(FULL, key[t][j] >= bound[t]);
            if (in == 0u) continue;
            const int to = count[t] + __popc(in & ((1u << lane) - 1u));
            if (key[t][j] >= bound[t] && to < 32) few[t][to] = make_uint2(key[t][j], 32 * j + lane);
            count[t] += __popc(in);
        }
    }
    __syncwarp();
    uint2 mine[T];
#pragma unroll
    for (int t = 0; t < T; ++t) mine[t] = lane < count[t] ? few[t][lane] : make_uint2(NONE, 0u);
    __syncwarp();
    // a key's place among them: how many are larger, or equal and of a lower expert
    int most = 0, place[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        most = max(most, min(count[t], 32));
        place[t] = 0;
    }
    for (int c = 0; c < most; ++c)
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const uint32_t other = __shfl_sync(FULL, mine[t].x, c);
            place[t] += other > mine[t].x || (other == mine[t].x && c < lane);
        }
#pragma unroll
    for (int t = 0; t < T; ++t)
        if (mine[t].x != NONE && place[t] < p.k) few[t][place[t]].y = mine[t].y;
    __syncwarp();
#pragma unroll
    for (int t = 0; t < T; ++t)
        if (lane < min(p.k, count[t])) expert[t] = (int)few[t][lane].y;
    __syncwarp();
#pragma unroll
    for (int t = 0; t < T; ++t)
        if (count[t] > 32) expert[t] = choose_slowly<NV>(key[t], p.k, lane);
    float l[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
        l[t] = expert[t] >= 0 ? load_logit<KIND>(p.logits, (token + t * step) * p.ldl + expert[t]) : -INFINITY;
#pragma unroll
    for (int t = 0; t < T; ++t) {
        float g;
        if (every) {
            g = expf(l[t] - top[t]) / total[t];
        } else if (!p.normalize) {
            g = score_sigmoid(l[t]);
        } else {
            const float v = p.score == PMN_SCORE_SOFTMAX ? l[t] : expert[t] >= 0 ? log_sigmoid(l[t]) : -INFINITY;
            float m = warp_max(v);
            if (m == -INFINITY) m = 0.0f;
            const float e = expert[t] >= 0 ? expf(v - m) : 0.0f;
            float sum = e;
            for (int o = p.half; o; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(FULL, sum, o));  // of the first k lanes
            g = e / sum;
        }
        gate[t] = expert[t] >= 0 ? __fmul_rn(p.scale, g) : 0.0f;
    }
}

// What the layout of a chunk needs in shared memory.
struct Layout {
    uint32_t mask[MAX_EXPERTS][SUB / 32];  // which of SUB tokens chose the expert
    int32_t base[MAX_EXPERTS];             // first row that is still free
    int32_t total[MAX_EXPERTS], first[MAX_EXPERTS + 1];
    int32_t sums[32];
};

// Padded running sum of the totals (first[e]: the expert's first row), by the whole CTA.
__device__ void scan_offsets(const RouteArgs &p, Layout &s)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto padded = [&](int e) { return e < p.experts ? (int)((uint32_t)(s.total[e] + p.pad - 1) / (uint32_t)p.pad) * p.pad : 0; };
    __syncthreads();
    for (int e0 = 0; e0 < p.experts; e0 += blockDim.x) {  // sums of 32 experts each
        const int e = e0 + threadIdx.x, n = __reduce_add_sync(FULL, padded(e));
        if (lane == 0 && e < p.experts) s.sums[e >> 5] = n;
    }
    __syncthreads();
    for (int e0 = 0; e0 < p.experts; e0 += blockDim.x) {
        const int e = e0 + 32 * warp + lane, n = padded(e);
        int run = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL, run, o);
            if (lane >= o) run += v;
        }
        run += __reduce_add_sync(FULL, lane < (e >> 5) ? s.sums[lane] : 0) - n;
        if (e < p.experts) s.first[e] = run;
        if (e == p.experts - 1) s.first[p.experts] = run + n;
    }
    __syncthreads();
}

// Rows of the chunk's choices: an expert's rows follow its tokens' order, so a choice's
// place is the number of earlier tokens that chose the expert -- a count of bits, the same
// in whatever order the bits were set.  s.base holds the rows left by earlier chunks, mine the
// thread's first choice.
__device__ void place(const RouteArgs &p, Layout &s, int64_t token0, int64_t token1, int mine)
{
    for (int64_t t0 = token0; t0 < token1; t0 += SUB) {
        const int n = (int)min((int64_t)SUB, token1 - t0) * p.k;
        for (int e = threadIdx.x; e < p.experts; e += blockDim.x)
#pragma unroll
            for (int w = 0; w < SUB / 32; ++w) s.mask[e][w] = 0u;
        __syncthreads();
        const int32_t *chosen = p.chosen + t0 * p.k;
        for (int c = threadIdx.x; c < n; c += blockDim.x) {
            const int e = t0 == token0 && c == (int)threadIdx.x ? mine : chosen[c], t = c / p.k;
            if (e >= 0) atomicOr(&s.mask[e][t >> 5], 1u << (t & 31));
        }
        __syncthreads();
        for (int c = threadIdx.x; c < n; c += blockDim.x) {
            const int e = t0 == token0 && c == (int)threadIdx.x ? mine : chosen[c], t = c / p.k;
            int row = -1;
            if (e >= 0) {
                row = s.base[e] + __popc(s.mask[e][t >> 5] & ((1u << (t & 31)) - 1u));
                for (int w = 0; w < t >> 5; ++w) row += __popc(s.mask[e][w]);
                p.row_choice[row] = (int32_t)(t0 * p.k + c);
            }
            p.row_index[t0 * p.k + c] = row;
        }
        if (t0 + SUB >= token1) break;
        __syncthreads();
        for (int e = threadIdx.x; e < p.experts; e += blockDim.x)
#pragma unroll
            for (int w = 0; w < SUB / 32; ++w) s.base[e] += __popc(s.mask[e][w]);
        __syncthreads();
    }
}

// -1 for the padding rows of the segments, -2 for the rows behind the last one.
__device__ void mark_padding(const RouteArgs &p, const Layout &s)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int e = blockIdx.x * warps + warp; e < p.experts; e += gridDim.x * warps)
        for (int r = s.first[e] + s.total[e] + lane; r < s.first[e + 1]; r += 32) p.row_choice[r] = -1;
    for (int64_t r = s.first[p.experts] + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < p.rows;
         r += (int64_t)gridDim.x * blockDim.x)
        p.row_choice[r] = -2;
}

// The tokens of a chunk chosen, T by a warp at a time, and counted.
template <int T, int NV, int KIND>
__device__ __forceinline__ void choose_chunk(const RouteArgs &p, int64_t t0, int64_t t1, uint2 (*few)[32], int32_t *count)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) count[e] = 0;
    __syncthreads();
    for (int64_t t = t0 + warp; t < t1; t += T * warps) {
        int expert[T];
        float gate[T];
        choose<T, NV, KIND>(p, t, warps, lane, few, expert, gate);
#pragma unroll
        for (int i = 0; i < T; ++i)
            if (lane < p.k && t + i * warps < t1) {
                p.chosen[(t + i * warps) * p.k + lane] = expert[i];
                p.gates[(t + i * warps) * p.k + lane] = gate[i];
                if (expert[i] >= 0) atomicAdd(count + expert[i], 1);
            }
    }
}

// One CTA per chunk.
template <int NV, int KIND>
__global__ void __launch_bounds__(NV > 16 ? 512 : 1024) route_choose_kernel(const RouteArgs p)
{
    __shared__ int32_t count[MAX_EXPERTS];
    constexpr int T = NV > 12 ? 1 : 2;
    __shared__ uint2 few[NV > 16 ? 16 : 32][T][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk, t1 = min(p.tokens, t0 + p.chunk);
    choose_chunk<T, NV, KIND>(p, t0, t1, few[threadIdx.x >> 5], count);
    __syncthreads();
    const int pitch = (p.experts + 1) / 2 * 2;
    for (int e = threadIdx.x; e < pitch; e += blockDim.x)
        p.counts[(int64_t)blockIdx.x * pitch + e] = e < p.experts ? (uint16_t)count[e] : (uint16_t)0;
}

// Few tokens: one cluster, whose CTAs read one another's counts.  (384 experts, 64 and 256 tokens, us back to
// back: 6.0 and 7.9; one CTA 9.7 and the two kernels 11.1.  512 tokens: 11.4 either way.  256 threads a CTA
// instead of 512: 6.5 and 7.9.)
template <int NV, int KIND>
__global__ void __launch_bounds__(NV > 16 ? 512 : 1024) route_few_kernel(const RouteArgs p)
{
    __shared__ Layout s;
    __shared__ int32_t count[MAX_EXPERTS];
    __shared__ uint2 few[NV > 16 ? 16 : 32][1][32];
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk, t1 = min(p.tokens, t0 + p.chunk);
    choose_chunk<1, NV, KIND>(p, t0, t1, few[threadIdx.x >> 5], count);
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    const uint32_t counts = (uint32_t)__cvta_generic_to_shared(count);
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) {
        int n[CLUSTER], before = 0, all = 0;
#pragma unroll
        for (int c = 0; c < CLUSTER; ++c) {
            n[c] = 0;
            if (c < (int)gridDim.x)
                asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.s32 %0, [a];\n\t}"
                             : "=r"(n[c])
                             : "r"(counts + 4 * e), "r"(c));
        }
#pragma unroll
        for (int c = 0; c < CLUSTER; ++c) {
            all += n[c];
            if (c < (int)blockIdx.x) before += n[c];
        }
        s.total[e] = all;
        s.base[e] = before;
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA has read the others
    const int mine = (int)threadIdx.x < (int)(t1 - t0) * p.k ? p.chosen[t0 * p.k + threadIdx.x] : -1;
    scan_offsets(p, s);
    for (int e = threadIdx.x; e <= p.experts; e += blockDim.x) {
        if (blockIdx.x == 0) p.offsets[e] = s.first[e];
        if (e < p.experts) s.base[e] += s.first[e];
    }
    place(p, s, t0, t1, mine);
    mark_padding(p, s);
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // and the others this one
}

__global__ void __launch_bounds__(1024) route_place_kernel(const RouteArgs p, int chunks)
{
    __shared__ Layout s;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the choosing kernel still runs
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk, t1 = min(p.tokens, t0 + p.chunk);
    const int mine = threadIdx.x < (t1 - t0) * p.k ? __ldcg(p.chosen + t0 * p.k + threadIdx.x) : -1;
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) s.total[e] = s.base[e] = 0;
    __syncthreads();
    // a thread adds up two experts over every `parts`th chunk
    const int pitch = (p.experts + 1) / 2, parts = max(1, (int)blockDim.x / pitch);
    for (int i = threadIdx.x; i < pitch * parts; i += blockDim.x) {
        const int pair = i % pitch;
        int before0 = 0, before1 = 0, all0 = 0, all1 = 0;
        const uint32_t *c = reinterpret_cast<const uint32_t *>(p.counts) + pair;
#pragma unroll 16
        for (int ch = i / pitch; ch < chunks; ch += parts) {
            const uint32_t n = __ldcg(c + (int64_t)ch * pitch);
            all0 += n & 0xFFFFu;
            all1 += n >> 16;
            if (ch < (int)blockIdx.x) {
                before0 += n & 0xFFFFu;
                before1 += n >> 16;
            }
        }
        atomicAdd(&s.total[2 * pair], all0);
        atomicAdd(&s.base[2 * pair], before0);
        if (2 * pair + 1 < p.experts) {
            atomicAdd(&s.total[2 * pair + 1], all1);
            atomicAdd(&s.base[2 * pair + 1], before1);
        }
    }
    scan_offsets(p, s);
    for (int e = threadIdx.x; e <= p.experts; e += blockDim.x) {
        if (blockIdx.x == 0) p.offsets[e] = s.first[e];
        if (e < p.experts) s.base[e] += s.first[e];
    }
    place(p, s, t0, t1, mine);
    mark_padding(p, s);
}

template <int NV, int KIND>
pmn_status launch_route(RouteArgs &p, cudaStream_t s)
{
    const int most = NV > 16 ? 512 : 1024;
    if (p.tokens <= FEW_TOKENS) {
        unsigned ctas = 1;
        while (ctas < CLUSTER && 2 * (int64_t)ctas < p.tokens) ctas *= 2;
        p.chunk = (p.tokens + ctas - 1) / ctas;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3((unsigned)std::min<int64_t>(most, std::max<int64_t>(512, 32 * p.chunk)));
        cfg.stream = s;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = ctas;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, route_few_kernel<NV, KIND>, p) == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
    }
    const int chunks = (int)chunk_count(p.tokens);
    // as many warps as share the chunk's tokens evenly (65536 tokens of 384 experts 67 -> 61 us by this and one CTA per SM)
    const int64_t side = NV > 12 ? 1 : 2, most_warps = most / 32, passes = (p.chunk + side * most_warps - 1) / (side * most_warps);
    const int threads = 32 * (int)((p.chunk + side * passes - 1) / (side * passes));
    route_choose_kernel<NV, KIND><<<chunks, threads, 0, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return PMN_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)chunks);
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_place_kernel, p, chunks) == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

template <int KIND>
pmn_status route_by_experts(RouteArgs &p, cudaStream_t s)
{
    if (p.experts <= 64) return launch_route<2, KIND>(p, s);
    if (p.experts <= 128) return launch_route<4, KIND>(p, s);
    if (p.experts <= 256) return launch_route<8, KIND>(p, s);
    if (p.experts <= 384) return launch_route<12, KIND>(p, s);
    if (p.experts <= 512) return launch_route<16, KIND>(p, s);
    return launch_route<32, KIND>(p, s);
}

__global__ void route_empty_kernel(int32_t *offsets, int experts, int32_t *row_choice, int64_t rows)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i <= experts) offsets[i] = 0;
    for (int64_t r = i; r < rows; r += (int64_t)gridDim.x * blockDim.x) row_choice[r] = -2;
}

struct RouteGradArgs {
    const void *logits;
    int64_t ldl;
    const int32_t *chosen;
    const float *dgates;
    int64_t tokens;
    int experts, k, score, normalize;
    float scale;
    void *dlogits;
    bool wide;  // dlogits is 16-byte aligned
};

template <int KIND>
__device__ __forceinline__ void store_grad(void *p, int64_t i, float v)
{
    if (KIND == PMN_OUT_F32) static_cast<float *>(p)[i] = v;
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// One warp per token: the k chosen entries from the chosen logits (every entry, where the
// gates' denominator runs over all experts), zeros elsewhere.
template <int KIND>
__global__ void __launch_bounds__(256) route_backward_kernel(const RouteGradArgs p)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    const int64_t at = t * p.ldl, out = t * p.experts;
    const bool every = p.score == PMN_SCORE_SOFTMAX && !p.normalize;
    if (!every) {  // the rest of the row, while the chosen logits are on their way
        constexpr int N = KIND == PMN_OUT_F32 ? 4 : 8;
        uint8_t *row = static_cast<uint8_t *>(p.dlogits) + out * (16 / N);
        if (p.experts % N == 0 && p.wide) {
            for (int c = lane; c < p.experts / N; c += 32) reinterpret_cast<uint4 *>(row)[c] = make_uint4(0u, 0u, 0u, 0u);
        } else {
            for (int c = lane; c < p.experts; c += 32) store_grad<KIND>(p.dlogits, out + c, 0.0f);
        }
    }
    int e = -1;
    float d = 0.0f;
    if (lane < p.k) {
        e = p.chosen[t * p.k + lane];
        d = p.dgates[t * p.k + lane];
    }
    if (e < 0 || e >= p.experts) {  // a dropped choice, or not an expert's number
        if (e >= p.experts) atomicOr(&g_route_error, PMN_DEVERR_BAD_OFFSETS);
        e = -1;
        d = 0.0f;
    }
    const float l = e >= 0 ? load_logit<KIND>(p.logits, at + e) : -INFINITY;
    float g = 0.0f, top = -INFINITY, total = 0.0f, sg = 0.0f;
    if (p.score == PMN_SCORE_SIGMOID) sg = score_sigmoid(-l);  // 1 - sigmoid, without its cancellation
    if (every) {
        for (int c = lane; c < p.experts; c += 32) top = fmaxf(top, load_logit<KIND>(p.logits, at + c));
        top = warp_max(top);
        if (top == -INFINITY) top = 0.0f;
        for (int c = lane; c < p.experts; c += 32) total += expf(load_logit<KIND>(p.logits, at + c) - top);
        total = warp_sum(total);
        g = e >= 0 ? expf(l - top) / total : 0.0f;
    } else if (p.normalize) {
        const float v = e < 0 ? -INFINITY : p.score == PMN_SCORE_SOFTMAX ? l : log_sigmoid(l);
        float m = warp_max(v);
        if (m == -INFINITY) m = 0.0f;
        const float x = e >= 0 ? expf(v - m) : 0.0f;
        const float sum = warp_sum(x);
        g = e >= 0 ? x / sum : 0.0f;
    } else {
        g = e >= 0 ? score_sigmoid(l) : 0.0f;
    }
    const float dot = p.score == PMN_SCORE_SIGMOID && !p.normalize ? 0.0f : warp_sum(__fmul_rn(g, d));
    float grad = __fmul_rn(__fmul_rn(p.scale, g), __fsub_rn(d, dot));
    if (p.score == PMN_SCORE_SIGMOID) grad = __fmul_rn(grad, sg);
    if (every) {
        for (int c = lane; c < p.experts; c += 32) {
            const float q = total > 0.0f || total != total ? expf(load_logit<KIND>(p.logits, at + c) - top) / total : 0.0f;
            store_grad<KIND>(p.dlogits, out + c, -__fmul_rn(__fmul_rn(p.scale, q), dot));
        }
    }
    __syncwarp();  // the chosen entries are written after the row
    if (e >= 0) store_grad<KIND>(p.dlogits, out + e, grad);
}

// ====================================================================== rows
// Sixteen bytes of a row: N values as float32.
template <int KIND>
struct Vec {
    static constexpr int N = KIND == PMN_OUT_F32 ? 4 : 8;
    static __device__ __forceinline__ void unpack(const uint4 &q, float (&v)[N])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = u4_word(q, i);
            if (KIND == PMN_OUT_F32) {
                v[i] = __uint_as_float(w);
            } else {
                v[(2 * i) % N] = __uint_as_float(w << 16);
                v[(2 * i + 1) % N] = __uint_as_float(w & 0xFFFF0000u);
            }
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[N])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (KIND == PMN_OUT_F32) {
                w[i] = __float_as_uint(v[i]);
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[(2 * i) % N], v[(2 * i + 1) % N]);
                w[i] = *reinterpret_cast<const uint32_t *>(&b);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The CTAs behind the tokens' look for padding rows and write zeros there, PAD_ROWS each.
constexpr int PAD_ROWS = 32;

__device__ __forceinline__ void zero_padding(const int32_t *row_choice, int64_t rows, uint4 *out, int vecs, int64_t block)
{
    const int64_t r0 = block * PAD_ROWS;
    const int n = (int)min((int64_t)PAD_ROWS, rows - r0), lane = threadIdx.x & 31;
    uint32_t pads = __ballot_sync(FULL, lane < n && __ldg(row_choice + r0 + lane) == -1);
    for (; pads; pads &= pads - 1) {
        uint4 *o = out + (r0 + __ffs(pads) - 1) * vecs;
        for (int v = threadIdx.x; v < vecs; v += blockDim.x) o[v] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// A row number of a choice: -1 where it was dropped, or is not a row (the error word then says so).
__device__ __forceinline__ int32_t checked_row(int32_t r, int64_t rows)
{
    if (r >= rows) {
        atomicOr(&g_route_error, PMN_DEVERR_BAD_OFFSETS);
        return -1;
    }
    return r;
}

// Tokens and 16-byte pieces of their rows over CTAs: `tokens` tokens of short rows in a CTA, one
// token's row in turns of `threads` pieces, or, where the tokens alone would not fill the GPU,
// 1 / `parts` of a row (64 tokens, eight rows each of 4096 bf16 columns: 7.0 us -> 4.5).  The sums of 8 bf16 rows a
// token in whole rows and in parts of 256 pieces: 128 tokens of 7168 columns 6.7 and 3.9 us, 256 tokens of 4096 4.9 and 5.2;
// 512 tokens of 1536 3.9 and 5.0, of 2048 5.2 either way, of 4096 8.8 and 8.1; 768 tokens of 1536 5.4 and 5.8, of 4096 10.7
// and 11.6.  1024 CTAs are some seven an SM.
struct Split {
    int tokens, parts, threads;
    static Split of(int64_t n, int vecs)
    {
        if (vecs <= 128) return Split{256 / vecs, 1, 256};
        const int turns = (vecs + 255) / 256;
        if (n >= 512) return Split{1, 1, ((vecs + turns - 1) / turns + 31) / 32 * 32};
        int threads = 256;
        while (threads > 64 && n * ((vecs + threads - 1) / threads) < 1024) threads /= 2;
        return Split{1, (vecs + threads - 1) / threads, threads};
    }
    int64_t blocks(int64_t n) const { return parts > 1 ? n * parts : (n + tokens - 1) / tokens; }
    // the thread's token and its pieces first, first + step, .. < end
    __device__ __forceinline__ bool place(int64_t &t, int &first, int &step, int64_t n, int vecs) const
    {
        step = parts > 1 || tokens > 1 ? vecs : threads;  // one piece
        if (parts > 1) {
            t = blockIdx.x / (unsigned)parts;
            first = (int)(blockIdx.x - t * parts) * threads + threadIdx.x;
            return first < vecs;
        }
        const int sub = tokens > 1 ? (int)threadIdx.x / vecs : 0;
        t = (int64_t)blockIdx.x * tokens + sub;
        first = threadIdx.x - sub * vecs;
        return sub < tokens && t < n;
    }
};

// Each token's row is read once and written to its k rows.
__global__ void __launch_bounds__(256)
    dispatch_kernel(const uint4 *__restrict__ x, int64_t ldv, int64_t tokens, int vecs, const int32_t *__restrict__ row_index,
                    int k, const int32_t *__restrict__ row_choice, int64_t rows, uint4 *out, int64_t token_blocks, Split by)
{
    if (blockIdx.x >= token_blocks) {
        zero_padding(row_choice, rows, out, vecs, blockIdx.x - token_blocks);
        return;
    }
    int64_t t;
    int v, step;
    if (!by.place(t, v, step, tokens, vecs)) return;
    const int32_t *idx = row_index + t * k;
    for (; v < vecs; v += step) {
        const uint4 q = __ldcs(x + t * ldv + v);
        for (int i = 0; i < k; ++i) {
            const int32_t r = checked_row(__ldg(idx + i), rows);
            if (r >= 0) __stcs(out + (int64_t)r * vecs + v, q);
        }
    }
}

// out = sum of gate * row, in the order of the choices.
template <int KIND, int OUT>
__global__ void __launch_bounds__(256)
    combine_kernel(const uint4 *__restrict__ z, int64_t rows, int vecs, const int32_t *__restrict__ row_index,
                   const float *__restrict__ gates, int64_t tokens, int k, void *out, Split by)
{
    constexpr int N = Vec<KIND>::N;
    int64_t t;
    int v, step;
    if (!by.place(t, v, step, tokens, vecs)) return;
    const int32_t *idx = row_index + t * k;
    for (; v < vecs; v += step) {
        float acc[N];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = 0.0f;
        for (int i0 = 0; i0 < k; i0 += 8) {
            uint4 q[8];
            float g[8];
            bool on[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int32_t r = i0 + i < k ? checked_row(__ldg(idx + i0 + i), rows) : -1;
                on[i] = r >= 0;
                if (on[i]) {
                    q[i] = __ldcs(z + (int64_t)r * vecs + v);
                    g[i] = gates ? __ldg(gates + t * k + i0 + i) : 1.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (on[i]) {
                    float w[N];
                    Vec<KIND>::unpack(q[i], w);
#pragma unroll
                    for (int j = 0; j < N; ++j) acc[j] = fmaf(g[i], w[j], acc[j]);
                }
        }
        if constexpr (KIND == OUT) {
            static_cast<uint4 *>(out)[t * vecs + v] = Vec<KIND>::pack(acc);
        } else if constexpr (OUT == PMN_OUT_F32) {
            float4 *o = static_cast<float4 *>(out) + (t * vecs + v) * 2;
            o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            o[1] = make_float4(acc[4 % N], acc[5 % N], acc[6 % N], acc[7 % N]);
        } else {
            uint2 *o = static_cast<uint2 *>(out) + t * vecs + v;
            const __nv_bfloat162 a = __floats2bfloat162_rn(acc[0], acc[1]), b = __floats2bfloat162_rn(acc[2], acc[3]);
            *o = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        }
    }
}

// One CTA per token: dz = gate * dout and the k sums <dout, z>, eight choices at a time.
template <int KIND>
__global__ void __launch_bounds__(256)
    combine_backward_kernel(const uint4 *__restrict__ dout, const uint4 *__restrict__ z, int64_t tokens, int vecs,
                            const int32_t *__restrict__ row_index, const int32_t *__restrict__ row_choice,
                            const float *__restrict__ gates, int k, int64_t rows, uint4 *dz, float *dgates)
{
    constexpr int N = Vec<KIND>::N;
    __shared__ float part[8][8];
    if (blockIdx.x >= tokens) {
        zero_padding(row_choice, rows, dz, vecs, blockIdx.x - tokens);
        return;
    }
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int i0 = 0; i0 < k; i0 += 8) {
        int32_t r[8];
        float g[8], dot[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[i] = i0 + i < k ? checked_row(__ldg(row_index + t * k + i0 + i), rows) : -1;
            g[i] = r[i] >= 0 && gates ? __ldg(gates + t * k + i0 + i) : 1.0f;
            dot[i] = 0.0f;
        }
        for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
            float d[N];
            Vec<KIND>::unpack(__ldg(dout + t * vecs + v), d);
            uint4 q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r[i] >= 0) q[i] = __ldcs(z + (int64_t)r[i] * vecs + v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r[i] >= 0) {
                    float w[N], o[N];
                    Vec<KIND>::unpack(q[i], w);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        dot[i] = fmaf(d[j], w[j], dot[i]);
                        o[j] = __fmul_rn(g[i], d[j]);
                    }
                    __stcs(dz + (int64_t)r[i] * vecs + v, Vec<KIND>::pack(o));
                }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[i] = warp_sum(dot[i]);
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < 8; ++i) part[warp][i] = dot[i];
        __syncthreads();
        if (threadIdx.x < 8 && i0 + (int)threadIdx.x < k) {
            float sum = 0.0f;
            for (int w = 0; w < warps; ++w) sum = __fadd_rn(sum, part[w][threadIdx.x]);
            dgates[t * k + i0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

int kind_bytes(int kind) { return kind == PMN_OUT_BF16 ? 2 : kind == PMN_OUT_F32 ? 4 : 0; }

// What the three row calls ask of their sizes.
bool good_rows(int64_t tokens, int64_t cols, int kind, int k, int64_t rows)
{
    const int b = kind_bytes(kind);
    return b && tokens >= 0 && tokens < (int64_t(1) << 31) - 1 && cols >= 0 && cols < (int64_t(1) << 28) && cols * b % 16 == 0 &&
           k >= 1 && k <= MAX_CHOICES && rows >= 0 && rows < (int64_t(1) << 31);
}

bool good_grid(int64_t blocks) { return blocks < (int64_t(1) << 31); }

}  // namespace

pmn_status pmn_route_error_word(int **word)
{
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_route_error) == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

extern "C" int64_t pmn_route_rows(int64_t tokens, int experts, int k, int pad)
{
    if (tokens < 0 || tokens >= (int64_t(1) << 31) || experts < 1 || experts > MAX_EXPERTS || k < 1 || k > MAX_K || k > experts ||
        pad < 1 || pad > (1 << 20))
        return -1;
    const int64_t n = tokens * k;
    return (n + std::min<int64_t>(experts, n) * (pad - 1)) / pad * pad;
}

extern "C" int64_t pmn_route_topk_workspace_bytes(int64_t tokens, int experts, int k)
{
    if (pmn_route_rows(tokens, experts, k, 1) < 0) return -1;
    return tokens <= FEW_TOKENS ? 0 : (chunk_count(tokens) * ((experts + 1) / 2 * 4) + 15) / 16 * 16;
}

extern "C" pmn_status pmn_route_topk(const void *logits, int64_t ldl, int logits_kind, const float *bias, int64_t tokens,
                                     int experts, int k, int score, int normalize, float scale, int pad, int64_t rows,
                                     int32_t *chosen, float *gates, int32_t *row_index, int32_t *row_choice,
                                     int32_t *offsets, void *workspace, int64_t workspace_bytes, void *stream)
{
    const int64_t need = pmn_route_rows(tokens, experts, k, pad);
    if (need < 0 || rows < need || rows >= (int64_t(1) << 31) || !kind_bytes(logits_kind) || ldl < experts ||
        (score != PMN_SCORE_SOFTMAX && score != PMN_SCORE_SIGMOID) || (normalize != 0 && normalize != 1))
        return PMN_ERR_INVALID_ARG;
    if (!offsets || (rows > 0 && !row_choice) || !aligned(offsets, 4) || !aligned(row_choice, 4)) return PMN_ERR_INVALID_ARG;
    if (tokens > MAX_TOKENS) return PMN_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (tokens == 0) {
        route_empty_kernel<<<64, 256, 0, s>>>(offsets, experts, row_choice, rows);
        return cudaGetLastError() == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
    }
    const int64_t ws = pmn_route_topk_workspace_bytes(tokens, experts, k);
    if (!logits || !chosen || !gates || !row_index || !aligned(logits, kind_bytes(logits_kind)) || !aligned(bias, 4) ||
        !aligned(chosen, 4) || !aligned(gates, 4) || !aligned(row_index, 4) || workspace_bytes < ws ||
        (ws > 0 && (!workspace || !aligned(workspace, 16))))
        return PMN_ERR_INVALID_ARG;
    if (among(chosen, {logits, bias, gates, row_index, row_choice, offsets}) ||
        among(gates, {logits, bias, row_index, row_choice, offsets}) || among(row_index, {logits, bias, row_choice, offsets}) ||
        among(row_choice, {logits, bias, offsets}) || among(offsets, {logits, bias}) ||
        (ws > 0 && among(workspace, {logits, bias, chosen, gates, row_index, row_choice, offsets})))
        return PMN_ERR_INVALID_ARG;
    int half = 0;
    while ((half ? 2 * half : 1) < k) half = half ? 2 * half : 1;
    RouteArgs a{logits, ldl, bias, tokens, chunk_tokens(tokens), rows, experts, k, half, score, normalize, pad, scale,
                      chosen, gates, row_index, row_choice, offsets, static_cast<uint16_t *>(workspace)};
    return logits_kind == PMN_OUT_F32 ? route_by_experts<PMN_OUT_F32>(a, s) : route_by_experts<PMN_OUT_BF16>(a, s);
}

extern "C" pmn_status pmn_route_topk_backward(const void *logits, int64_t ldl, int logits_kind, const int32_t *chosen,
                                              const float *dgates, int64_t tokens, int experts, int k, int score,
                                              int normalize, float scale, void *dlogits, void *stream)
{
    if (pmn_route_rows(tokens, experts, k, 1) < 0 || !kind_bytes(logits_kind) || ldl < experts ||
        (score != PMN_SCORE_SOFTMAX && score != PMN_SCORE_SIGMOID) || (normalize != 0 && normalize != 1))
        return PMN_ERR_INVALID_ARG;
    if (tokens == 0) return PMN_OK;
    if (!logits || !chosen || !dgates || !dlogits || !aligned(logits, kind_bytes(logits_kind)) ||
        !aligned(dlogits, kind_bytes(logits_kind)) || !aligned(chosen, 4) || !aligned(dgates, 4) ||
        among(dlogits, {logits, chosen, dgates}))
        return PMN_ERR_INVALID_ARG;
    const RouteGradArgs a{logits, ldl, chosen, dgates, tokens, experts, k, score, normalize, scale, dlogits, aligned(dlogits, 16)};
    const unsigned blocks = (unsigned)((tokens + 7) / 8);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (logits_kind == PMN_OUT_F32) route_backward_kernel<PMN_OUT_F32><<<blocks, 256, 0, s>>>(a);
    else route_backward_kernel<PMN_OUT_BF16><<<blocks, 256, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

extern "C" pmn_status pmn_dispatch_rows(const void *x, int64_t ldx, int kind, int64_t tokens, int64_t cols,
                                        const int32_t *row_index, int k, const int32_t *row_choice, int64_t rows, void *out,
                                        void *stream)
{
    if (!good_rows(tokens, cols, kind, k, rows) || ldx < cols || ldx * kind_bytes(kind) % 16 != 0) return PMN_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return PMN_OK;
    if (!out || !aligned(out, 16) || !aligned(row_choice, 4)) return PMN_ERR_INVALID_ARG;
    if (tokens > 0 && (!x || !row_index || !aligned(x, 16) || !aligned(row_index, 4) || among(out, {x, row_index})))
        return PMN_ERR_INVALID_ARG;
    if (among(out, {row_choice})) return PMN_ERR_INVALID_ARG;
    const int vecs = (int)(cols * kind_bytes(kind) / 16);
    const Split by = Split::of(tokens, vecs);
    const int64_t token_blocks = by.blocks(tokens);
    const int64_t blocks = token_blocks + (row_choice ? (rows + PAD_ROWS - 1) / PAD_ROWS : 0);
    if (!good_grid(blocks)) return PMN_ERR_UNSUPPORTED;
    if (blocks == 0) return PMN_OK;
    dispatch_kernel<<<(unsigned)blocks, by.threads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4 *>(x), ldx * kind_bytes(kind) / 16, tokens, vecs, row_index, k, row_choice, rows,
        static_cast<uint4 *>(out), token_blocks, by);
    return cudaGetLastError() == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

extern "C" pmn_status pmn_combine_rows(const void *z, int kind, int64_t rows, int64_t cols, const int32_t *row_index,
                                       const float *gates, int64_t tokens, int k, int out_kind, void *out, void *stream)
{
    if (!good_rows(tokens, cols, kind, k, rows) || !kind_bytes(out_kind) || cols * kind_bytes(out_kind) % 16 != 0)
        return PMN_ERR_INVALID_ARG;
    if (tokens == 0 || cols == 0) return PMN_OK;
    if ((rows > 0 && !z) || !row_index || !out || !aligned(z, 16) || !aligned(out, 16) || !aligned(row_index, 4) ||
        !aligned(gates, 4) || (rows > 0 && out == z) || among(out, {row_index, gates}))
        return PMN_ERR_INVALID_ARG;
    const int vecs = (int)(cols * kind_bytes(kind) / 16);
    const Split by = Split::of(tokens, vecs);
    if (!good_grid(by.blocks(tokens))) return PMN_ERR_UNSUPPORTED;
    const unsigned blocks = (unsigned)by.blocks(tokens);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define PMN_COMBINE(IN, OUT)                                                                                          \
    combine_kernel<IN, OUT><<<blocks, by.threads, 0, s>>>(static_cast<const uint4 *>(z), rows, vecs, row_index, gates, tokens, k, \
                                                   out, by)
    if (kind == PMN_OUT_F32 && out_kind == PMN_OUT_F32) PMN_COMBINE(PMN_OUT_F32, PMN_OUT_F32);
    else if (kind == PMN_OUT_F32) PMN_COMBINE(PMN_OUT_F32, PMN_OUT_BF16);
    else if (out_kind == PMN_OUT_F32) PMN_COMBINE(PMN_OUT_BF16, PMN_OUT_F32);
    else PMN_COMBINE(PMN_OUT_BF16, PMN_OUT_BF16);
#undef PMN_COMBINE
    return cudaGetLastError() == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}

extern "C" pmn_status pmn_combine_rows_backward(const void *dout, const void *z, int kind, int64_t rows, int64_t cols,
                                                const int32_t *row_index, const int32_t *row_choice, const float *gates,
                                                int64_t tokens, int k, void *dz, float *dgates, void *stream)
{
    if (!good_rows(tokens, cols, kind, k, rows) || cols == 0) return PMN_ERR_INVALID_ARG;
    if (tokens > 0 && (!dout || !row_index || !dgates || !aligned(dout, 16) || !aligned(row_index, 4) || !aligned(dgates, 4)))
        return PMN_ERR_INVALID_ARG;
    if (rows > 0 && (!z || !dz || !aligned(z, 16) || !aligned(dz, 16))) return PMN_ERR_INVALID_ARG;
    if (!aligned(row_choice, 4) || !aligned(gates, 4) || among(dz, {z, dout, row_choice}) || among(dgates, {gates})) return PMN_ERR_INVALID_ARG;
    if (tokens > 0 && (among(dz, {row_index, gates, dgates}) || among(dgates, {dout, z, row_index, row_choice})))
        return PMN_ERR_INVALID_ARG;
    const int vecs = (int)(cols * kind_bytes(kind) / 16);
    const int64_t blocks = tokens + (row_choice ? (rows + PAD_ROWS - 1) / PAD_ROWS : 0);
    if (!good_grid(blocks)) return PMN_ERR_UNSUPPORTED;
    if (blocks == 0) return PMN_OK;
    const int passes = (vecs + 255) / 256, threads = ((vecs + passes - 1) / passes + 31) / 32 * 32;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define PMN_BACKWARD(KIND)                                                                                         \
    combine_backward_kernel<KIND><<<(unsigned)blocks, threads, 0, s>>>(                                            \
        static_cast<const uint4 *>(dout), static_cast<const uint4 *>(z), tokens, vecs, row_index, row_choice, gates, k, rows, \
        static_cast<uint4 *>(dz), dgates)
    if (kind == PMN_OUT_F32) PMN_BACKWARD(PMN_OUT_F32);
    else PMN_BACKWARD(PMN_OUT_BF16);
#undef PMN_BACKWARD
    return cudaGetLastError() == cudaSuccess ? PMN_OK : PMN_ERR_CUDA;
}
