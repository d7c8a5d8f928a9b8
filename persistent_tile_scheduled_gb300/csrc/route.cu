// A router's choice: each token's top_k experts and their weights, and the
// gradient of its logits.
//
// G lanes per token (8, 16 or a warp), lane l of them with the logits of experts PER l ..
// PER l + PER - 1 in registers, loaded together (where rows do not allow it, of experts l,
// l + G, ..., one by one).  The key of a 16-bit logit, unsigned and in the order of the
// values, holds its expert too, the lower first.  A lane sorts its keys; then the top_k
// are taken one by one, each the largest of the lanes' first, which its lane pops.  fp32
// logits, and more than 8 choices, take a warp per token and redux.sync, and the lowest
// expert that has the largest.  Lane j keeps the j-th choice, so the softmax over the
// chosen is a sum over lanes.  The gradient brings dweights to the lanes that own their
// logits through shared memory.
//
// Instructions bound it, and fetching them: every warp runs through the code once.
// 16384 tokens, 8 of 128 experts, bf16 (4 MB in, 1 MB out): 5.5 us, and 4.1 back (16
// lanes per token; 8 lanes of 16 logits 6.2 and 4.2, a warp 6.9 and 6.2; merging sorted
// lists of 8 across the lanes instead of taking choices one by one 6.9).  16 tokens 1.2,
// a launch.
#include "activation.cuh"
#include "launch.cuh"
#include "layer_launch.h"
#include "ptx.cuh"

namespace pts {

namespace {

enum : int { ROUTE_SELECTED = 0, ROUTE_ALL = 1, ROUTE_SIGMOID = 2 };

constexpr int kRouteWarps = 4;
constexpr float kMaxFinite = 3.402823466e38f;
// What +infinity counts as: fp32's largest value; of 16-bit logits one above all of
// theirs whose lowest 13 bits are 0.
template <int KIND>
__device__ __forceinline__ float infinite()
{
    return KIND == 3 ? kMaxFinite : __int_as_float(0x7F7FE000);
}
#define kNothing __int_as_float(0xFF800000)   // -infinity
constexpr uint32_t kIndex = 0x1FFFu;   // of a 16-bit logit's fp32 bits the lowest 13 are 0: they hold the expert

// Unsigned keys in the order of the values.  -0 and 0 are one value; what cannot be chosen (-infinity, NaN) is below kLeast.
constexpr uint32_t kLeast = 0x00800000u;   // the key of the lowest finite value

template <int KIND>
__device__ __forceinline__ float cleaned(float v)   // (NaN: -infinity)
{
    return fminf(fmaxf(v, kNothing), infinite<KIND>());
}

template <int KIND>
__device__ __forceinline__ uint32_t key_of(float v, int e)   // v: cleaned
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    const uint32_t key = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return KIND == 3 ? key : (key & ~kIndex) | (kIndex - static_cast<uint32_t>(e));
}

template <int KIND>
__device__ __forceinline__ float value_of(uint32_t key)
{
    // (of a negative value the key's bits are the complement: the expert's place is filled with ones)
    if constexpr (KIND != 3) key = key & 0x80000000u ? key & ~kIndex : key | kIndex;
    return __uint_as_float(key ^ (static_cast<uint32_t>(~static_cast<int32_t>(key) >> 31) | 0x80000000u));
}

// A lane's i-th expert.
template <int PER, int G, bool WHOLE>
__device__ __forceinline__ int expert_of(int sub, int i)
{
    return WHOLE ? sub * PER + i : sub + G * i;
}

// A lane's PER logits of a row, cleaned (-infinity behind the last).  WHOLE: rows are a
// multiple of PER long and aligned to PER logits.
template <int KIND, int PER, int G, bool WHOLE>
__device__ __forceinline__ void load_logits(float (&x)[PER], const void *logits, long long row, int sub, int experts)
{
    constexpr int kBytes = PER * (KIND == 3 ? 4 : 2);
    if constexpr (WHOLE) {
        const int e0 = sub * PER;
        uint32_t v[(kBytes + 3) / 4] = {};
        const uint8_t *at = static_cast<const uint8_t *>(logits) + (row + (e0 < experts ? e0 : 0)) * (KIND == 3 ? 4 : 2);
        if constexpr (kBytes == 2) v[0] = ld_global(reinterpret_cast<const uint16_t *>(at));
        if constexpr (kBytes == 4) v[0] = ld_global(reinterpret_cast<const uint32_t *>(at));
        if constexpr (kBytes == 8) {
            const uint2 q = ld_global(reinterpret_cast<const uint2 *>(at));
            v[0] = q.x, v[1] = q.y;
        }
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) {
                const uint4 q = ld_global(reinterpret_cast<const uint4 *>(at) + i);
                v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
            }
        }
        const float most = e0 < experts ? infinite<KIND>() : kNothing;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if constexpr (KIND == 3) x[i] = __uint_as_float(v[i]);
            else x[i] = i % 2 ? unpack2<KIND>(v[i / 2]).y : unpack2<KIND>(v[i / 2]).x;
            x[i] = fminf(fmaxf(x[i], kNothing), most);   // (cleaned)
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = sub + G * i;
            x[i] = kNothing;
            if (e >= experts) continue;
            if constexpr (KIND == 3) x[i] = ld_global(static_cast<const float *>(logits) + row + e);
            else x[i] = unpack1<KIND>(ld_global(static_cast<const uint16_t *>(logits) + row + e));
            x[i] = cleaned<KIND>(x[i]);
        }
    }
}

__device__ __forceinline__ float exp_fast(float x) { return exp2_fast(kLog2E * x); }

// exp(l - best); SIGMOID: 1 / (1 + exp(-l)) = exp(min(l, 0)) / (1 + exp(-|l|)), scaled
// by exp(-min(best, 0)), so that the best one's is 1/2 at least however low all are.
__device__ __forceinline__ float share_of(float l, float best, int mode)
{
    if (mode != ROUTE_SIGMOID) return exp_fast(l - best);
    return exp_fast(fminf(l, 0.0f) - fminf(best, 0.0f)) * rcp_fast(1.0f + exp_fast(-fabsf(l)));
}

// The sum of exp(x - best) of a lane.
template <int PER>
__device__ __forceinline__ float exp_sum(const float (&x)[PER], float best)
{
    best = fmaxf(best, -kMaxFinite);   // (a row of nothing: 0)
    float all = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) all += exp_fast(x[i] - best);
    return all;
}

__device__ __forceinline__ void order(uint32_t &a, uint32_t &b)
{
    const uint32_t hi = max(a, b), lo = min(a, b);
    a = hi, b = lo;
}

// Sums and maxima over the G lanes of a token.
template <int G>
__device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int s = 1; s < G; s <<= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

template <int G, class T>
__device__ __forceinline__ T lanes_max(T v)
{
#pragma unroll
    for (int s = 1; s < G; s <<= 1) {
        const T o = __shfl_xor_sync(0xffffffffu, v, s);
        v = o > v ? o : v;
    }
    return v;
}

// Descending (Batcher's odd-even merge sort).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&a)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order(a[i + j], a[i + j + k]);
}

// The choice's weight, and the stores, of lane j < top_k of a token.
__device__ __forceinline__ void write_choice(const RouteParams &p, long long t, int j, bool there, int id, float w, float all)
{
    p.ids[t * p.top_k + j] = there ? id : -1;
    p.weights[t * p.top_k + j] = there ? w * rcp_fast(all) : 0.0f;
}

// 16-bit logits, top_k <= 8: G lanes per token
template <int KIND, int PER, int G, bool WHOLE>
__global__ void __launch_bounds__(32 * kRouteWarps) route_lanes_kernel(const RouteParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int sub = static_cast<int>(lane_id()) % G;
    const long long t = (static_cast<long long>(blockIdx.x) * (32 * kRouteWarps) + threadIdx.x) / G;
    float x[PER];
    uint32_t key[PER];
    // (behind the last token: the last again, not written)
    load_logits<KIND, PER, G, WHOLE>(x, p.logits, (t < p.tokens ? t : p.tokens - 1) * p.experts, sub, p.experts);
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = key_of<KIND>(x[i], expert_of<PER, G, WHOLE>(sub, i));
    sort_keys(key);
    const float best = value_of<KIND>(lanes_max<G>(key[0]));
    float all = p.mode == ROUTE_ALL ? lanes_sum<G>(exp_sum(x, best)) : 0.0f;
    constexpr int kKeep = PER < 8 ? PER : 8;   // (a lane has 8 choices at most)
    uint32_t mine = 0u;                        // this lane's choice
#pragma unroll 1
    for (int j = 0; j < p.top_k; ++j) {
        const uint32_t top = lanes_max<G>(key[0]);   // (below kLeast where nothing is left)
        if (sub == j) mine = top;
        if (key[0] == top) {
#pragma unroll
            for (int i = 0; i + 1 < kKeep; ++i) key[i] = key[i + 1];
            key[kKeep - 1] = 0u;
        }
    }
    const float w = mine >= kLeast ? share_of(value_of<KIND>(mine), best, p.mode) : 0.0f;
    if (p.mode != ROUTE_ALL) all = lanes_sum<G>(w);
    if (sub < p.top_k && t < p.tokens) write_choice(p, t, sub, mine >= kLeast, static_cast<int>(kIndex - (mine & kIndex)), w, all);
}

// A warp per token, PER logits per lane.
template <int KIND, int PER, bool WHOLE>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = static_cast<int>(lane_id());
    const long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    uint32_t key[PER], most = 0u;
    float x[PER];
    load_logits<KIND, PER, 32, WHOLE>(x, p.logits, t * p.experts, lane, p.experts);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        key[i] = key_of<KIND>(x[i], expert_of<PER, 32, WHOLE>(lane, i));
        most = max(most, key[i]);
    }
    const float best = value_of<KIND>(__reduce_max_sync(0xffffffffu, most));
    float all = p.mode == ROUTE_ALL ? lanes_sum<32>(exp_sum(x, best)) : 0.0f;
    uint32_t mine = 0u;   // this lane's choice
    int mine_id = -1;
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < PER; ++i) m = max(m, key[i]);
        const uint32_t top = __reduce_max_sync(0xffffffffu, m);
        if (top < kLeast) break;
        // the lowest expert that has it
        uint32_t e = 0xffffffffu;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if (key[i] == top) e = static_cast<uint32_t>(expert_of<PER, 32, WHOLE>(lane, i));
        const int id = static_cast<int>(__reduce_min_sync(0xffffffffu, e));
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (expert_of<PER, 32, WHOLE>(lane, i) == id) key[i] = 0u;
        if (lane == j) mine = top, mine_id = id;
    }
    const float w = mine ? share_of(value_of<KIND>(mine), best, p.mode) : 0.0f;
    if (p.mode != ROUTE_ALL) all = lanes_sum<32>(w);
    if (lane < p.top_k) write_choice(p, t, lane, mine != 0u, mine_id, w, all);
}

// With w = softmax of the scores over the chosen (ALL: over all experts):
// dl_i = w_i (dw_i - sum_j w_j dw_j) u'(l_i), dw = 0 where nothing was chosen.
template <int KIND, int PER, int G, bool WHOLE>
__global__ void __launch_bounds__(32 * kRouteWarps) route_grad_kernel(const RouteParams p)
{
    constexpr int kTokens = 32 * kRouteWarps / G;   // of a CTA
    __shared__ __align__(16) float gradient[kTokens][G * PER];   // dweights by expert
    __shared__ uint32_t chosen[kTokens][G];                      // by lane, a bit per logit of it
    pdl_launch_dependents();
    pdl_wait();
    const int sub = static_cast<int>(lane_id()) % G, mine = static_cast<int>(threadIdx.x) / G;
    const long long t = static_cast<long long>(blockIdx.x) * kTokens + mine;
    const bool there = t < p.tokens;
    float x[PER];
    load_logits<KIND, PER, G, WHOLE>(x, p.logits, (there ? t : p.tokens - 1) * p.experts, sub, p.experts);
    chosen[mine][sub] = 0u;
    __syncwarp();
    // (a token's ids differ; were one there twice, its dweights would add up)
    for (int j0 = 0; j0 < p.top_k; j0 += G) {
        int id = -1;
        float d = 0.0f;
        if (there && j0 + sub < p.top_k) {
            id = ld_global(p.ids + t * p.top_k + j0 + sub);
            d = ld_global(p.dweights + t * p.top_k + j0 + sub);
        }
        const bool counts = id >= 0 && id < p.experts;
        const int lane = WHOLE ? id / PER : id % G, place = WHOLE ? id % PER : id / G;
        const uint32_t bit = counts ? 1u << place : 0u;
        const bool again = counts && (atomicOr(&chosen[mine][lane], bit) & bit);
        if (counts && !again) gradient[mine][lane * PER + place] = d;
        __syncwarp();
        if (again) atomicAdd(&gradient[mine][lane * PER + place], d);
        __syncwarp();
    }
    const uint32_t in = chosen[mine][sub], counted = p.mode == ROUTE_ALL ? 0xffffffffu : in;
    float g[PER], best = kNothing;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (!(counted >> i & 1u)) x[i] = kNothing;
        best = fmaxf(best, x[i]);
        g[i] = (in >> i & 1u) && x[i] > kNothing ? gradient[mine][sub * PER + i] : 0.0f;
    }
    best = fmaxf(lanes_max<G>(best), -kMaxFinite);
    float all = 0.0f, inner = 0.0f, w[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        w[i] = share_of(x[i], best, p.mode);   // (0 of -infinity)
        all += w[i];
        inner = fmaf(w[i], g[i], inner);
    }
    all = lanes_sum<G>(all);
    const float scale = all > 0.0f ? rcp_fast(all) : 0.0f;
    inner = lanes_sum<G>(inner) * scale;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        // (a logit that nothing depends on has none, also where a dweight is infinite)
        w[i] = x[i] > kNothing ? w[i] * scale * (g[i] - inner) : 0.0f;
        if (p.mode == ROUTE_SIGMOID) w[i] *= rcp_fast(1.0f + exp_fast(x[i]));
    }
    if (!there) return;
    const int e0 = sub * PER;
    const long long at = t * p.experts + (WHOLE ? e0 : sub);
    if constexpr (KIND == 3) {
        float *out = static_cast<float *>(p.dlogits) + at;
        if constexpr (WHOLE && PER >= 4) {
#pragma unroll
            for (int i = 0; i < PER / 4; ++i)
                if (e0 < p.experts) reinterpret_cast<float4 *>(out)[i] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (expert_of<PER, G, WHOLE>(sub, i) < p.experts) out[WHOLE ? i : G * i] = w[i];
        }
    } else {
        uint16_t *out = static_cast<uint16_t *>(p.dlogits) + at;
        if constexpr (WHOLE && PER >= 4) {
#pragma unroll
            for (int i = 0; i < PER / 4; ++i)
                if (e0 < p.experts)
                    reinterpret_cast<uint2 *>(out)[i] = make_uint2(pack2f<KIND>(w[4 * i], w[4 * i + 1]), pack2f<KIND>(w[4 * i + 2], w[4 * i + 3]));
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (expert_of<PER, G, WHOLE>(sub, i) < p.experts) out[WHOLE ? i : G * i] = static_cast<uint16_t>(pack2f<KIND>(w[i], 0.0f));
        }
    }
}

template <int KIND, int PER, int G>
cudaError_t go(bool grad, const RouteParams &p, cudaStream_t stream, bool overlap)
{
    // (a lane's logits at once: up to 16 bytes at a time)
    constexpr uintptr_t kBytes = PER * (KIND == 3 ? 4 : 2), kAlign = kBytes < 16 ? kBytes : 16;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(p.dlogits);
    const bool whole = p.experts % PER == 0 && at % kAlign == 0;
    constexpr int64_t kTokens = 32 * kRouteWarps / G;
    const dim3 grid(static_cast<unsigned>((p.tokens + kTokens - 1) / kTokens));
    const auto run = [&](auto kernel) { return launch_kernel(kernel, grid, 32 * kRouteWarps, 0, 1, stream, overlap, p); };
    if (grad) return whole ? run(route_grad_kernel<KIND, PER, G, true>) : run(route_grad_kernel<KIND, PER, G, false>);
    if constexpr (G < 32 && KIND != 3) return whole ? run(route_lanes_kernel<KIND, PER, G, true>) : run(route_lanes_kernel<KIND, PER, G, false>);
    else if constexpr (G < 32) return cudaErrorInvalidValue;   // (not picked)
    else return whole ? run(route_kernel<KIND, PER, true>) : run(route_kernel<KIND, PER, false>);
}

template <int KIND>
cudaError_t pick(bool grad, const RouteParams &p, cudaStream_t stream, bool overlap)
{
    if (grad || (KIND != 3 && p.top_k <= 8)) {
        if (p.experts <= 32) return go<KIND, 4, 8>(grad, p, stream, overlap);
        if (p.experts <= 64) return go<KIND, 4, 16>(grad, p, stream, overlap);
        if (p.experts <= 128) return go<KIND, 8, 16>(grad, p, stream, overlap);
        if (p.experts <= 256) return go<KIND, 16, 16>(grad, p, stream, overlap);
    }
    if (p.experts <= 32) return go<KIND, 1, 32>(grad, p, stream, overlap);
    if (p.experts <= 64) return go<KIND, 2, 32>(grad, p, stream, overlap);
    if (p.experts <= 128) return go<KIND, 4, 32>(grad, p, stream, overlap);
    if (p.experts <= 256) return go<KIND, 8, 32>(grad, p, stream, overlap);
    if (p.experts <= 512) return go<KIND, 16, 32>(grad, p, stream, overlap);
    return go<KIND, 32, 32>(grad, p, stream, overlap);
}

cudaError_t run(bool grad, int kind, const RouteParams &p, cudaStream_t stream, bool overlap)
{
    if (kind == 0) return pick<0>(grad, p, stream, overlap);
    if (kind == 1) return pick<1>(grad, p, stream, overlap);
    return pick<3>(grad, p, stream, overlap);
}

}  // namespace

cudaError_t launch_route(int kind, const RouteParams &p, cudaStream_t stream, bool overlap) { return run(false, kind, p, stream, overlap); }
cudaError_t launch_route_grad(int kind, const RouteParams &p, cudaStream_t stream, bool overlap) { return run(true, kind, p, stream, overlap); }

}  // namespace pts
