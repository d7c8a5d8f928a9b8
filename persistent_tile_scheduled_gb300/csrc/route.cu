// A router's choice: each token's top_k experts and their weights, and the
// gradient of its logits.
//
// A warp per token; lane l holds the logits of experts l, l + 32, ... in
// registers.  The top_k are taken one by one: the largest key of the warp
// (redux.sync on keys that order like the values), then the lowest index that
// has it.  Lane j keeps the j-th choice, so the softmax over the chosen is a
// reduction over lanes.
#include "activation.cuh"
#include "launch.cuh"
#include "layer_launch.h"
#include "ptx.cuh"

namespace pts {

namespace {

enum : int { ROUTE_SELECTED = 0, ROUTE_ALL = 1, ROUTE_SIGMOID = 2 };

constexpr int kRouteWarps = 4;
constexpr float kMaxFinite = 3.402823466e38f;

// Unsigned keys in the order of the values; 0 where there is nothing to choose
// (-infinity, NaN).  -0 and 0 are one value, +infinity is the largest finite one.
__device__ __forceinline__ uint32_t key_of(float v)
{
    if (!(v >= -kMaxFinite)) return 0u;
    const uint32_t b = __float_as_uint(fminf(v, kMaxFinite) + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

template <int KIND>
__device__ __forceinline__ float load_logit(const void *p, long long i)
{
    if constexpr (KIND == 3) return ld_global(static_cast<const float *>(p) + i);
    else return unpack1<KIND>(ld_global(static_cast<const uint16_t *>(p) + i));
}

// What the softmax is taken of.
__device__ __forceinline__ float score(float l, int mode)
{
    l = fminf(l, kMaxFinite);
    return mode == ROUTE_SIGMOID ? fminf(l, 0.0f) - log1pf(expf(-fabsf(l))) : l;   // (log sigmoid)
}

// PER: logits per lane
template <int KIND, int PER>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = static_cast<int>(lane_id());
    const long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    const long long row = t * p.experts;
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < p.experts ? key_of(load_logit<KIND>(p.logits, row + e)) : 0u;
    }
    float best = 0.0f, all = 0.0f;
    if (p.mode == ROUTE_ALL) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < PER; ++i) m = max(m, key[i]);
        best = value_of(__reduce_max_sync(0xffffffffu, m));
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i]) all += expf(value_of(key[i]) - best);
        all = warp_sum(all);
    }
    uint32_t mine = 0u;   // this lane's choice
    int mine_id = -1;
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t m = 0u;
        int e = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > m) m = key[i], e = lane + 32 * i;
        const uint32_t top = __reduce_max_sync(0xffffffffu, m);
        if (top == 0u) break;
        const int id = static_cast<int>(__reduce_min_sync(0xffffffffu, m == top ? static_cast<uint32_t>(e) : 0xffffffffu));
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i == id) key[i] = 0u;
        if (lane == j) mine = top, mine_id = id;
    }
    const float u = mine ? score(value_of(mine), p.mode) : 0.0f;
    if (p.mode != ROUTE_ALL) best = __shfl_sync(0xffffffffu, u, 0);   // (the scores descend as the values do)
    const float w = mine ? expf(u - best) : 0.0f;
    if (p.mode != ROUTE_ALL) all = warp_sum(w);
    if (lane < p.top_k) {
        p.ids[t * p.top_k + lane] = mine_id;
        p.weights[t * p.top_k + lane] = mine ? w / all : 0.0f;
    }
}

// With w = softmax of the scores: dl_i = w_i (dw_i - sum_j w_j dw_j) u'(l_i).
template <int KIND, int PER>
__global__ void __launch_bounds__(32 * kRouteWarps) route_grad_kernel(const RouteParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = static_cast<int>(lane_id());
    const long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    const long long row = t * p.experts;
    // this lane's choice, its logit and gradient
    int id = -1;
    float l = 0.0f, dw = 0.0f;
    if (lane < p.top_k) {
        id = ld_global(p.ids + t * p.top_k + lane);
        if (id < 0 || id >= p.experts) id = -1;
        if (id >= 0) {
            const uint32_t k = key_of(load_logit<KIND>(p.logits, row + id));
            l = value_of(k);
            dw = ld_global(p.dweights + t * p.top_k + lane);
            if (k == 0u) id = -1;
        }
    }
    float out[PER];
    if (p.mode == ROUTE_ALL) {
        float prob[PER], best = 0.0f, all = 0.0f;
        uint32_t key[PER], m = 0u;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            key[i] = e < p.experts ? key_of(load_logit<KIND>(p.logits, row + e)) : 0u;
            m = max(m, key[i]);
        }
        best = value_of(__reduce_max_sync(0xffffffffu, m));
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            prob[i] = key[i] ? expf(value_of(key[i]) - best) : 0.0f;
            all += prob[i];
            out[i] = 0.0f;
        }
        all = warp_sum(all);
        const float scale = all > 0.0f ? 1.0f / all : 0.0f;
        const float inner = warp_sum(id >= 0 ? expf(l - best) * scale * dw : 0.0f);
        for (int j = 0; j < p.top_k; ++j) {
            const int e = __shfl_sync(0xffffffffu, id, j);
            const float d = __shfl_sync(0xffffffffu, dw, j);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i == e) out[i] += d;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) out[i] = prob[i] * scale * (out[i] - inner);
    } else {
        const float u = id >= 0 ? score(l, p.mode) : -kMaxFinite;
        float best = u;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, s));
        float w = id >= 0 ? expf(u - best) : 0.0f;
        const float all = warp_sum(w);
        w = id >= 0 ? w / all : 0.0f;
        const float inner = warp_sum(id >= 0 ? w * dw : 0.0f);
        float g = id >= 0 ? w * (dw - inner) : 0.0f;
        if (p.mode == ROUTE_SIGMOID) g /= 1.0f + expf(l);
#pragma unroll
        for (int i = 0; i < PER; ++i) out[i] = 0.0f;
        for (int j = 0; j < p.top_k; ++j) {
            const int e = __shfl_sync(0xffffffffu, id, j);
            const float d = __shfl_sync(0xffffffffu, g, j);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i == e) out[i] += d;
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        if (e >= p.experts) continue;
        if constexpr (KIND == 3) static_cast<float *>(p.dlogits)[row + e] = out[i];
        else static_cast<uint16_t *>(p.dlogits)[row + e] = static_cast<uint16_t>(pack2f<KIND>(out[i], 0.0f));
    }
}

template <int KIND, int PER>
cudaError_t go(bool grad, const RouteParams &p, cudaStream_t stream, bool overlap)
{
    const dim3 grid(static_cast<unsigned>((p.tokens + kRouteWarps - 1) / kRouteWarps));
    return launch_kernel(grad ? route_grad_kernel<KIND, PER> : route_kernel<KIND, PER>, grid, 32 * kRouteWarps, 0, 1, stream, overlap, p);
}

template <int KIND>
cudaError_t pick(bool grad, const RouteParams &p, cudaStream_t stream, bool overlap)
{
    if (p.experts <= 32) return go<KIND, 1>(grad, p, stream, overlap);
    if (p.experts <= 64) return go<KIND, 2>(grad, p, stream, overlap);
    if (p.experts <= 128) return go<KIND, 4>(grad, p, stream, overlap);
    if (p.experts <= 256) return go<KIND, 8>(grad, p, stream, overlap);
    return go<KIND, 32>(grad, p, stream, overlap);
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
