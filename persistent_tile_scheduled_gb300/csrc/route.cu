// A router's choice: each token's top_k experts and their weights, and the
// gradient of its logits.
//
// A warp per token; lane l holds the logits of experts PER l .. PER l + PER - 1 in
// registers, loaded together where rows allow it.  The top_k are taken one by one:
// the largest key of the warp (redux.sync on unsigned keys that order like the
// values).  The key of a 16-bit logit holds its expert too, the lower first, so one
// reduction finds both; of fp32 logits the lowest lane that has the largest.  Lane
// j keeps the j-th choice, so the softmax over the chosen is a sum over lanes.  The
// gradient brings dweights to the lanes that own their logits through shared memory.
//
// Instructions bound it, 320 a token (an integer one takes a scheduler two cycles):
// 16384 tokens, 8 of 128 experts, bf16 (4 MB in, 1 MB out), 6.4 us and 5.9 back; 16
// tokens 1.5, a launch.
#include "activation.cuh"
#include "launch.cuh"
#include "layer_launch.h"
#include "ptx.cuh"

namespace pts {

namespace {

enum : int { ROUTE_SELECTED = 0, ROUTE_ALL = 1, ROUTE_SIGMOID = 2 };

constexpr int kRouteWarps = 4;
constexpr float kMaxFinite = 3.402823466e38f;
constexpr uint32_t kIndex = 0x1FFFu;   // of a 16-bit logit's fp32 bits the lowest 13 are 0: they hold the expert

// Unsigned keys in the order of the values, 0 where there is nothing to choose
// (-infinity, NaN).  -0 and 0 are one value, +infinity is the largest finite one.
__device__ __forceinline__ uint32_t ordered(float v)   // v: finite
{
    const uint32_t b = __float_as_uint(v);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float unordered(uint32_t key)
{
    return __uint_as_float(key ^ (static_cast<uint32_t>(~static_cast<int32_t>(key) >> 31) | 0x80000000u));
}

template <int KIND>
__device__ __forceinline__ uint32_t key_of(float v, int e)
{
    const bool there = v >= -kMaxFinite;
    if constexpr (KIND == 3) return there ? ordered(fminf(v, kMaxFinite) + 0.0f) : 0u;
    constexpr float kMost = 3.40261e38f;   // (above both types' finite values; its lowest 13 bits are cleared)
    return there ? (ordered(fminf(v, kMost) + 0.0f) & ~kIndex) | (kIndex - static_cast<uint32_t>(e)) : 0u;
}

template <int KIND>
__device__ __forceinline__ float value_of(uint32_t key)
{
    // (of a negative value the key's bits are the complement: the expert's place is filled with ones)
    if constexpr (KIND != 3) key = key & 0x80000000u ? key & ~kIndex : key | kIndex;
    return unordered(key);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

// A lane's PER logits of a row as keys; `whole`: rows are a multiple of PER long and
// aligned to PER logits.
template <int KIND, int PER>
__device__ __forceinline__ void load_keys(uint32_t (&key)[PER], const void *logits, long long row, int experts, bool whole)
{
    const int e0 = static_cast<int>(lane_id()) * PER;
    constexpr int kBytes = PER * (KIND == 3 ? 4 : 2);
    if (whole) {
        uint32_t v[(kBytes + 3) / 4] = {};
        if (e0 < experts) {
            const uint8_t *at = static_cast<const uint8_t *>(logits) + (row + e0) * (KIND == 3 ? 4 : 2);
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
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float x;
            if constexpr (KIND == 3) x = __uint_as_float(v[i]);
            else x = i % 2 ? unpack2<KIND>(v[i / 2]).y : unpack2<KIND>(v[i / 2]).x;
            key[i] = key_of<KIND>(x, e0 + i);
            if (e0 >= experts) key[i] = 0u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            key[i] = 0u;
            if (e0 + i >= experts) continue;
            if constexpr (KIND == 3) key[i] = key_of<KIND>(ld_global(static_cast<const float *>(logits) + row + e0 + i), e0 + i);
            else key[i] = key_of<KIND>(unpack1<KIND>(ld_global(static_cast<const uint16_t *>(logits) + row + e0 + i)), e0 + i);
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

__device__ __forceinline__ void order(uint32_t &a, uint32_t &b)
{
    const uint32_t hi = max(a, b), lo = min(a, b);
    a = hi, b = lo;
}

// PER: logits per lane, TOKENS: tokens of a warp
template <int KIND, int PER, int TOKENS>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteParams p, bool whole)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = static_cast<int>(lane_id());
    const long long first = (static_cast<long long>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5)) * TOKENS;
    uint32_t key[TOKENS][PER];
    float best[TOKENS], all[TOKENS];
#pragma unroll
    for (int q = 0; q < TOKENS; ++q)   // (behind the last token: the last again, not written)
        load_keys<KIND, PER>(key[q], p.logits, (first + q < p.tokens ? first + q : p.tokens - 1) * p.experts, p.experts, whole);
    if (p.mode == ROUTE_ALL) {
#pragma unroll
        for (int q = 0; q < TOKENS; ++q) {
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < PER; ++i) m = max(m, key[q][i]);
            best[q] = value_of<KIND>(__reduce_max_sync(0xffffffffu, m));
            all[q] = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) all[q] += key[q][i] ? exp_fast(value_of<KIND>(key[q][i]) - best[q]) : 0.0f;
            all[q] = warp_sum(all[q]);
        }
    }
    uint32_t mine[TOKENS];   // this lane's choice
    int mine_id[TOKENS];
    // (the keys of a lane in descending order: the largest is the first, and is popped)
    constexpr bool kSorted = KIND != 3 && PER <= 4;
#pragma unroll
    for (int q = 0; q < TOKENS; ++q) {
        mine[q] = 0u, mine_id[q] = -1;
        if constexpr (kSorted && PER >= 2) {
            order(key[q][0], key[q][1]);
            if constexpr (PER == 4) {
                order(key[q][2], key[q][3]);
                order(key[q][0], key[q][2]);
                order(key[q][1], key[q][3]);
                order(key[q][1], key[q][2]);
            }
        }
    }
    for (int j = 0; j < p.top_k; ++j) {
#pragma unroll
        for (int q = 0; q < TOKENS; ++q) {
            uint32_t m = key[q][0];
            if constexpr (!kSorted) {
#pragma unroll
                for (int i = 1; i < PER; ++i) m = max(m, key[q][i]);
            }
            const uint32_t top = __reduce_max_sync(0xffffffffu, m);   // (0: nothing is left, and mine stays 0)
            if (lane == j) mine[q] = top;
            if constexpr (KIND == 3) {
                const int owner = __ffs(__ballot_sync(0xffffffffu, m == top)) - 1;
                int at = 0;
                bool taken = lane != owner;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (!taken && key[q][i] == top) key[q][i] = 0u, at = i, taken = true;
                const int id = __shfl_sync(0xffffffffu, lane * PER + at, owner);
                if (lane == j) mine_id[q] = id;
            } else if constexpr (kSorted) {
                if (m == top) {
#pragma unroll
                    for (int i = 0; i + 1 < PER; ++i) key[q][i] = key[q][i + 1];
                    key[q][PER - 1] = 0u;
                }
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (key[q][i] == top) key[q][i] = 0u;
            }
        }
    }
#pragma unroll
    for (int q = 0; q < TOKENS; ++q) {
        if (KIND != 3) mine_id[q] = static_cast<int>(kIndex - (mine[q] & kIndex));
        const float l = value_of<KIND>(mine[q]);
        if (p.mode != ROUTE_ALL) best[q] = __shfl_sync(0xffffffffu, l, 0);
        const float w = mine[q] ? share_of(l, best[q], p.mode) : 0.0f;
        if (p.mode != ROUTE_ALL) all[q] = warp_sum(w);
        if (lane < p.top_k && first + q < p.tokens) {
            p.ids[(first + q) * p.top_k + lane] = mine[q] ? mine_id[q] : -1;
            p.weights[(first + q) * p.top_k + lane] = mine[q] ? __fdividef(w, all[q]) : 0.0f;
        }
    }
}

// With w = softmax of the scores over the chosen (ALL: over all experts):
// dl_i = w_i (dw_i - sum_j w_j dw_j) u'(l_i), dw = 0 where nothing was chosen.
template <int KIND, int PER, int TOKENS>
__global__ void __launch_bounds__(32 * kRouteWarps) route_grad_kernel(const RouteParams p, bool whole)
{
    __shared__ __align__(16) float gradient[kRouteWarps][TOKENS][32 * PER];   // dweights by expert
    __shared__ uint32_t chosen[kRouteWarps][TOKENS][32];                      // by lane, a bit per logit of it
    pdl_launch_dependents();
    pdl_wait();
    const int lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x >> 5);
    const long long first = (static_cast<long long>(blockIdx.x) * kRouteWarps + warp) * TOKENS;
    uint32_t key[TOKENS][PER];
    int id[TOKENS];
    float d[TOKENS];
#pragma unroll
    for (int q = 0; q < TOKENS; ++q) {
        const bool there = first + q < p.tokens;
        load_keys<KIND, PER>(key[q], p.logits, (there ? first + q : p.tokens - 1) * p.experts, p.experts, whole);
        id[q] = -1, d[q] = 0.0f;
        if (there && lane < p.top_k) {
            id[q] = ld_global(p.ids + (first + q) * p.top_k + lane);
            d[q] = ld_global(p.dweights + (first + q) * p.top_k + lane);
        }
        chosen[warp][q][lane] = 0u;
    }
    __syncwarp();
    bool again[TOKENS];   // (a token's ids differ; were one there twice, its dweights would add up)
#pragma unroll
    for (int q = 0; q < TOKENS; ++q) {
        again[q] = false;
        if (id[q] < 0 || id[q] >= p.experts) continue;
        const uint32_t bit = 1u << (id[q] % PER);
        again[q] = atomicOr(&chosen[warp][q][id[q] / PER], bit) & bit;
        if (!again[q]) gradient[warp][q][id[q]] = d[q];
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < TOKENS; ++q)
        if (again[q]) atomicAdd(&gradient[warp][q][id[q]], d[q]);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < TOKENS; ++q) {
        const uint32_t in = chosen[warp][q][lane];
        float w[PER], g[PER];
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (p.mode != ROUTE_ALL && !(in >> i & 1u)) key[q][i] = 0u;   // (those that do not count)
            g[i] = key[q][i] && (in >> i & 1u) ? gradient[warp][q][lane * PER + i] : 0.0f;
            m = max(m, key[q][i]);
        }
        const float best = value_of<KIND>(__reduce_max_sync(0xffffffffu, m));
        float all = 0.0f, inner = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            w[i] = key[q][i] ? share_of(value_of<KIND>(key[q][i]), best, p.mode) : 0.0f;
            all += w[i];
            inner = fmaf(w[i], g[i], inner);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
            all += __shfl_xor_sync(0xffffffffu, all, s);
            inner += __shfl_xor_sync(0xffffffffu, inner, s);
        }
        const float scale = all > 0.0f ? __fdividef(1.0f, all) : 0.0f;
        inner *= scale;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            w[i] = w[i] * scale * (g[i] - inner);
            if (p.mode == ROUTE_SIGMOID && key[q][i]) w[i] *= rcp_fast(1.0f + exp_fast(value_of<KIND>(key[q][i])));
        }
        const int e0 = lane * PER;
        if (first + q >= p.tokens || e0 >= p.experts) continue;
        const long long at = (first + q) * p.experts + e0;
        if constexpr (KIND == 3) {
            float *out = static_cast<float *>(p.dlogits) + at;
            if (whole && PER >= 4) {
#pragma unroll
                for (int i = 0; i < PER / 4; ++i) reinterpret_cast<float4 *>(out)[i] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (e0 + i < p.experts) out[i] = w[i];
            }
        } else {
            uint16_t *out = static_cast<uint16_t *>(p.dlogits) + at;
            if (whole && PER >= 4) {
#pragma unroll
                for (int i = 0; i < PER / 4; ++i)
                    reinterpret_cast<uint2 *>(out)[i] = make_uint2(pack2f<KIND>(w[4 * i], w[4 * i + 1]), pack2f<KIND>(w[4 * i + 2], w[4 * i + 3]));
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (e0 + i < p.experts) out[i] = static_cast<uint16_t>(pack2f<KIND>(w[i], 0.0f));
            }
        }
    }
}

template <int KIND, int PER>
cudaError_t go(bool grad, const RouteParams &p, cudaStream_t stream, bool overlap)
{
    // (a lane's logits at once: up to 16 bytes at a time)
    constexpr uintptr_t kBytes = PER * (KIND == 3 ? 4 : 2), kAlign = kBytes < 16 ? kBytes : 16;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(p.dlogits);
    const bool whole = p.experts % PER == 0 && at % kAlign == 0;
    const auto run = [&](auto kernel, int tokens) {
        const int64_t each = kRouteWarps * tokens;
        return launch_kernel(kernel, dim3(static_cast<unsigned>((p.tokens + each - 1) / each)), 32 * kRouteWarps, 0, 1, stream, overlap, p, whole);
    };
    // (16384 tokens, 2 of 8 experts, and back: two tokens to a warp 7.8 us, one 8.7; 8 of 128 14.1 and 13.2)
    constexpr int kTokens = PER <= 2 ? 2 : 1;
    if (p.tokens <= 4096) return grad ? run(route_grad_kernel<KIND, PER, 1>, 1) : run(route_kernel<KIND, PER, 1>, 1);
    return grad ? run(route_grad_kernel<KIND, PER, kTokens>, kTokens) : run(route_kernel<KIND, PER, kTokens>, kTokens);
}

template <int KIND>
cudaError_t pick(bool grad, const RouteParams &p, cudaStream_t stream, bool overlap)
{
    if (p.experts <= 32) return go<KIND, 1>(grad, p, stream, overlap);
    if (p.experts <= 64) return go<KIND, 2>(grad, p, stream, overlap);
    if (p.experts <= 128) return go<KIND, 4>(grad, p, stream, overlap);
    if (p.experts <= 256) return go<KIND, 8>(grad, p, stream, overlap);
    if (p.experts <= 512) return go<KIND, 16>(grad, p, stream, overlap);
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
