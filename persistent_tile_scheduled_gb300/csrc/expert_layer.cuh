// A whole layer of experts for a few tokens: two kernels that stream the weights
// of the experts that some token chose, once, from memory into registers.
//
//   up     h[t, j] = act(W1_e x[t] + b1_e)                  e = ids[t, j]
//   down   y[t] = res[t] + sum_j w[t, j] (W2_e h[t, j] + b2_e)
//
// The tokens of an expert, up to 16 at a time (a block), are the M side of
// mma.sync, 8 rows of the weights its N side.  The contraction's order is free as
// long as both operands take the same one, so a lane loads 16 contiguous bytes
// of its row, 8 values, and feeds them to two instructions; the weights need no
// shared memory, no shuffles and no conversion.  Sorting is not needed either:
// 64 tokens are 64 bits, and an expert's tokens the bits that its mask has.
#pragma once
#include "activation.cuh"
#include "launch.cuh"
#include "layer_launch.h"
#include "ptx.cuh"

namespace pts {

constexpr int kLayerThreads = 256;
constexpr int kLayerWarps = kLayerThreads / 32;
constexpr int kLayerBlock = 16;                // tokens of a block

// Blocks that tokens * top_k assignments over the experts can make.
__host__ __device__ constexpr int layer_max_blocks(int assignments, int experts)
{
    return (assignments < experts ? assignments : experts) + assignments / kLayerBlock;
}

// The blocks of the experts' tokens, made by every CTA for itself in shared memory.
struct LayerBlocks {
    unsigned long long *mask;   // [experts]: the tokens that chose it
    float *weight;              // [blocks][16]: a token's weight (the sum, if it names the expert more than once)
    uint32_t *expert;           // [blocks]: the expert, and from bit 16 on the tokens
    uint16_t *row;              // [blocks][16]: its row of Hs (the first that names the expert)
    uint8_t *token;             // [blocks][16]
    int *count;                 // blocks

    __host__ __device__ static constexpr size_t bytes(int blocks, int experts)
    {
        return static_cast<size_t>(experts) * 8 + static_cast<size_t>(blocks) * (64 + 4 + 32 + 16) + 16;
    }

    __device__ LayerBlocks(uint8_t *at, int blocks, int experts)
    {
        mask = reinterpret_cast<unsigned long long *>(at);
        weight = reinterpret_cast<float *>(mask + experts);
        expert = reinterpret_cast<uint32_t *>(weight + blocks * kLayerBlock);
        count = reinterpret_cast<int *>(expert + blocks);
        row = reinterpret_cast<uint16_t *>(count + 4);
        token = reinterpret_cast<uint8_t *>(row + blocks * kLayerBlock);
    }

    // By the whole CTA.
    __device__ void make(const LayerParams &p) const
    {
        const int n = p.tokens * p.top_k;
        for (int e = threadIdx.x; e < p.experts; e += blockDim.x) mask[e] = 0ull;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int e = ld_global(p.ids + i);
            if (e >= 0 && e < p.experts) atomicOr(mask + e, 1ull << (i / p.top_k));
        }
        __syncthreads();
        if (threadIdx.x < 32) {
            const int lane = static_cast<int>(threadIdx.x);
            int before = 0;
            for (int e0 = 0; e0 < p.experts; e0 += 32) {
                const int tokens = e0 + lane < p.experts ? __popcll(mask[e0 + lane]) : 0;
                const int mine = (tokens + kLayerBlock - 1) / kLayerBlock;
                int incl = mine;
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, incl, s);
                    if (lane >= s) incl += o;
                }
                for (int b = 0; b < mine; ++b) {
                    const int left = tokens - b * kLayerBlock;
                    // (the block's place among the expert's goes where its weights come to stand)
                    reinterpret_cast<int *>(weight)[(before + incl - mine + b) * kLayerBlock] = b;
                    expert[before + incl - mine + b] = static_cast<uint32_t>(e0 + lane) | static_cast<uint32_t>(left < kLayerBlock ? left : kLayerBlock) << 16;
                }
                before += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) *count = before;
        }
        __syncthreads();
        const int places = *count * kLayerBlock;
        for (int i0 = 0; i0 < places; i0 += blockDim.x) {   // (blockDim.x is a multiple of 16: a block's places are one warp's)
            const int i = i0 + static_cast<int>(threadIdx.x), b = i / kLayerBlock, at = i % kLayerBlock;
            const int part = i < places ? reinterpret_cast<const int *>(weight)[b * kLayerBlock] : 0;
            __syncwarp();
            if (i < places) {
                const uint32_t x = expert[b];
                const int e = static_cast<int>(x & 0xffffu);
                int t = 0, row_ = 0;
                float w = 0.0f;
                if (at < static_cast<int>(x >> 16)) {
                    unsigned long long m = mask[e];
                    for (int k = part * kLayerBlock + at; k > 0; --k) m &= m - 1;
                    t = __ffsll(static_cast<long long>(m)) - 1;
                    for (int j = p.top_k - 1; j >= 0; --j)
                        if (ld_global(p.ids + t * p.top_k + j) == e) row_ = t * p.top_k + j;
                    for (int j = 0; j < p.top_k; ++j)
                        if (ld_global(p.ids + t * p.top_k + j) == e) w += ld_global(p.weights + t * p.top_k + j);
                }
                weight[i] = w;
                row[i] = static_cast<uint16_t>(row_);
                token[i] = static_cast<uint8_t>(t);
            }
        }
        __syncthreads();
    }
};

// 16 bytes of the weights: read once, kept out of L1, which holds the tokens' rows.
__device__ __forceinline__ uint4 ld_weights(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// c += a (16 tokens x 16) . b (16 x 8 rows of the weights)
template <int KIND>
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (KIND == 0)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c += 16 tokens x 32 . 32 x 8 rows: x0, x1 a lane's 8 values of tokens g and g + 8, w of weights row g
template <int KIND>
__device__ __forceinline__ void mma_chunk(float (&c)[4], const uint4 &x0, const uint4 &x1, const uint4 &w)
{
    mma_16x8x16<KIND>(c, x0.x, x1.x, x0.y, x1.y, w.x, w.y);
    mma_16x8x16<KIND>(c, x0.z, x1.z, x0.w, x1.w, w.z, w.w);
}

constexpr int kUpChunks = 4;     // chunks of 32 of the contraction that are loaded together, of two rows of weights
constexpr int kDownChunks = 4;   // the same, of one row

// ---- up ------------------------------------------------------------------------
//
// An item is a block and 8 hidden features (their gate and up rows; without a
// gate 16 features).  The CTA's warps share the contraction.
template <int KIND, bool GATED>
__global__ void __launch_bounds__(kLayerThreads, 2) layer_up_kernel(const LayerParams p, int max_blocks)
{
    extern __shared__ __align__(16) uint8_t smem[];
    float *part = reinterpret_cast<float *>(smem);   // [2][warps][32 lanes][8]
    const LayerBlocks blocks(smem + 2 * kLayerWarps * 1024, max_blocks, p.experts);
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id()), g = lane >> 2, t4 = lane & 3;
    pdl_wait();
    // (only now: the down kernel loads weights before it waits, which whatever ran before this kernel may have written)
    pdl_launch_dependents();
    blocks.make(p);

    constexpr int kFeatures = GATED ? 8 : 16;
    const int tiles = (p.hidden + kFeatures - 1) / kFeatures, groups = (p.dim + 32 * kUpChunks - 1) / (32 * kUpChunks);
    const int items = *blocks.count * tiles;
    const uint16_t *up = static_cast<const uint16_t *>(p.up), *x = static_cast<const uint16_t *>(p.x);
    const long long hidden2 = static_cast<long long>(p.hidden) * (GATED ? 2 : 1);

    // a group's weights: rows f0 + g of the gate (or the first 8 features) and of the other
    auto load = [&](int item, int group, uint4 (&w)[2][kUpChunks]) {
        const int b = item / tiles, f = (item - b * tiles) * kFeatures + g;
        const long long e = blocks.expert[b] & 0xffffu;
        const uint16_t *first = up + (e * hidden2 + f) * p.dim, *second = first + static_cast<long long>(GATED ? p.hidden : 8) * p.dim;
        const bool two = GATED || f + 8 < p.hidden;
#pragma unroll
        for (int c = 0; c < kUpChunks; ++c) {
            const int k = (group * kUpChunks + c) * 32 + t4 * 8;
            w[0][c] = w[1][c] = make_uint4(0u, 0u, 0u, 0u);
            if (k < p.dim) {
                w[0][c] = ld_weights(first + k);
                if (two) w[1][c] = ld_weights(second + k);
            }
        }
    };

    uint4 w[2][kUpChunks];
    const int step = static_cast<int>(gridDim.x);
    int item = static_cast<int>(blockIdx.x);
    if (item < items && warp < groups) load(item, warp, w);
    for (int n = 0; item < items; item += step, ++n) {
        const int b = item / tiles, f0 = (item - b * tiles) * kFeatures;
        const int have = static_cast<int>(blocks.expert[b] >> 16);
        const uint16_t *x0 = x + static_cast<long long>(blocks.token[b * kLayerBlock + g]) * p.dim;
        const uint16_t *x1 = x + static_cast<long long>(blocks.token[b * kLayerBlock + g + 8]) * p.dim;
        float acc[2][4] = {};
        for (int group = warp; group < groups; group += kLayerWarps) {
            uint4 cur[2][kUpChunks], v0[kUpChunks], v1[kUpChunks];
#pragma unroll
            for (int c = 0; c < kUpChunks; ++c) {
                cur[0][c] = w[0][c], cur[1][c] = w[1][c];
                const int k = (group * kUpChunks + c) * 32 + t4 * 8;
                v0[c] = v1[c] = make_uint4(0u, 0u, 0u, 0u);
                if (k < p.dim) {
                    if (g < have) v0[c] = ld_global(reinterpret_cast<const uint4 *>(x0 + k));
                    if (g + 8 < have) v1[c] = ld_global(reinterpret_cast<const uint4 *>(x1 + k));
                }
            }
            if (group + kLayerWarps < groups) load(item, group + kLayerWarps, w);
            else if (item + step < items) load(item + step, warp, w);
#pragma unroll
            for (int c = 0; c < kUpChunks; ++c) {
                mma_chunk<KIND>(acc[0], v0[c], v1[c], cur[0][c]);
                mma_chunk<KIND>(acc[1], v0[c], v1[c], cur[1][c]);
            }
        }
        // over the warps: [lane][token half][set][feature of the pair]
        float *mine = part + (n & 1) * kLayerWarps * 256;
        float4 *to = reinterpret_cast<float4 *>(mine + warp * 256 + lane * 8);
        to[0] = make_float4(acc[0][0], acc[0][1], acc[1][0], acc[1][1]);
        to[1] = make_float4(acc[0][2], acc[0][3], acc[1][2], acc[1][3]);
        __syncthreads();
        // a thread per token and pair of features (ungated: of each set of 8)
        if (threadIdx.x < 64) {
            const int from = static_cast<int>(threadIdx.x) & 31, half = static_cast<int>(threadIdx.x) >> 5;
            const int at = (from >> 2) + 8 * half, f = f0 + 2 * (from & 3);
            if (at < have) {
                float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int v = 0; v < kLayerWarps; ++v) {
                    const float4 q = *reinterpret_cast<const float4 *>(mine + v * 256 + from * 8 + half * 4);
                    s.x += q.x, s.y += q.y, s.z += q.z, s.w += q.w;
                }
                const long long e = blocks.expert[b] & 0xffffu;
                const int f2 = GATED ? p.hidden + f : f + 8;
                const bool two = GATED || f2 < p.hidden;
                if (p.up_bias) {
                    const uint16_t *bias = static_cast<const uint16_t *>(p.up_bias) + e * hidden2;
                    const float2 b0 = unpack2<KIND>(ld_global(reinterpret_cast<const uint32_t *>(bias + f)));
                    s.x += b0.x, s.y += b0.y;
                    if (two) {
                        const float2 b1 = unpack2<KIND>(ld_global(reinterpret_cast<const uint32_t *>(bias + f2)));
                        s.z += b1.x, s.w += b1.y;
                    }
                }
                uint16_t *h = static_cast<uint16_t *>(p.hs) + static_cast<long long>(blocks.row[b * kLayerBlock + at]) * p.hidden;
                with_act(p.act, [&](auto tag) {
                    constexpr int A = decltype(tag)::value;
                    if constexpr (GATED) {
                        *reinterpret_cast<uint32_t *>(h + f) = pack2f<KIND>(act<A>(s.x) * s.z, act<A>(s.y) * s.w);
                    } else {
                        *reinterpret_cast<uint32_t *>(h + f) = pack2f<KIND>(act<A>(s.x), act<A>(s.y));
                        if (two) *reinterpret_cast<uint32_t *>(h + f2) = pack2f<KIND>(act<A>(s.z), act<A>(s.w));
                    }
                });
            }
        }
    }
}

// ---- down ----------------------------------------------------------------------
//
// An item is 8 rows of every expert's matrix; its contraction runs over all
// blocks.  The warps take equal stretches of it.  A block's sums are added, with
// the tokens' weights and in fp32, to the warp's own sums per token in shared
// memory when the warp is through with it: an infinity in one expert's matrix
// meets only the tokens that chose it.
template <int KIND>
__global__ void __launch_bounds__(kLayerThreads, 2) layer_down_kernel(const LayerParams p, int max_blocks)
{
    extern __shared__ __align__(16) uint8_t smem[];
    float *sums = reinterpret_cast<float *>(smem);   // [warps][tokens][8]
    const LayerBlocks blocks(smem + kLayerWarps * p.tokens * 32, max_blocks, p.experts);
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id()), g = lane >> 2, t4 = lane & 3;
    pdl_launch_dependents();
    blocks.make(p);   // (ids and weights were there before the up kernel began)

    const int tiles = (p.dim + 7) / 8, groups = (p.hidden + 32 * kDownChunks - 1) / (32 * kDownChunks);
    const int all = *blocks.count * groups;
    const int first = static_cast<int>(static_cast<long long>(all) * warp / kLayerWarps);
    const int end = static_cast<int>(static_cast<long long>(all) * (warp + 1) / kLayerWarps);
    const uint16_t *down = static_cast<const uint16_t *>(p.down), *hs = static_cast<const uint16_t *>(p.hs);
    float *mine = sums + warp * p.tokens * 8;

    auto load = [&](int tile, int at, uint4 (&w)[kDownChunks]) {
        const int b = at / groups, group = at - b * groups;
        const long long e = blocks.expert[b] & 0xffffu;
        const uint16_t *row = down + (e * p.dim + tile * 8 + g) * p.hidden;
#pragma unroll
        for (int c = 0; c < kDownChunks; ++c) {
            const int k = (group * kDownChunks + c) * 32 + t4 * 8;
            w[c] = k < p.hidden ? ld_weights(row + k) : make_uint4(0u, 0u, 0u, 0u);
        }
    };

    uint4 w[kDownChunks];
    if (static_cast<int>(blockIdx.x) < tiles && first < end) load(static_cast<int>(blockIdx.x), first, w);
    pdl_wait();   // the hidden rows
    for (int tile = static_cast<int>(blockIdx.x); tile < tiles; tile += static_cast<int>(gridDim.x)) {
        for (int i = lane; i < p.tokens * 8; i += 32) mine[i] = 0.0f;
        __syncwarp();
        float acc[4] = {};
        for (int at = first; at < end; ++at) {
            const int b = at / groups, group = at - b * groups;
            const int have = static_cast<int>(blocks.expert[b] >> 16);
            const uint16_t *h0 = hs + static_cast<long long>(blocks.row[b * kLayerBlock + g]) * p.hidden;
            const uint16_t *h1 = hs + static_cast<long long>(blocks.row[b * kLayerBlock + g + 8]) * p.hidden;
            uint4 cur[kDownChunks], v0[kDownChunks], v1[kDownChunks];
#pragma unroll
            for (int c = 0; c < kDownChunks; ++c) {
                cur[c] = w[c];
                const int k = (group * kDownChunks + c) * 32 + t4 * 8;
                v0[c] = v1[c] = make_uint4(0u, 0u, 0u, 0u);
                if (k < p.hidden) {
                    if (g < have) v0[c] = ld_global(reinterpret_cast<const uint4 *>(h0 + k));
                    if (g + 8 < have) v1[c] = ld_global(reinterpret_cast<const uint4 *>(h1 + k));
                }
            }
            if (at + 1 < end) load(tile, at + 1, w);
            else if (tile + static_cast<int>(gridDim.x) < tiles) load(tile + static_cast<int>(gridDim.x), first, w);
#pragma unroll
            for (int c = 0; c < kDownChunks; ++c) mma_chunk<KIND>(acc, v0[c], v1[c], cur[c]);
            if (group + 1 == groups || at + 1 == end) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int i = b * kLayerBlock + g + 8 * half;
                    if (g + 8 * half < have) {
                        float2 *to = reinterpret_cast<float2 *>(mine + blocks.token[i] * 8 + 2 * t4);
                        const float f = blocks.weight[i];
                        float2 s = *to;
                        s.x = fmaf(f, acc[2 * half], s.x);
                        s.y = fmaf(f, acc[2 * half + 1], s.y);
                        *to = s;
                    }
                    acc[2 * half] = acc[2 * half + 1] = 0.0f;
                }
            }
        }
        __syncthreads();
        for (int i = static_cast<int>(threadIdx.x); i < p.tokens * 4; i += kLayerThreads) {
            const int t = i >> 2;
            const long long n = static_cast<long long>(tile) * 8 + 2 * (i & 3);
            float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int v = 0; v < kLayerWarps; ++v) {
                const float2 q = *reinterpret_cast<const float2 *>(sums + (v * p.tokens + t) * 8 + 2 * (i & 3));
                s.x += q.x, s.y += q.y;
            }
            if (p.down_bias)
                for (int j = 0; j < p.top_k; ++j) {
                    const int e = ld_global(p.ids + t * p.top_k + j);
                    if (e < 0 || e >= p.experts) continue;
                    const float f = ld_global(p.weights + t * p.top_k + j);
                    const float2 q = unpack2<KIND>(ld_global(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.down_bias) + static_cast<long long>(e) * p.dim + n)));
                    s.x = fmaf(f, q.x, s.x);
                    s.y = fmaf(f, q.y, s.y);
                }
            if (p.residual) {
                const float2 q = unpack2<KIND>(ld_global(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.residual) + t * static_cast<long long>(p.dim) + n)));
                s.x += q.x, s.y += q.y;
            }
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.y) + t * static_cast<long long>(p.dim) + n) = pack2f<KIND>(s.x, s.y);
        }
        __syncthreads();
    }
}

template <class... P>
cudaError_t launch_layer_kernel(void (*kernel)(P...), long long items, size_t smem, int blocks, const LayerParams &p, cudaStream_t stream, bool overlap)
{
    // (the limit is the function's: always the most that any call needs)
    constexpr int kMostSmem = 96 * 1024;
    static_assert(LayerBlocks::bytes(layer_max_blocks(kLayerMaxAssignments, kLayerMaxExperts), kLayerMaxExperts)
                  + 2 * kLayerWarps * 1024 <= kMostSmem && kLayerMaxTokens * 32 <= 2 * 1024, "");
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e != cudaSuccess) return e;
    }
    const long long grid = items < 2 * p.sms ? items : 2 * p.sms;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(grid)), kLayerThreads, smem, 1, stream, overlap, p, blocks);
}

template <int KIND>
cudaError_t launch_layer(const LayerParams &p, cudaStream_t stream, bool overlap)
{
    const int n = p.tokens * p.top_k, blocks = layer_max_blocks(n, p.experts);
    const bool gated = p.act & ACT_GATED;
    const size_t tables = LayerBlocks::bytes(blocks, p.experts);
    if (p.hidden > 0) {
        const int features = gated ? 8 : 16;
        const long long items = static_cast<long long>(blocks) * ((p.hidden + features - 1) / features);
        const cudaError_t e = launch_layer_kernel(gated ? layer_up_kernel<KIND, true> : layer_up_kernel<KIND, false>, items,
                                                  2 * kLayerWarps * 1024 + tables, blocks, p, stream, overlap);
        if (e != cudaSuccess) return e;
    }
    // (without an up kernel before it nothing may be read early)
    return launch_layer_kernel(layer_down_kernel<KIND>, (p.dim + 7) / 8, kLayerWarps * p.tokens * 32 + tables, blocks, p, stream,
                               overlap && p.hidden > 0);
}

}  // namespace pts
