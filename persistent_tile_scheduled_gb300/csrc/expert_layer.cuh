// A whole layer of experts for a few tokens: two kernels that stream the weights
// of the experts that some token chose, once, from memory into registers.
//
//   up     h[t, j] = act(W1_e x[t] + b1_e)                  e = ids[t, j]
//   down   y[t] = res[t] + sum_j w[t, j] (W2_e h[t, j] + b2_e)
//
// 16 rows of the weights are the M side of mma.sync, 8 of an expert's tokens its
// N side; a block is 8 or 16 tokens of one expert.  The contraction's order is
// free as long as both operands take the same one, so a lane loads 16 contiguous
// bytes of its row, 8 values, and feeds them to two instructions: the weights need
// no shared memory, no shuffles and no conversion.  Sorting is not needed either:
// 64 tokens are 64 bits, and an expert's tokens the bits that its mask has.
#pragma once
#include "activation.cuh"
#include "launch.cuh"
#include "layer_launch.h"
#include "ptx.cuh"

namespace pts {

constexpr int kLayerThreads = 256;
constexpr int kLayerWarps = kLayerThreads / 32;
constexpr int kLayerRows = 16;                 // rows of the weights of an item
constexpr int kLayerChunks = 8;                // chunks of 32 of the contraction on their way to a warp
constexpr int kLayerAhead = 4;                 // of them, those whose tokens' values are

// Blocks of 8 * nb tokens that so many assignments to the experts can make.
__host__ __device__ constexpr int layer_max_blocks(int assignments, int experts, int nb)
{
    return (assignments < experts ? assignments : experts) + assignments / (8 * nb);
}

// The blocks of the experts' tokens (8 * NB each), made by every CTA for itself in
// shared memory.
template <int NB>
struct LayerBlocks {
    static constexpr int kBlock = 8 * NB;
    unsigned long long *mask;   // [experts]: the tokens that chose it
    float *weight;              // [blocks][kBlock]: a token's weight (the sum, if it names the expert more than once)
    uint32_t *expert;           // [blocks]: the expert, and from bit 16 on the tokens
    int32_t *ids;               // [assignments]
    int *count;                 // blocks; and behind it a sum per warp
    uint16_t *base;             // [experts]: its first block
    uint16_t *row;              // [blocks][kBlock]: its row of Hs (the first that names the expert)
    uint8_t *token;             // [blocks][kBlock]

    __host__ __device__ static constexpr size_t bytes(int blocks, int experts, int assignments)
    {
        return static_cast<size_t>(experts) * 10 + static_cast<size_t>(blocks) * (7 * kBlock + 4) + 4 * assignments + 4 * (4 + kLayerWarps);
    }

    __device__ LayerBlocks(uint8_t *at, int blocks, int experts, int assignments)
    {
        mask = reinterpret_cast<unsigned long long *>(at);
        weight = reinterpret_cast<float *>(mask + experts);
        expert = reinterpret_cast<uint32_t *>(weight + blocks * kBlock);
        ids = reinterpret_cast<int32_t *>(expert + blocks);
        count = reinterpret_cast<int *>(ids + assignments);
        base = reinterpret_cast<uint16_t *>(count + 4 + kLayerWarps);
        row = base + experts;
        token = reinterpret_cast<uint8_t *>(row + blocks * kBlock);
    }

    // By the whole CTA.
    __device__ void make(const LayerParams &p) const
    {
        const int n = p.tokens * p.top_k, lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x >> 5);
        for (int e = threadIdx.x; e < p.experts; e += kLayerThreads) mask[e] = 0ull;
        for (int i = threadIdx.x; i < n; i += kLayerThreads) {
            const int e = ld_global(p.ids + i);
            ids[i] = e >= 0 && e < p.experts ? e : -1;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kLayerThreads)
            if (ids[i] >= 0) atomicOr(mask + ids[i], 1ull << (i / p.top_k));
        __syncthreads();
        // each expert's first block: sums over the experts before it
        int carry = 0;
        for (int e0 = 0; e0 < p.experts; e0 += kLayerThreads) {
            const int e = e0 + static_cast<int>(threadIdx.x);
            const int tokens = e < p.experts ? __popcll(mask[e]) : 0, mine = (tokens + kBlock - 1) / kBlock;
            int incl = mine;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, s);
                if (lane >= s) incl += o;
            }
            if (lane == 31) count[4 + warp] = incl;
            __syncthreads();
            int before = carry;
#pragma unroll
            for (int w = 0; w < kLayerWarps; ++w) {
                const int v = count[4 + w];
                if (w < warp) before += v;
                carry += v;
            }
            const int first = before + incl - mine;
            if (mine) base[e] = static_cast<uint16_t>(first);
            for (int b = 0; b < mine; ++b) {
                const int left = tokens - b * kBlock;
                expert[first + b] = static_cast<uint32_t>(e) | static_cast<uint32_t>(left < kBlock ? left : kBlock) << 16;
            }
            __syncthreads();
        }
        if (threadIdx.x == 0) *count = carry;
        // every assignment's place: behind the lower tokens of its expert
        for (int i = threadIdx.x; i < n; i += kLayerThreads) {
            const int e = ids[i], t = i / p.top_k;
            if (e < 0) continue;
            bool again = false;
            for (int j = t * p.top_k; j < i; ++j) again |= ids[j] == e;
            if (again) continue;
            float w = ld_global(p.weights + i);
            for (int j = i + 1; j < (t + 1) * p.top_k; ++j)
                if (ids[j] == e) w += ld_global(p.weights + j);
            const int at = base[e] * kBlock + __popcll(mask[e] & ((1ull << t) - 1ull));
            weight[at] = w;
            row[at] = static_cast<uint16_t>(i);
            token[at] = static_cast<uint8_t>(t);
        }
        __syncthreads();
    }
};

// 16 bytes of the weights: read once, kept out of L1, which holds the tokens' rows.
// Memory is asked for 256 bytes of the row at a time (2 % faster than without).
__device__ __forceinline__ uint4 ld_weights(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// c += a (16 rows of the weights x 16) . b (16 x 8 tokens)
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

// Up to kLayerChunks chunks of 32 of the contraction, as a lane reads them: 8 values
// from 32 i + 8 (lane % 4) on, of rows g = lane / 4 and g + 8 of the weights and of
// tokens g, g + 8, ... (none: null).
template <int NB>
struct LayerGroup {
    const uint16_t *w[2], *x[NB];
    int n;   // chunks that this lane reads

    __device__ __forceinline__ void none()
    {
        w[0] = w[1] = nullptr;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) x[nb] = nullptr;
        n = 0;
    }
    // chunks [at, end) of rows of `width` values
    __device__ __forceinline__ void set(const uint16_t *row, const uint16_t *second, const uint16_t *const (&tokens)[NB], int at, int end, int width)
    {
        const int k = at * 32 + static_cast<int>(lane_id() & 3u) * 8, left = (width - k + 31) / 32;   // (width is a multiple of 8)
        n = end - at < left ? end - at : left;
        w[0] = row + k;
        w[1] = second ? second + k : nullptr;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) x[nb] = tokens[nb] ? tokens[nb] + k : nullptr;
    }
};

// The chunks on their way.  A chunk's registers are loaded anew as soon as it has
// been multiplied, so that 16 loads of 16 bytes are always outstanding per lane, 128
// KB per SM, whatever the groups; the tokens' values, mostly in L1, kLayerAhead
// chunks ahead.  (Whole groups of 4 chunks, loaded while the one before is
// multiplied: 40.5 us for one token through 8 experts of 4096 x 4096.)
template <int KIND, int NB>
struct LayerStream {
    uint4 w[2][kLayerChunks], x[NB][kLayerAhead];

    __device__ __forceinline__ void load_w(const LayerGroup<NB> &g, int i)
    {
        w[0][i] = w[1][i] = make_uint4(0u, 0u, 0u, 0u);
        if (i < g.n) {
            w[0][i] = ld_weights(g.w[0] + 32 * i);
            if (g.w[1]) w[1][i] = ld_weights(g.w[1] + 32 * i);
        }
    }
    __device__ __forceinline__ void load_x(const LayerGroup<NB> &g, int i)
    {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            x[nb][i % kLayerAhead] = make_uint4(0u, 0u, 0u, 0u);
            if (i < g.n && g.x[nb]) x[nb][i % kLayerAhead] = ld_global(reinterpret_cast<const uint4 *>(g.x[nb] + 32 * i));
        }
    }
    __device__ __forceinline__ void start_w(const LayerGroup<NB> &g)
    {
#pragma unroll
        for (int i = 0; i < kLayerChunks; ++i) load_w(g, i);
    }
    __device__ __forceinline__ void start_x(const LayerGroup<NB> &g)
    {
#pragma unroll
        for (int i = 0; i < kLayerAhead; ++i) load_x(g, i);
    }
    // c[nb] += the group: rows g and g + 8 of tokens 8 nb + 2 (lane % 4), + 1; and the next one's loads
    __device__ __forceinline__ void multiply(float (&c)[NB][4], const LayerGroup<NB> &group, const LayerGroup<NB> &next)
    {
#pragma unroll
        for (int i = 0; i < kLayerChunks; ++i) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const uint4 &v = x[nb][i % kLayerAhead];
                mma_16x8x16<KIND>(c[nb], w[0][i].x, w[1][i].x, w[0][i].y, w[1][i].y, v.x, v.y);
                mma_16x8x16<KIND>(c[nb], w[0][i].z, w[1][i].z, w[0][i].w, w[1][i].w, v.z, v.w);
            }
            load_w(next, i);
            if (i + kLayerAhead < kLayerChunks) load_x(group, i + kLayerAhead);
            else load_x(next, i + kLayerAhead - kLayerChunks);
        }
    }
};

// ---- up ------------------------------------------------------------------------
//
// An item is a block and 8 hidden features (their gate and up rows; without a
// gate 16 features).  The CTA's warps share the contraction.
template <int KIND, bool GATED, int NB>
__global__ void __launch_bounds__(kLayerThreads, 2) layer_up_kernel(const LayerParams p, int max_blocks)
{
    extern __shared__ __align__(16) uint8_t smem[];
    float *part = reinterpret_cast<float *>(smem);   // [kLayerWarps items][warps][NB][32 lanes][4]
    constexpr int kPart = kLayerWarps * NB * 128;
    const LayerBlocks<NB> blocks(smem + kLayerWarps * kPart * 4, max_blocks, p.experts, p.tokens * p.top_k);
    constexpr int kBlock = 8 * NB;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id()), g = lane >> 2;
    pdl_wait();
    // (only now: the down kernel loads weights before it waits, which whatever ran before this kernel may have written)
    pdl_launch_dependents();
    blocks.make(p);

    constexpr int kFeatures = GATED ? 8 : 16;
    const int tiles = (p.hidden + kFeatures - 1) / kFeatures, chunks = (p.dim + 31) / 32;
    const int first = chunks * warp / kLayerWarps, end = chunks * (warp + 1) / kLayerWarps;   // this warp's share
    const int items = *blocks.count * tiles, step = static_cast<int>(gridDim.x);
    const uint16_t *up = static_cast<const uint16_t *>(p.up), *x = static_cast<const uint16_t *>(p.x);
    const long long hidden2 = static_cast<long long>(p.hidden) * (GATED ? 2 : 1);

    auto group_of = [&](int item, int at) {
        LayerGroup<NB> group;
        if (item >= items || at >= end) {
            group.none();
            return group;
        }
        const int b = item / tiles, f = (item - b * tiles) * kFeatures + g, have = static_cast<int>(blocks.expert[b] >> 16);
        const long long e = blocks.expert[b] & 0xffffu;
        const uint16_t *row = up + (e * hidden2 + f) * p.dim, *tokens[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            tokens[nb] = 8 * nb + g < have ? x + static_cast<long long>(blocks.token[b * kBlock + 8 * nb + g]) * p.dim : nullptr;
        group.set(row, GATED || f + 8 < p.hidden ? row + static_cast<long long>(GATED ? p.hidden : 8) * p.dim : nullptr, tokens, at, end, p.dim);
        return group;
    };

    LayerStream<KIND, NB> stream;
    int item = static_cast<int>(blockIdx.x);
    LayerGroup<NB> group = group_of(item, first);
    stream.start_w(group);
    stream.start_x(group);
    for (int n = 0; item < items; item += step, ++n) {
        const int b = item / tiles, f0 = (item - b * tiles) * kFeatures;
        const int have = static_cast<int>(blocks.expert[b] >> 16);
        float acc[NB][4] = {};
        for (int at = first; at < end; at += kLayerChunks) {
            const LayerGroup<NB> next = at + kLayerChunks < end ? group_of(item, at + kLayerChunks) : group_of(item + step, first);
            stream.multiply(acc, group, next);
            group = next;
        }
        // Over the warps: one of them in turn, the others run on.  It waits for all at
        // this item, so every warp does once in kLayerWarps items: none can come back
        // to an item's place (and barrier) before its reader is through with it.
        const int turn = n % kLayerWarps;
        float *mine = part + turn * kPart;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            *reinterpret_cast<float4 *>(mine + ((warp * NB + nb) * 32 + lane) * 4) = make_float4(acc[nb][0], acc[nb][1], acc[nb][2], acc[nb][3]);
        if (warp != turn) {
            asm volatile("bar.arrive %0, %1;" ::"r"(1 + turn), "n"(kLayerThreads) : "memory");
            continue;
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + turn), "n"(kLayerThreads) : "memory");
        // a lane has rows g and g + 8 of two tokens
        for (int nb = 0; nb < NB && 8 * nb < have; ++nb) {
            float s[4] = {};
#pragma unroll
            for (int v = 0; v < kLayerWarps; ++v) {
                const float4 q = *reinterpret_cast<const float4 *>(mine + ((v * NB + nb) * 32 + lane) * 4);
                s[0] += q.x, s[1] += q.y, s[2] += q.z, s[3] += q.w;
            }
            const long long e = blocks.expert[b] & 0xffffu;
            const int f = f0 + g, f2 = GATED ? p.hidden + f : f + 8;
            const bool two = GATED || f2 < p.hidden;
            if (p.up_bias) {
                const uint16_t *bias = static_cast<const uint16_t *>(p.up_bias) + e * hidden2;
                const float b0 = unpack1<KIND>(ld_global(bias + f)), b1 = two ? unpack1<KIND>(ld_global(bias + f2)) : 0.0f;
                s[0] += b0, s[1] += b0, s[2] += b1, s[3] += b1;
            }
            with_act(p.act, [&](auto tag) {
                constexpr int A = decltype(tag)::value;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    s[i] = act<A>(s[i]);
                    if constexpr (GATED) s[i] *= s[2 + i];
                    else s[2 + i] = act<A>(s[2 + i]);
                }
            });
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = 8 * nb + 2 * (lane & 3) + i;
                if (at >= have) break;
                uint16_t *h = static_cast<uint16_t *>(p.hs) + static_cast<long long>(blocks.row[b * kBlock + at]) * p.hidden;
                const uint32_t both = pack2f<KIND>(s[i], s[2 + i]);
                h[f] = static_cast<uint16_t>(both);
                if (!GATED && two) h[f2] = static_cast<uint16_t>(both >> 16);
            }
        }
    }
}

// ---- down ----------------------------------------------------------------------
//
// An item is 16 rows of every expert's matrix; its contraction runs over all
// blocks.  The warps of a cluster's CTAs take equal stretches of it.  A block's
// sums are added, with the tokens' weights and in fp32, to the warp's own sums per
// token in shared memory when the warp is through with it: an infinity in one
// expert's matrix meets only the tokens that chose it.
constexpr int kDownPitch = 20;   // floats of a token's 16 sums (lanes of a warp meet different banks)

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t cluster_addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(cluster_addr) : "memory");
    return v;
}

template <int KIND, int NB>
__global__ void __launch_bounds__(kLayerThreads, 2) layer_down_kernel(const LayerParams p, int max_blocks, int ctas)
{
    extern __shared__ __align__(16) uint8_t smem[];
    float *sums = reinterpret_cast<float *>(smem);   // [warps][tokens][kDownPitch]
    const LayerBlocks<NB> blocks(smem + kLayerWarps * p.tokens * kDownPitch * 4, max_blocks, p.experts, p.tokens * p.top_k);
    constexpr int kBlock = 8 * NB;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id()), g = lane >> 2, t4 = lane & 3;
    const int share = static_cast<int>(blockIdx.x) % ctas, step = static_cast<int>(gridDim.x) / ctas;
    pdl_launch_dependents();
    blocks.make(p);   // (ids and weights were there before the up kernel began)

    const int tiles = (p.dim + kLayerRows - 1) / kLayerRows, chunks = (p.hidden + 31) / 32;
    const long long all = static_cast<long long>(*blocks.count) * chunks;   // block by block
    const int first = static_cast<int>(all * (share * kLayerWarps + warp) / (ctas * kLayerWarps));
    const int end = static_cast<int>(all * (share * kLayerWarps + warp + 1) / (ctas * kLayerWarps));
    const uint16_t *down = static_cast<const uint16_t *>(p.down), *hs = static_cast<const uint16_t *>(p.hs);
    float *mine = sums + warp * p.tokens * kDownPitch;

    // the chunks from `at` on, up to kLayerChunks of one block
    auto group_of = [&](int tile, int at) {
        LayerGroup<NB> group;
        if (tile >= tiles || at >= end) {
            group.none();
            return group;
        }
        const int b = at / chunks, c = at - b * chunks, n = tile * kLayerRows + g, have = static_cast<int>(blocks.expert[b] >> 16);
        const long long e = blocks.expert[b] & 0xffffu;
        const uint16_t *row = down + (e * p.dim + n) * p.hidden, *tokens[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            tokens[nb] = 8 * nb + g < have ? hs + static_cast<long long>(blocks.row[b * kBlock + 8 * nb + g]) * p.hidden : nullptr;
        group.set(row, n + 8 < p.dim ? row + 8ll * p.hidden : nullptr, tokens, c, c + end - at, p.hidden);
        return group;
    };

    LayerStream<KIND, NB> stream;
    int tile = static_cast<int>(blockIdx.x) / ctas;
    LayerGroup<NB> group = group_of(tile, first);
    stream.start_w(group);
    pdl_wait();   // the hidden rows
    stream.start_x(group);
    for (; tile < tiles; tile += step) {
        for (int i = lane; i < p.tokens * kDownPitch; i += 32) mine[i] = 0.0f;
        __syncwarp();
        float acc[NB][4] = {};
        for (int at = first; at < end;) {
            const int b = at / chunks, c = at - b * chunks;
            const int left = end - at < chunks - c ? end - at : chunks - c;   // of this block
            const int take = left < kLayerChunks ? left : kLayerChunks;
            const LayerGroup<NB> next = at + take < end ? group_of(tile, at + take) : group_of(tile + step, first);
            stream.multiply(acc, group, next);
            group = next;
            at += take;
            if (left == take) {
                const int have = static_cast<int>(blocks.expert[b] >> 16);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int place = 8 * nb + 2 * t4 + i;
                        if (place < have) {
                            float *to = mine + blocks.token[b * kBlock + place] * kDownPitch + g;
                            const float f = blocks.weight[b * kBlock + place];
                            to[0] = fmaf(f, acc[nb][i], to[0]);
                            to[8] = fmaf(f, acc[nb][2 + i], to[8]);
                        }
                        acc[nb][i] = acc[nb][2 + i] = 0.0f;
                    }
                __syncwarp();   // (another lane may have this token in the next block)
            }
        }
        __syncthreads();
        // over the warps, then over the cluster's CTAs: a thread per token and pair of rows
        for (int pass = ctas > 1 ? 0 : 1; pass < 2; ++pass) {
            for (int i = static_cast<int>(threadIdx.x) * (pass ? ctas : 1) + (pass ? share : 0); i < p.tokens * 8; i += kLayerThreads * (pass ? ctas : 1)) {
                const int t = i >> 3, at = t * kDownPitch + 2 * (i & 7);
                float2 s = make_float2(0.0f, 0.0f);
                if (pass && ctas > 1) {
                    for (int k = 0; k < ctas; ++k) {
                        const float2 q = ld_cluster_f32x2(mapa(smem_u32(sums + at), static_cast<uint32_t>(k)));
                        s.x += q.x, s.y += q.y;
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < kLayerWarps; ++v) {
                        const float2 q = *reinterpret_cast<const float2 *>(sums + v * p.tokens * kDownPitch + at);
                        s.x += q.x, s.y += q.y;
                    }
                    if (!pass) {   // (in the first warp's place, which only this thread reads)
                        *reinterpret_cast<float2 *>(sums + at) = s;
                        continue;
                    }
                }
                const long long n = static_cast<long long>(tile) * kLayerRows + 2 * (i & 7);
                if (n >= p.dim) continue;
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
            if (ctas > 1) cluster_sync();
            else __syncthreads();
        }
    }
}

template <int NB>
constexpr size_t layer_tables(int assignments, int experts)
{
    return LayerBlocks<NB>::bytes(layer_max_blocks(assignments, experts, NB), experts, assignments);
}
template <int NB>
constexpr size_t layer_smem(int tokens, int assignments, int experts)   // the larger of the two kernels'
{
    const size_t up = kLayerWarps * kLayerWarps * NB * 512, down = kLayerWarps * kDownPitch * 4 * tokens;
    return layer_tables<NB>(assignments, experts) + (up > down ? up : down);
}

template <class... P, class... A>
cudaError_t launch_layer_kernel(void (*kernel)(P...), long long items, int ctas, size_t smem, const LayerParams &p, cudaStream_t stream, bool overlap, A... args)
{
    // (the limit is the function's: always the most that any call needs)
    constexpr int kMostSmem = 150 * 1024;
    static_assert(layer_smem<1>(kLayerMaxTokens, kLayerMaxAssignments, kLayerMaxExperts) <= kMostSmem
                  && layer_smem<2>(kLayerMaxTokens, kLayerMaxAssignments, kLayerMaxExperts) <= kMostSmem, "");
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e != cudaSuccess) return e;
    }
    const long long most = 2 * p.sms / ctas, clusters = items < most ? items : most;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(clusters * ctas)), kLayerThreads, smem, ctas, stream, overlap, p, args...);
}

template <int KIND, int NB>
cudaError_t launch_layer_of(const LayerParams &p, cudaStream_t stream, bool overlap)
{
    const int n = p.tokens * p.top_k, blocks = layer_max_blocks(n, p.experts, NB);
    const bool gated = p.act & ACT_GATED;
    const size_t tables = layer_tables<NB>(n, p.experts);
    if (p.hidden > 0) {
        const int features = gated ? 8 : 16;
        const long long items = static_cast<long long>(blocks) * ((p.hidden + features - 1) / features);
        const cudaError_t e = launch_layer_kernel(gated ? layer_up_kernel<KIND, true, NB> : layer_up_kernel<KIND, false, NB>, items, 1,
                                                  kLayerWarps * kLayerWarps * NB * 512 + tables, p, stream, overlap, blocks);
        if (e != cudaSuccess) return e;
    }
    // few tiles: CTAs share one's contraction
    const long long tiles = (p.dim + kLayerRows - 1) / kLayerRows;
    int ctas = 1;
    while (ctas < 8 && tiles * ctas * 2 <= 2 * p.sms) ctas *= 2;
    // (without an up kernel before it nothing may be read early)
    return launch_layer_kernel(layer_down_kernel<KIND, NB>, tiles, ctas, kLayerWarps * p.tokens * kDownPitch * 4 + tables, p, stream,
                               overlap && p.hidden > 0, blocks, ctas);
}

template <int KIND>
cudaError_t launch_layer(const LayerParams &p, cudaStream_t stream, bool overlap)
{
    // blocks of 8 tokens where hardly an expert has more
    return p.tokens <= 8 || p.tokens * p.top_k <= 4 * p.experts ? launch_layer_of<KIND, 1>(p, stream, overlap)
                                                               : launch_layer_of<KIND, 2>(p, stream, overlap);
}

}  // namespace pts
