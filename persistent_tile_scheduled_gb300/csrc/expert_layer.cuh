// A whole layer of experts for a few tokens: two kernels that stream the weights
// of the experts that some token chose, once, from memory into registers.
//
//   up     h[t, j] = act(W1_e x[t] + b1_e)                  e = ids[t, j]
//   down   y[t] = res[t] + sum_j w[t, j] (W2_e h[t, j] + b2_e)
//
// rows_stream.cuh says how.  Sorting is not needed: 64 tokens are 64 bits, and an
// expert's tokens the bits that its mask has.
#pragma once
#include "layer_launch.h"
#include "rows_stream.cuh"

namespace pts {

constexpr int kLayerRows = 16;   // rows of the weights of a down item

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
        return static_cast<size_t>(experts) * 10 + static_cast<size_t>(blocks) * (7 * kBlock + 4) + 4 * assignments + 4 * (4 + kRowsWarps);
    }

    __device__ LayerBlocks(uint8_t *at, int blocks, int experts, int assignments)
    {
        mask = reinterpret_cast<unsigned long long *>(at);
        weight = reinterpret_cast<float *>(mask + experts);
        expert = reinterpret_cast<uint32_t *>(weight + blocks * kBlock);
        ids = reinterpret_cast<int32_t *>(expert + blocks);
        count = reinterpret_cast<int *>(ids + assignments);
        base = reinterpret_cast<uint16_t *>(count + 4 + kRowsWarps);
        row = base + experts;
        token = reinterpret_cast<uint8_t *>(row + blocks * kBlock);
    }

    // Up to 32 assignments, by one warp, a lane each, without the other way's barriers and
    // sums over the experts, for which all of the up kernel waits (with what finish adds
    // loaded early, 4 tokens, 2 of 11 experts of 872 x 560 take 10.8 us instead of 13.6):
    // experts in the order in which they are first named.
    template <bool WEIGHTS>
    __device__ __forceinline__ void make_few(const LayerParams &p, int n) const
    {
        constexpr uint32_t kAll = 0xffffffffu;
        const int i = static_cast<int>(threadIdx.x), t = i / p.top_k;
        int e = i < n ? ld_global(p.ids + i) : -1;
        float w = WEIGHTS && i < n ? ld_global(p.weights + i) : 0.0f;
        if (e < 0 || e >= p.experts) e = -1;
        const uint32_t lower = (1u << i) - 1u, same = __match_any_sync(kAll, e);
        const uint32_t own = same & (p.top_k >= 32 ? kAll : ((1u << p.top_k) - 1u) << (t * p.top_k));   // the token's that name this expert
        const bool counts = e >= 0 && !(own & lower);
        const uint32_t tokens = same & __ballot_sync(kAll, counts);   // the expert's, a lane each
        if constexpr (WEIGHTS) {
            if (__any_sync(kAll, counts && (own & ~lower & ~(1u << i)))) {
                float sum = w;
                for (int j = 1; j < 32; ++j) {
                    const float other = __shfl_sync(kAll, w, j);
                    if (j > i && (own >> j & 1u)) sum += other;
                }
                w = sum;
            }
        }
        const int place = __popc(tokens & lower), have = __popc(tokens), mine = counts && place == 0 ? (have + kBlock - 1) / kBlock : 0;
        int incl = mine;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int o = __shfl_up_sync(kAll, incl, s);
            if (i >= s) incl += o;
        }
        const int first = __shfl_sync(kAll, incl - mine, tokens ? __ffs(tokens) - 1 : 0);   // (its lowest lane has the sum before it)
        for (int b = 0; b < mine; ++b) expert[first + b] = static_cast<uint32_t>(e) | static_cast<uint32_t>(have - b * kBlock < kBlock ? have - b * kBlock : kBlock) << 16;
        if (i < n) ids[i] = e;
        if (i == 31) *count = incl;
        if (counts) {
            const int at = first * kBlock + place;
            if constexpr (WEIGHTS) weight[at] = w;
            row[at] = static_cast<uint16_t>(i);
            token[at] = static_cast<uint8_t>(t);
        }
    }

    // By the whole CTA.
    template <bool WEIGHTS>
    __device__ void make(const LayerParams &p) const
    {
        const int n = p.tokens * p.top_k;
        if (n <= 32) {
            if (threadIdx.x < 32) make_few<WEIGHTS>(p, n);
            __syncthreads();
            return;
        }
        for (int e = threadIdx.x; e < p.experts; e += kRowsThreads) mask[e] = 0ull;
        for (int i = threadIdx.x; i < n; i += kRowsThreads) {
            const int e = ld_global(p.ids + i);
            ids[i] = e >= 0 && e < p.experts ? e : -1;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kRowsThreads)
            if (ids[i] >= 0) atomicOr(mask + ids[i], 1ull << (i / p.top_k));
        __syncthreads();
        // each expert's first block: sums over the experts before it
        int carry = 0;
        for (int e0 = 0; e0 < p.experts; e0 += kRowsThreads) {
            const int e = e0 + static_cast<int>(threadIdx.x);
            const int tokens = e < p.experts ? __popcll(mask[e]) : 0, mine = (tokens + kBlock - 1) / kBlock;
            const int first = rows_scan(mine, carry, count + 4);
            if (mine) base[e] = static_cast<uint16_t>(first);
            for (int b = 0; b < mine; ++b) {
                const int left = tokens - b * kBlock;
                expert[first + b] = static_cast<uint32_t>(e) | static_cast<uint32_t>(left < kBlock ? left : kBlock) << 16;
            }
        }
        if (threadIdx.x == 0) *count = carry;
        __syncthreads();
        // every assignment's place: behind the lower tokens of its expert
        for (int i = threadIdx.x; i < n; i += kRowsThreads) {
            const int e = ids[i], t = i / p.top_k;
            if (e < 0) continue;
            bool again = false;
            for (int j = t * p.top_k; j < i; ++j) again |= ids[j] == e;
            if (again) continue;
            const int at = base[e] * kBlock + __popcll(mask[e] & ((1ull << t) - 1ull));
            if constexpr (WEIGHTS) {
                float w = ld_global(p.weights + i);
                for (int j = i + 1; j < (t + 1) * p.top_k; ++j)
                    if (ids[j] == e) w += ld_global(p.weights + j);
                weight[at] = w;
            }
            row[at] = static_cast<uint16_t>(i);
            token[at] = static_cast<uint8_t>(t);
        }
        __syncthreads();
    }
};

// ---- up ------------------------------------------------------------------------

template <int KIND, bool GATED, int NB>
struct UpSource {
    const LayerParams &p;
    const LayerBlocks<NB> &blocks;

    __device__ __forceinline__ int count() const { return *blocks.count; }
    __device__ __forceinline__ long long expert(int b) const { return blocks.expert[b] & 0xffffu; }
    __device__ __forceinline__ int have(int b) const { return static_cast<int>(blocks.expert[b] >> 16); }
    __device__ __forceinline__ const uint16_t *row(int b, int place) const
    {
        return static_cast<const uint16_t *>(p.x) + static_cast<long long>(blocks.token[b * 8 * NB + place]) * p.dim;
    }
    struct Early {
        uint32_t bias[2];
    };
    __device__ __forceinline__ Early early(int b, int, int f, bool two) const
    {
        Early v{};
        if (p.up_bias) {
            const uint16_t *bias = static_cast<const uint16_t *>(p.up_bias) + expert(b) * p.hidden * (GATED ? 2 : 1);
            v.bias[0] = ld_global(bias + f);
            if (two) v.bias[1] = ld_global(bias + (GATED ? p.hidden + f : f + 8));
        }
        return v;
    }
    __device__ __forceinline__ void finish(int b, int place, int have, int f, float (&s)[4], bool two, const Early &early) const
    {
        if (p.up_bias) {
            const float b0 = unpack1<KIND>(early.bias[0]), b1 = unpack1<KIND>(early.bias[1]);
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
            if (place + i >= have) break;
            uint16_t *h = static_cast<uint16_t *>(p.hs) + static_cast<long long>(blocks.row[b * 8 * NB + place + i]) * p.hidden;
            const uint32_t both = pack2f<KIND>(s[i], s[2 + i]);
            h[f] = static_cast<uint16_t>(both);
            if (!GATED && two) h[f + 8] = static_cast<uint16_t>(both >> 16);
        }
    }
};

// The chunks of the hidden rows, block by block, that a warp of the down kernel takes.
struct DownShare {
    int first, end;
    __device__ __forceinline__ DownShare(int blocks, int chunks, int warp, int ctas)
    {
        const long long all = static_cast<long long>(blocks) * chunks;
        first = static_cast<int>(all * warp / (ctas * kRowsWarps));
        end = static_cast<int>(all * (warp + 1) / (ctas * kRowsWarps));
    }
};

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int KIND, bool GATED, int NB, bool SHARED>
__global__ void __launch_bounds__(kRowsThreads, 2) layer_up_kernel(const LayerParams p, int max_blocks, int kw, int ctas, int down_ctas)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const LayerBlocks<NB> blocks(smem + rows_part_bytes(NB, kw), max_blocks, p.experts, p.tokens * p.top_k);
    pdl_wait();
    // (only now: the down kernel loads weights before it waits, which whatever ran before this kernel may have written)
    pdl_launch_dependents();
    blocks.template make<false>(p);
    stream_items<KIND, GATED, NB, SHARED>(UpSource<KIND, GATED, NB>{p, blocks}, static_cast<const uint16_t *>(p.up), p.hidden, p.dim,
                                  reinterpret_cast<float *>(smem), kw, ctas);
    // While the last CTAs finish and the down kernel starts, memory would idle: what its
    // warps load first is brought to L2.
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id());
    const int row = static_cast<int>(blockIdx.x) / down_ctas * kLayerRows + (lane >> 1), chunks = (p.hidden + 31) / 32;
    const DownShare share(*blocks.count, chunks, static_cast<int>(blockIdx.x) % down_ctas * kRowsWarps + warp, down_ctas);
    if (row < p.dim && share.first < share.end) {
        const int b = share.first / chunks, k = (share.first - b * chunks) * 32 + (lane & 1) * 128;
        const uint16_t *at = static_cast<const uint16_t *>(p.down) + ((blocks.expert[b] & 0xffffu) * static_cast<long long>(p.dim) + row) * p.hidden;
        if (k < p.hidden) prefetch_l2(at + k);
        if (k + 64 < p.hidden) prefetch_l2(at + k + 64);
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
__global__ void __launch_bounds__(kRowsThreads, 2) layer_down_kernel(const LayerParams p, int max_blocks, int ctas)
{
    extern __shared__ __align__(16) uint8_t smem[];
    float *sums = reinterpret_cast<float *>(smem);   // [warps][tokens][kDownPitch]
    const LayerBlocks<NB> blocks(smem + kRowsWarps * p.tokens * kDownPitch * 4, max_blocks, p.experts, p.tokens * p.top_k);
    constexpr int kBlock = 8 * NB;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id()), g = lane >> 2, t4 = lane & 3;
    const int share = static_cast<int>(blockIdx.x) % ctas, step = static_cast<int>(gridDim.x) / ctas;
    pdl_launch_dependents();
    blocks.template make<true>(p);   // (ids and weights were there before the up kernel began)

    const int tiles = (p.dim + kLayerRows - 1) / kLayerRows, chunks = (p.hidden + 31) / 32;
    const DownShare mine_of(*blocks.count, chunks, share * kRowsWarps + warp, ctas);
    const int first = mine_of.first, end = mine_of.end;
    const uint16_t *down = static_cast<const uint16_t *>(p.down), *hs = static_cast<const uint16_t *>(p.hs);
    float *mine = sums + warp * p.tokens * kDownPitch;

    // the chunks from `at` on, up to rows_chunks() of one block
    auto group_of = [&](int tile, int at) {
        RowsGroup<NB> group;
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

    // what is added to the sums, of this thread's tokens and pairs of rows: biases and residual
    constexpr int kOutputs = kLayerMaxTokens * (kLayerRows / 2) / kRowsThreads;
    float2 base[kOutputs];
    auto load_base = [&](int tile) {
#pragma unroll
        for (int m = 0; m < kOutputs; ++m) {
            base[m] = make_float2(0.0f, 0.0f);
            const int i = (m * kRowsThreads + static_cast<int>(threadIdx.x)) * ctas + share, t = i >> 3;
            const long long n = static_cast<long long>(tile) * kLayerRows + 2 * (i & 7);
            if (tile >= tiles || t >= p.tokens || n >= p.dim) continue;
            if (p.down_bias)
                for (int j = 0; j < p.top_k; ++j) {
                    const int e = blocks.ids[t * p.top_k + j];
                    if (e < 0) continue;
                    const float f = ld_global(p.weights + t * p.top_k + j);
                    const float2 q = unpack2<KIND>(ld_global(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.down_bias) + static_cast<long long>(e) * p.dim + n)));
                    base[m].x = fmaf(f, q.x, base[m].x);
                    base[m].y = fmaf(f, q.y, base[m].y);
                }
            if (p.residual) {
                const float2 q = unpack2<KIND>(ld_global(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.residual) + t * static_cast<long long>(p.dim) + n)));
                base[m].x += q.x;
                base[m].y += q.y;
            }
        }
    };

    RowsStream<KIND, NB> stream;
    int tile = static_cast<int>(blockIdx.x) / ctas;
    RowsGroup<NB> group = group_of(tile, first);
    stream.start_w(group);
    if (NB == 1) load_base(tile);   // (inputs of the up kernel too, or its caller's: they are there.  By 32 the registers are taken)
    pdl_wait();   // the hidden rows
    stream.start_x(group);
    for (bool again = false; tile < tiles; tile += step, again = true) {
        if (NB == 1 && again) load_base(tile);
        for (int i = lane; i < p.tokens * kDownPitch; i += 32) mine[i] = 0.0f;
        __syncwarp();
        float acc[NB][4] = {};
        for (int at = first; at < end;) {
            const int b = at / chunks, c = at - b * chunks;
            const int left = end - at < chunks - c ? end - at : chunks - c;   // of this block
            const int take = left < rows_chunks(NB) ? left : rows_chunks(NB);
            const bool more = at + take < end;
            const RowsGroup<NB> next = group_of(more ? tile : tile + step, more ? at + take : first);
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
        if (NB > 1) load_base(tile);
        // over the warps, then over the cluster's CTAs: a thread per token and pair of rows
        for (int pass = ctas > 1 ? 0 : 1; pass < 2; ++pass) {
#pragma unroll
            for (int m = 0; m < kOutputs; ++m) {
                const int i = pass ? (m * kRowsThreads + static_cast<int>(threadIdx.x)) * ctas + share : m * kRowsThreads + static_cast<int>(threadIdx.x);
                if (i >= p.tokens * 8) break;
                const int t = i >> 3, at = t * kDownPitch + 2 * (i & 7);
                float2 s = make_float2(0.0f, 0.0f);
                if (pass && ctas > 1) {
                    for (int k = 0; k < ctas; ++k) {
                        const float2 q = ld_cluster_f32x2(mapa(smem_u32(sums + at), static_cast<uint32_t>(k)));
                        s.x += q.x, s.y += q.y;
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < kRowsWarps; ++v) {
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
                *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.y) + t * static_cast<long long>(p.dim) + n) = pack2f<KIND>(s.x + base[m].x, s.y + base[m].y);
            }
            if (ctas > 1) cluster_sync();
            else __syncthreads();
        }
    }
}

// Blocks of 8 tokens, or of 32 where experts have more than so many on average and there
// is so much to multiply: a second block reads its weights from L2, but of 32 fewer chunks
// are on their way, and fewer items (us by 8 / by 32, gated; 13 and 20 tokens, 4 of 4
// experts of 4096 x 1024 31 / 40, 39 / 41; 32 51 / 44; 20 of 2048^2 42 / 34; 16 and 64,
// 1 of 1 of 2048^2 13.7 / 15.3, 37.6 / 32.8; 64, 2 of 8 of 1024^2 26.6 / 24.6, of 4096^2
// 246 / 176; 64, 8 of 32 of 2048^2 230 / 175).
constexpr int kLayerManyMean = 14;
constexpr long long kLayerManyProducts = 500000000;   // of a weight and a token's value

// Warps of a team by 32: 2, since the sums of larger ones take room that L1 needs, unless
// there are too few items for all teams.
inline int layer_many_kw(long long items, const RowsRoom &room)
{
    return items <= room.clusters[1] / 2 ? 8 : items <= 2 * room.clusters[1] ? 4 : 2;
}

template <int NB>
constexpr size_t layer_tables(int assignments, int experts)
{
    return LayerBlocks<NB>::bytes(layer_max_blocks(assignments, experts, NB), experts, assignments);
}
template <int NB>
constexpr size_t layer_smem(int tokens, int assignments, int experts)   // the larger of the two kernels'
{
    const size_t up = rows_part_bytes(NB, 8), down = kRowsWarps * kDownPitch * 4 * tokens;
    return layer_tables<NB>(assignments, experts) + (up > down ? up : down);
}

template <class... P, class... A>
cudaError_t launch_layer_kernel(void (*kernel)(P...), long long items, int ctas, size_t smem, const LayerParams &p, const RowsRoom &room, cudaStream_t stream, bool overlap, A... args)
{
    // (the limit is the function's: always the most that any call needs)
    constexpr int kMostSmem = 150 * 1024;
    static_assert(layer_smem<1>(kLayerMaxTokens, kLayerMaxAssignments, kLayerMaxExperts) <= kMostSmem
                  && layer_smem<4>(kLayerMaxTokens, kLayerMaxAssignments, kLayerMaxAssignments / kLayerManyMean) <= kMostSmem, "");
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e != cudaSuccess) return e;
    }
    const long long most = room.clusters[ctas], clusters = items < most ? items : most;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(clusters * ctas)), kRowsThreads, smem, ctas, stream, overlap, p, args...);
}

template <int KIND, int NB>
cudaError_t launch_layer_of(const LayerParams &p, const RowsRoom &room, cudaStream_t stream, bool overlap)
{
    const int n = p.tokens * p.top_k, blocks = layer_max_blocks(n, p.experts, NB);
    const bool gated = p.act & ACT_GATED;
    const size_t tables = layer_tables<NB>(n, p.experts);
    // few tiles: CTAs share one's contraction
    const long long tiles = (p.dim + kLayerRows - 1) / kLayerRows;
    int down_ctas = 1;
    for (int c = 2; c <= 8; c *= 2)   // (75 tiles by 4, of which 74 find room: 29.5 us, by 2 25.7)
        if (tiles <= room.clusters[c]) down_ctas = c;
    if (p.hidden > 0) {
        const int features = gated ? 8 : 16;
        const long long items = static_cast<long long>(blocks) * ((p.hidden + features - 1) / features);
        const int kw = NB == 1 ? rows_kw(items, p.dim, room) : layer_many_kw(items, room), ctas = NB == 1 ? rows_ctas(items, p.dim, room) : 1;
        const auto kernel = ctas > 1 ? (gated ? layer_up_kernel<KIND, true, NB, NB == 1> : layer_up_kernel<KIND, false, NB, NB == 1>)
                                     : (gated ? layer_up_kernel<KIND, true, NB, false> : layer_up_kernel<KIND, false, NB, false>);
        const cudaError_t e = launch_layer_kernel(kernel, items, ctas, rows_part_bytes(NB, kw) + tables, p, room, stream, overlap, blocks, kw, ctas, down_ctas);
        if (e != cudaSuccess) return e;
    }
    // (without an up kernel before it nothing may be read early)
    return launch_layer_kernel(layer_down_kernel<KIND, NB>, tiles, down_ctas, kRowsWarps * p.tokens * kDownPitch * 4 + tables, p, room, stream,
                               overlap && p.hidden > 0, blocks, down_ctas);
}

template <int KIND>
cudaError_t launch_layer(const LayerParams &p, const RowsRoom &room, cudaStream_t stream, bool overlap)
{
    const int n = p.tokens * p.top_k;
    const bool many = n > kLayerManyMean * p.experts && static_cast<double>(n) * p.dim * p.hidden * (p.act & ACT_GATED ? 3 : 2) > kLayerManyProducts;
    return many ? launch_layer_of<KIND, 4>(p, room, stream, overlap) : launch_layer_of<KIND, 1>(p, room, stream, overlap);
}

}  // namespace pts
