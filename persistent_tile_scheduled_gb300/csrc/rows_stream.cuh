// A few rows times matrices that are streamed once from memory into registers: what
// the layer of experts for a few tokens and the product with an epilogue share.
//
// 16 rows of the weights are the M side of mma.sync, 8 of an expert's tokens its
// N side; a block is 8 (or 32) tokens of one expert.  The contraction's order is
// free as long as both operands take the same one, so a lane loads 16 contiguous
// bytes of its row, 8 values, and feeds them to two instructions: the weights need
// no shared memory, no shuffles and no conversion.
//
// The weights' bytes bound it: 7.0 TB/s over long matrices (one token through 2
// experts of 4096 x 16384, 122 us), and some 3 us to start and end a launch.
#pragma once
#include "activation.cuh"
#include "expert_launch.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace pts {

constexpr int kRowsThreads = 256;
constexpr int kRowsWarps = kRowsThreads / 32;

// Chunks of 32 of the contraction that are on their way to a warp, and of them those
// whose tokens' values are: what 128 registers hold.
__host__ __device__ constexpr int rows_chunks(int nb) { return nb == 1 ? 8 : 4; }
__host__ __device__ constexpr int rows_ahead(int nb) { return nb == 1 ? 4 : 2; }

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

// Up to rows_chunks() chunks of 32 of the contraction, as a lane reads them: 8 values
// from 32 i + 8 (lane % 4) on, of rows g = lane / 4 and g + 8 of the weights and of
// tokens g, g + 8, ... (none: null).
template <int NB>
struct RowsGroup {
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
// KB per SM, whatever the groups; the tokens' values, mostly in L1, fewer
// chunks ahead.  (Whole groups of 4 chunks, loaded while the one before is
// multiplied: 40.5 us for one token through 8 experts of 4096 x 4096.)
template <int KIND, int NB>
struct RowsStream {
    static constexpr int kChunks = rows_chunks(NB), kAhead = rows_ahead(NB);
    uint4 w[2][kChunks], x[NB][kAhead];

    __device__ __forceinline__ void load_w(const RowsGroup<NB> &g, int i)
    {
        w[0][i] = w[1][i] = make_uint4(0u, 0u, 0u, 0u);
        if (i < g.n) {
            w[0][i] = ld_weights(g.w[0] + 32 * i);
            if (g.w[1]) w[1][i] = ld_weights(g.w[1] + 32 * i);
        }
    }
    __device__ __forceinline__ void load_x(const RowsGroup<NB> &g, int i)
    {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            x[nb][i % kAhead] = make_uint4(0u, 0u, 0u, 0u);
            if (i < g.n && g.x[nb]) x[nb][i % kAhead] = ld_global(reinterpret_cast<const uint4 *>(g.x[nb] + 32 * i));
        }
    }
    __device__ __forceinline__ void start_w(const RowsGroup<NB> &g)
    {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) load_w(g, i);
    }
    __device__ __forceinline__ void start_x(const RowsGroup<NB> &g)
    {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load_x(g, i);
    }
    // c[nb] += the group: rows g and g + 8 of tokens 8 nb + 2 (lane % 4), + 1; and the next one's loads
    __device__ __forceinline__ void multiply(float (&c)[NB][4], const RowsGroup<NB> &group, const RowsGroup<NB> &next)
    {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const uint4 &v = x[nb][i % kAhead];
                mma_16x8x16<KIND>(c[nb], w[0][i].x, w[1][i].x, w[0][i].y, w[1][i].y, v.x, v.y);
                mma_16x8x16<KIND>(c[nb], w[0][i].z, w[1][i].z, w[0][i].w, w[1][i].w, v.z, v.w);
            }
            load_w(next, i);
            if (i + kAhead < kChunks) load_x(group, i + kAhead);
            else load_x(next, i + kAhead - kChunks);
        }
    }
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t cluster_addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_addr) : "memory");
    return v;
}

// Exclusive sums over the CTA's threads; `carry` is the sum of what came before and
// comes back with these added.  sums: kRowsWarps ints of shared memory.
__device__ __forceinline__ int rows_scan(int mine, int &carry, int *sums)
{
    const int lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x >> 5);
    int incl = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += o;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) {
        const int v = sums[w];
        if (w < warp) before += v;
        carry += v;
    }
    __syncthreads();
    return before + incl - mine;
}

// ---- items: a block of tokens and 16 rows of its expert's matrix ---------------------
//
// Gated 8 features, their gate and up rows; else 16 features.  kw warps, a team,
// share an item's contraction; the teams of all CTAs stride over the items.  Few
// items (SHARED): all warps of `ctas` CTAs of a cluster share one's, and a cluster has
// one item.
// Source: what a block is:
//   count(), expert(b), have(b)          blocks; a block's expert and tokens
//   row(b, place)                        a token's row of the operand
//   early(b, have, f, two)               what finish adds, loaded when a cluster's only item begins: bias, residual
//   finish(b, place, have, f, s, two, early)
//                                        s[0], s[1]: feature f of tokens place and place + 1, s[2], s[3]:
//                                        feature f + 8 (gated: the gate's f and the other's f)
template <int KIND, bool GATED, int NB, bool SHARED, class Source>
__device__ __forceinline__ void stream_items(const Source &source, const uint16_t *weights, int features, int width, float *part, int kw, int ctas)
{
    if constexpr (SHARED) kw = kRowsWarps;
    else ctas = 1;
    constexpr int kChunks = rows_chunks(NB), kFeatures = GATED ? 8 : 16;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id()), g = lane >> 2;
    const int tiles = (features + kFeatures - 1) / kFeatures, chunks = (width + 31) / 32;
    const int team = warp / kw, member = warp % kw;
    const int share = static_cast<int>(blockIdx.x) % ctas * kw + member;   // this warp's
    const int first = static_cast<int>(static_cast<long long>(chunks) * share / (ctas * kw));
    const int end = static_cast<int>(static_cast<long long>(chunks) * (share + 1) / (ctas * kw));
    const int items = source.count() * tiles, step = static_cast<int>(gridDim.x) / ctas * (kRowsWarps / kw);
    const long long matrix = static_cast<long long>(features) * (GATED ? 2 : 1);

    auto group_of = [&](int item, int at) {
        RowsGroup<NB> group;
        if (item >= items || at >= end) {
            group.none();
            return group;
        }
        const int b = item / tiles, f = (item - b * tiles) * kFeatures + g, have = source.have(b);
        const uint16_t *row = weights + (source.expert(b) * matrix + f) * width, *tokens[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) tokens[nb] = 8 * nb + g < have ? source.row(b, 8 * nb + g) : nullptr;
        group.set(row, GATED || f + 8 < features ? row + static_cast<long long>(GATED ? features : 8) * width : nullptr,
                  tokens, at, end, width);
        return group;
    };

    RowsStream<KIND, NB> stream;
    int item = static_cast<int>(blockIdx.x) / ctas + static_cast<int>(gridDim.x) * team;
    const int only = item;
    typename Source::Early early{};
    RowsGroup<NB> group = group_of(item, first);
    stream.start_w(group);
    stream.start_x(group);
    for (int n = 0; item < items; item += step, ++n) {
        const int b = item / tiles, f = (item - b * tiles) * kFeatures + g, have = source.have(b);
        const bool two = GATED || f + 8 < features;
        if (SHARED && warp == 0) early = source.early(b, have, f, two);
        float acc[NB][4] = {};
        for (int at = first; at < end; at += kChunks) {
            const bool more = at + kChunks < end;
            const RowsGroup<NB> next = group_of(more ? item : item + step, more ? at + kChunks : first);
            stream.multiply(acc, group, next);
            group = next;
        }
        // Over the team's warps: one of them in turn, the others run on.  It waits for all
        // at this item, so every warp does once in kw items: none can come back to an
        // item's place (and barrier) before its reader is through with it.
        const int turn = n % kw, bar = 1 + team * kw + turn;
        float *mine = part + (team * kw + turn) * kw * NB * 128;   // [member][NB][32 lanes][4]
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            *reinterpret_cast<float4 *>(mine + ((member * NB + nb) * 32 + lane) * 4) = make_float4(acc[nb][0], acc[nb][1], acc[nb][2], acc[nb][3]);
        if (member != turn) {
            asm volatile("bar.arrive %0, %1;" ::"r"(bar), "r"(32 * kw) : "memory");
            continue;
        }
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * kw) : "memory");
        if constexpr (!SHARED) early = source.early(b, have, f, two);   // (while weights are multiplied the registers are taken: 4 % slower)
        // a lane has rows g and g + 8 of two tokens
        for (int nb = 0; nb < NB && 8 * nb < have; ++nb) {
            float s[4] = {};
            for (int v = 0; v < kw; ++v) {
                const float4 q = *reinterpret_cast<const float4 *>(mine + ((v * NB + nb) * 32 + lane) * 4);
                s[0] += q.x, s[1] += q.y, s[2] += q.z, s[3] += q.w;
            }
            if constexpr (SHARED)   // (where the first warp's were, which only this lane has read)
                *reinterpret_cast<float4 *>(mine + (nb * 32 + lane) * 4) = make_float4(s[0], s[1], s[2], s[3]);
            else
                source.finish(b, 8 * nb + 2 * (lane & 3), have, f, s, two, early);
        }
    }
    if constexpr (SHARED) {
        cluster_sync();
        if (only < items && warp == 0 && blockIdx.x % ctas == 0) {   // (the first warp of the first CTA adds up the CTAs')
            const int b = only / tiles, f = (only - b * tiles) * kFeatures + g, have = source.have(b);
            for (int nb = 0; nb < NB && 8 * nb < have; ++nb) {
                float s[4] = {};
                for (int c = 0; c < ctas; ++c) {
                    const float4 q = ld_cluster_f32x4(mapa(smem_u32(part + (nb * 32 + lane) * 4), static_cast<uint32_t>(c)));
                    s[0] += q.x, s[1] += q.y, s[2] += q.z, s[3] += q.w;
                }
                source.finish(b, 8 * nb + 2 * (lane & 3), have, f, s, GATED || f + 8 < features, early);
            }
        }
        cluster_sync();
    }
}

// CTAs of a cluster for at most so many items: one wave of clusters, and stretches of
// 4 chunks a warp at least (one row of 1024 x 8192: 4 CTAs to each of 64 items).  Powers
// of 2: others find less room than they are said to (one row of 1536 x 8192, 96 items, by
// 3 8.2 us, by 2 7.5).
inline int rows_ctas(long long items, int width, const RowsRoom &room)
{
    int ctas = 1;
    for (int c = 2; c <= 8; c *= 2)
        if (items <= room.clusters[c] && width >= 32 * 4 * kRowsWarps * c) ctas = c;
    return ctas;
}

// Warps of a team (blocks of 8): all, unless half of them have a full group each and
// there are items for more teams (8 rows of 8192 x 1024 5.1 us by 4, 6.3 by 8; but
// one of 1024^2 2.9 and 2.8, and of 4096 x 8192 16.6 and 12.6).
inline int rows_kw(long long items, int width, const RowsRoom &room) { return width < 64 * 32 && items > room.clusters[1] ? 4 : 8; }

// Shared memory of the sums.
__host__ __device__ constexpr size_t rows_part_bytes(int nb, int kw) { return static_cast<size_t>(kRowsWarps) * kw * nb * 512; }

}  // namespace pts
