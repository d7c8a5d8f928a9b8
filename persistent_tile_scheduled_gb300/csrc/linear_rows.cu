// The product with an epilogue for one to a few rows per matrix: the weights are
// streamed into registers (rows_stream.cuh) instead of through shared memory.
#include <type_traits>

#include "expert_launch.h"
#include "rows_stream.cuh"

namespace pts {

namespace {

// The blocks of 8 rows of the experts, made by every CTA for itself in shared memory.
struct RowBlocks {
    int2 *block;   // [blocks]: expert | rows << 16, first row
    int *count;    // blocks; and behind it a sum per warp

    static constexpr size_t bytes(int blocks) { return static_cast<size_t>(blocks) * 8 + 4 * (1 + kRowsWarps); }

    // (at most max_blocks, which ascending offsets do not pass)
    __device__ void make(const LinearRowsParams &p, int max_blocks) const
    {
        if (!p.offsets) {   // (one matrix)
            const int n = (p.rows + 7) / 8;
            for (int b = threadIdx.x; b < n; b += kRowsThreads) block[b] = make_int2((p.rows - 8 * b < 8 ? p.rows - 8 * b : 8) << 16, 8 * b);
            if (threadIdx.x == 0) *count = n;
            __syncthreads();
            return;
        }
        int carry = 0;
        for (int e0 = 0; e0 < p.experts; e0 += kRowsThreads) {
            const int e = e0 + static_cast<int>(threadIdx.x);
            int lo = 0, hi = 0;
            if (e < p.experts) {
                lo = ld_global(p.offsets + e), hi = ld_global(p.offsets + e + 1);
                lo = lo < 0 ? 0 : (lo > p.rows ? p.rows : lo);
                hi = hi < lo ? lo : (hi > p.rows ? p.rows : hi);
            }
            const int mine = (hi - lo + 7) / 8, first = rows_scan(mine, carry, count + 1);
            for (int b = 0; b < mine && first + b < max_blocks; ++b) {
                const int left = hi - lo - 8 * b;
                block[first + b] = make_int2(e | (left < 8 ? left : 8) << 16, lo + 8 * b);
            }
        }
        if (threadIdx.x == 0) *count = carry < max_blocks ? carry : max_blocks;
        __syncthreads();
    }
};

template <int KIND, bool GATED>
struct LinearSource {
    const LinearRowsParams &p;
    const RowBlocks &blocks;

    __device__ __forceinline__ int count() const { return *blocks.count; }
    __device__ __forceinline__ long long expert(int b) const { return blocks.block[b].x & 0xffff; }
    __device__ __forceinline__ int have(int b) const { return blocks.block[b].x >> 16; }
    __device__ __forceinline__ const uint16_t *row(int b, int place) const
    {
        return static_cast<const uint16_t *>(p.x) + static_cast<long long>(blocks.block[b].y + place) * p.K;
    }
    struct Early {
        uint32_t bias[2], residual[2][2];   // [token][feature f, f + 8]
    };
    __device__ __forceinline__ Early early(int b, int have, int f, bool two) const
    {
        Early v{};
        if (p.bias) {
            const uint16_t *bias = static_cast<const uint16_t *>(p.bias) + expert(b) * p.N * (GATED ? 2 : 1);
            v.bias[0] = ld_global(bias + f);
            if (two) v.bias[1] = ld_global(bias + (GATED ? p.N + f : f + 8));
        }
        if (p.residual) {
            const int place = 2 * static_cast<int>(lane_id() & 3u);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (place + i >= have) break;
                const uint16_t *r = static_cast<const uint16_t *>(p.residual) + static_cast<long long>(blocks.block[b].y + place + i) * p.N + f;
                v.residual[i][0] = ld_global(r);
                if (!GATED && two) v.residual[i][1] = ld_global(r + 8);
            }
        }
        return v;
    }
    __device__ __forceinline__ void finish(int b, int place, int have, int f, float (&s)[4], bool two, const Early &early) const
    {
        constexpr int kBoth = GATED ? 2 : 1;
        const int f2 = GATED ? p.N + f : f + 8;   // of Z
        if (p.bias) {
            const float b0 = unpack1<KIND>(early.bias[0]), b1 = unpack1<KIND>(early.bias[1]);
            s[0] += b0, s[1] += b0, s[2] += b1, s[3] += b1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!p.z || place + i >= have) break;
            uint16_t *z = static_cast<uint16_t *>(p.z) + static_cast<long long>(blocks.block[b].y + place + i) * p.N * kBoth;
            const uint32_t both = pack2f<KIND>(s[i], s[2 + i]);
            z[f] = static_cast<uint16_t>(both);
            if (two) z[f2] = static_cast<uint16_t>(both >> 16);
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
            const long long at = static_cast<long long>(blocks.block[b].y + place + i) * p.N + f;
            const bool second = !GATED && two;
            if (p.residual) {
                s[i] += unpack1<KIND>(early.residual[i][0]);
                if (second) s[2 + i] += unpack1<KIND>(early.residual[i][1]);
            }
            uint16_t *c = static_cast<uint16_t *>(p.c) + at;
            const uint32_t both = pack2f<KIND>(s[i], s[2 + i]);
            c[0] = static_cast<uint16_t>(both);
            if (second) c[8] = static_cast<uint16_t>(both >> 16);
        }
    }
};

template <int KIND, bool GATED, bool SHARED>
__global__ void __launch_bounds__(kRowsThreads, 2) linear_rows_kernel(const LinearRowsParams p, int max_blocks, int kw, int ctas)
{
    extern __shared__ __align__(16) uint8_t smem[];
    RowBlocks blocks;
    blocks.block = reinterpret_cast<int2 *>(smem + rows_part_bytes(1, kw));
    blocks.count = reinterpret_cast<int *>(blocks.block + max_blocks);
    pdl_launch_dependents();
    if (p.offsets) pdl_wait();
    blocks.make(p, max_blocks);
    if (!p.offsets) pdl_wait();
    stream_items<KIND, GATED, 1, SHARED>(LinearSource<KIND, GATED>{p, blocks}, static_cast<const uint16_t *>(p.w), p.N, p.K,
                                 reinterpret_cast<float *>(smem), kw, ctas);
}

}  // namespace

void ask_rows_room(RowsRoom &room, int sms)
{
    room.clusters[1] = 2 * sms;
    for (int c = 2; c <= 8; c *= 2) {
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = static_cast<unsigned>(c);
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(c));
        cfg.blockDim = dim3(kRowsThreads);
        cfg.dynamicSmemBytes = rows_part_bytes(1, 8);
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&room.clusters[c], linear_rows_kernel<0, false, true>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            room.clusters[c] = 0;
        }
    }
}

cudaError_t launch_linear_rows(int kind, const LinearRowsParams &p, const RowsRoom &room, cudaStream_t stream, bool overlap)
{
    const bool gated = p.act & ACT_GATED;
    const int blocks = p.experts == 1 ? (p.rows + 7) / 8 : (p.rows < p.experts ? p.rows : p.experts) + p.rows / 8;
    const int features = gated ? 8 : 16, tiles = (p.N + features - 1) / features;
    const long long items = static_cast<long long>(blocks) * tiles;
    const int kw = rows_kw(items, p.K, room), ctas = rows_ctas(items, p.K, room), teams = kRowsWarps / kw;
    const long long most = room.clusters[ctas], wanted = (items + teams - 1) / teams, clusters = wanted < most ? wanted : most;
    const size_t smem = rows_part_bytes(1, kw) + RowBlocks::bytes(blocks);
    static_assert(rows_part_bytes(1, 8) + RowBlocks::bytes(kLinearRowsMax + kLinearRowsMax / 8) <= 48 * 1024, "");
    const auto run = [&](auto kernel) {
        return launch_kernel(kernel, dim3(static_cast<unsigned>(clusters * ctas)), kRowsThreads, smem, ctas, stream, overlap, p, blocks, kw, ctas);
    };
    const auto pick = [&](auto shared) {
        constexpr bool S = decltype(shared)::value;
        if (kind == 0) return gated ? run(linear_rows_kernel<0, true, S>) : run(linear_rows_kernel<0, false, S>);
        return gated ? run(linear_rows_kernel<1, true, S>) : run(linear_rows_kernel<1, false, S>);
    };
    return ctas > 1 ? pick(std::true_type()) : pick(std::false_type());
}

}  // namespace pts
