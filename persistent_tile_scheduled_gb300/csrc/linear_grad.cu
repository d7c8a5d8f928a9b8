// The backward pass through a product's epilogue: dZ = dC act'(Z), gated both
// halves of it, and the bias's gradient, the column sums of dZ per expert.
//
// One pass over dC and Z.  A thread owns 8 columns (16 bytes) and every TY-th
// row of its CTA's stretch, so it keeps its columns' sums in registers, in fp32
// and before dZ is rounded.  The rows of an expert and column block are shared
// by a cluster of CTAs, which add up through distributed shared memory: always
// in the same order, without atomics and without a workspace (two captured graphs
// share nothing).
//
// The bytes bound it: 16384 rows of 8192 columns, bf16, 805 MB in 133 us, 6.0 TB/s (0.89
// of the copy bandwidth; relu^2, which computes next to nothing, 133).  Loading the next
// rows while the last are computed took it there from 162; two values to an instruction
// (f32x2) keep the arithmetic out of the way.
#include "activation.cuh"
#include "launch.cuh"
#include "layer_launch.h"
#include "linear_plan.h"
#include "ptx.cuh"

namespace pts {

namespace {

constexpr int kGradRows = 2;   // rows of a thread that are loaded together, while those before are computed

__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// tx: threads side by side (a power of two), ctas: CTAs of a cluster
template <int KIND, bool GATED>
__global__ void __launch_bounds__(2 * kGradThreads)
    linear_grad_kernel(const LinearGradParams p, int tx, int ctas, int blocks)
{
    extern __shared__ float sums[];   // [GATED + 1][rows at a time][8 tx], then [GATED + 1][8 tx]
    const int rank = static_cast<int>(blockIdx.x) % ctas, unit = static_cast<int>(blockIdx.x) / ctas;
    const int e = unit / blocks, block = unit - e * blocks;
    const int threads = static_cast<int>(blockDim.x), ty = threads / tx, my = static_cast<int>(threadIdx.x) / tx, mx = static_cast<int>(threadIdx.x) % tx;
    const long long col = (static_cast<long long>(block) * tx + mx) * 8;
    const bool in = col < p.N;
    const long long pitch = static_cast<long long>(p.N) * (GATED ? 2 : 1);
    const uint16_t *dc = static_cast<const uint16_t *>(p.dc), *z = static_cast<const uint16_t *>(p.z);
    uint16_t *dz = static_cast<uint16_t *>(p.dz);
    pdl_launch_dependents();
    pdl_wait();
    long long lo = 0, hi = p.rows;
    if (p.offsets) {
        lo = ld_global(p.offsets + e), hi = ld_global(p.offsets + e + 1);
        lo = lo < 0 ? 0 : (lo > p.rows ? p.rows : lo);
        hi = hi < lo ? lo : (hi > p.rows ? p.rows : hi);
    }
    const long long first = lo + (hi - lo) * rank / ctas, end = lo + (hi - lo) * (rank + 1) / ctas;
    Pair sum[GATED ? 2 : 1][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        sum[0][q] = both(0.0f);
        if constexpr (GATED) sum[1][q] = both(0.0f);
    }
    struct Rows {
        uint4 d[kGradRows], g[kGradRows], u[GATED ? kGradRows : 1];
    };
    auto load = [&](Rows &v, long long r0) {
#pragma unroll
        for (int i = 0; i < kGradRows; ++i) {
            const long long r = r0 + static_cast<long long>(i) * ty;
            if (r >= end) break;
            v.d[i] = ld_global_streamed(reinterpret_cast<const uint4 *>(dc + r * p.N + col));
            v.g[i] = ld_global_streamed(reinterpret_cast<const uint4 *>(z + r * pitch + col));
            if constexpr (GATED) v.u[i] = ld_global_streamed(reinterpret_cast<const uint4 *>(z + r * pitch + p.N + col));
        }
    };
    with_act(p.act, [&](auto tag) {
        constexpr int A = decltype(tag)::value;
        const long long step = static_cast<long long>(ty) * kGradRows;
        Rows v, next;
        long long r0 = in ? first + my : end;
        load(v, r0);
        for (; r0 < end; r0 += step) {
            load(next, r0 + step);
#pragma unroll
            for (int i = 0; i < kGradRows; ++i) {
                const long long r = r0 + static_cast<long long>(i) * ty;
                if (r >= end) break;
                const uint32_t dw[4] = {v.d[i].x, v.d[i].y, v.d[i].z, v.d[i].w}, gw[4] = {v.g[i].x, v.g[i].y, v.g[i].z, v.g[i].w};
                uint32_t o[4];
                [[maybe_unused]] uint32_t uw[4], o2[4];
                if constexpr (GATED) uw[0] = v.u[i].x, uw[1] = v.u[i].y, uw[2] = v.u[i].z, uw[3] = v.u[i].w;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const Pair c = pair(unpack2<KIND>(dw[q]));
                    Pair value, d;
                    act_and_slope<A>(pair(unpack2<KIND>(gw[q])), value, d);
                    d = d * c;
                    if constexpr (GATED) {
                        d = d * pair(unpack2<KIND>(uw[q]));
                        const Pair d2 = value * c;
                        sum[1][q] = sum[1][q] + d2;
                        const float2 f2 = values(d2);
                        o2[q] = pack2f<KIND>(f2.x, f2.y);
                    }
                    sum[0][q] = sum[0][q] + d;
                    const float2 f = values(d);
                    o[q] = pack2f<KIND>(f.x, f.y);
                }
                *reinterpret_cast<uint4 *>(dz + r * pitch + col) = make_uint4(o[0], o[1], o[2], o[3]);
                if constexpr (GATED) *reinterpret_cast<uint4 *>(dz + r * pitch + p.N + col) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
            }
            v = next;
        }
    });
    if (!p.dbias) return;
    // over the CTA's rows, then over the cluster's CTAs
    const int width = 8 * tx;
    constexpr int kHalves = GATED ? 2 : 1;
    float *total = sums + kHalves * ty * width;
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) *reinterpret_cast<float2 *>(sums + (h * ty + my) * width + mx * 8 + 2 * q) = values(sum[h][q]);
    __syncthreads();
    for (int c = static_cast<int>(threadIdx.x); c < kHalves * width; c += threads) {
        const float *from = sums + c / width * ty * width + c % width;
        float s = 0.0f;
        for (int y = 0; y < ty; ++y) s += from[y * width];
        total[c] = s;
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    for (int c = static_cast<int>(threadIdx.x) * ctas + rank; c < kHalves * width; c += threads * ctas) {
        float s = 0.0f;
        for (int k = 0; k < ctas; ++k) s += ctas > 1 ? ld_cluster_f32(mapa(smem_u32(total + c), static_cast<uint32_t>(k))) : total[c];
        const long long at = static_cast<long long>(block) * width + c % width;
        if (at < p.N) p.dbias[e * pitch + c / width * p.N + at] = s;
    }
    if (ctas > 1) cluster_sync();   // (the others have read this CTA's sums)
}

// Shared memory of the sums: of each thread's columns, then of the CTA's.
constexpr size_t grad_smem(bool gated, int threads, int tx) { return (gated ? 2 : 1) * static_cast<size_t>(threads + tx) * 8 * sizeof(float); }

template <int KIND, bool GATED>
cudaError_t go(const LinearGradParams &p, int room, cudaStream_t stream, bool overlap)
{
    const GradShape g = grad_shape(p.rows, p.experts, p.N, GATED, p.dbias != nullptr, p.sms, room);
    // (clusters need not be whole where nothing is added up)
    return launch_kernel(linear_grad_kernel<KIND, GATED>, dim3(static_cast<unsigned>(g.units * g.ctas)), g.threads, grad_smem(GATED, g.threads, g.tx),
                         p.dbias ? g.ctas : 1, stream, overlap, p, g.tx, g.ctas, static_cast<int>(g.blocks));
}

// Clusters of kGradMaxCtas CTAs that the device holds at once, 0 where it places none.
template <int KIND, bool GATED>
int ask_room()
{
    const auto kernel = linear_grad_kernel<KIND, GATED>;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kGradMaxCtas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(kGradMaxCtas);
    cfg.blockDim = dim3(kGradThreads);
    cfg.dynamicSmemBytes = grad_smem(GATED, kGradThreads, 8);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess
        || cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return clusters;
}

}  // namespace

int ask_linear_grad_room(int kind, bool gated)
{
    if (gated) return kind == 0 ? ask_room<0, true>() : ask_room<1, true>();
    return kind == 0 ? ask_room<0, false>() : ask_room<1, false>();
}

cudaError_t launch_linear_grad(int kind, const LinearGradParams &p, int room, cudaStream_t stream, bool overlap)
{
    if (p.act & ACT_GATED) return kind == 0 ? go<0, true>(p, room, stream, overlap) : go<1, true>(p, room, stream, overlap);
    return kind == 0 ? go<0, false>(p, room, stream, overlap) : go<1, false>(p, room, stream, overlap);
}

}  // namespace pts
