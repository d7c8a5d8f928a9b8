// The backward pass through a product's epilogue: dZ = dC act'(Z), gated both
// halves of it, and the bias's gradient, the column sums of dZ per expert.
//
// One pass over dC and Z.  A thread owns 8 columns (16 bytes) and every TY-th
// row of its CTA's stretch, so it keeps its columns' sums in registers, in fp32
// and before dZ is rounded.  The rows of an expert and column block are shared
// by a cluster of up to 8 CTAs, which add up through distributed shared memory:
// always in the same order, without atomics and without a workspace (two
// captured graphs share nothing).
#include "activation.cuh"
#include "launch.cuh"
#include "layer_launch.h"
#include "ptx.cuh"

namespace pts {

namespace {

constexpr int kGradThreads = 256;
constexpr int kGradRows = 4;      // rows of a thread whose loads are on their way together
constexpr int kGradMaxCtas = 8;   // CTAs that share an expert's rows

__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// tx: threads side by side (a power of two), ctas: CTAs of a cluster
template <int KIND, bool GATED>
__global__ void __launch_bounds__(kGradThreads)
    linear_grad_kernel(const LinearGradParams p, int tx, int ctas, int blocks)
{
    extern __shared__ float sums[];   // [GATED + 1][rows at a time][8 tx], then [GATED + 1][8 tx]
    const int rank = static_cast<int>(blockIdx.x) % ctas, unit = static_cast<int>(blockIdx.x) / ctas;
    const int e = unit / blocks, block = unit - e * blocks;
    const int ty = kGradThreads / tx, my = static_cast<int>(threadIdx.x) / tx, mx = static_cast<int>(threadIdx.x) % tx;
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
    float sum[GATED ? 2 : 1][8] = {};
    with_act(p.act, [&](auto tag) {
        constexpr int A = decltype(tag)::value;
        for (long long r0 = first + my; in && r0 < end; r0 += static_cast<long long>(ty) * kGradRows) {
            uint4 d[kGradRows], g[kGradRows], u[kGradRows];
#pragma unroll
            for (int i = 0; i < kGradRows; ++i) {
                const long long r = r0 + static_cast<long long>(i) * ty;
                if (r >= end) continue;
                d[i] = ld_global_streamed(reinterpret_cast<const uint4 *>(dc + r * p.N + col));
                g[i] = ld_global_streamed(reinterpret_cast<const uint4 *>(z + r * pitch + col));
                if constexpr (GATED) u[i] = ld_global_streamed(reinterpret_cast<const uint4 *>(z + r * pitch + p.N + col));
            }
#pragma unroll
            for (int i = 0; i < kGradRows; ++i) {
                const long long r = r0 + static_cast<long long>(i) * ty;
                if (r >= end) continue;
                const uint32_t dw[4] = {d[i].x, d[i].y, d[i].z, d[i].w}, gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
                uint32_t uw[4] = {}, o[4], o2[4];
                if constexpr (GATED) uw[0] = u[i].x, uw[1] = u[i].y, uw[2] = u[i].z, uw[3] = u[i].w;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 c = unpack2<KIND>(dw[q]), x = unpack2<KIND>(gw[q]);
                    const float2 s0 = act_and_slope<A>(x.x), s1 = act_and_slope<A>(x.y);
                    float a = c.x * s0.y, b = c.y * s1.y;
                    if constexpr (GATED) {
                        const float2 y = unpack2<KIND>(uw[q]);
                        a *= y.x;
                        b *= y.y;
                        const float a2 = c.x * s0.x, b2 = c.y * s1.x;
                        sum[1][2 * q] += a2;
                        sum[1][2 * q + 1] += b2;
                        o2[q] = pack2f<KIND>(a2, b2);
                    }
                    sum[0][2 * q] += a;
                    sum[0][2 * q + 1] += b;
                    o[q] = pack2f<KIND>(a, b);
                }
                *reinterpret_cast<uint4 *>(dz + r * pitch + col) = make_uint4(o[0], o[1], o[2], o[3]);
                if constexpr (GATED) *reinterpret_cast<uint4 *>(dz + r * pitch + p.N + col) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
            }
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
        for (int q = 0; q < 8; ++q) sums[(h * ty + my) * width + mx * 8 + q] = sum[h][q];
    __syncthreads();
    for (int c = static_cast<int>(threadIdx.x); c < kHalves * width; c += kGradThreads) {
        const float *from = sums + c / width * ty * width + c % width;
        float s = 0.0f;
        for (int y = 0; y < ty; ++y) s += from[y * width];
        total[c] = s;
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    for (int c = static_cast<int>(threadIdx.x) * ctas + rank; c < kHalves * width; c += kGradThreads * ctas) {
        float s = 0.0f;
        for (int k = 0; k < ctas; ++k) s += ctas > 1 ? ld_cluster_f32(mapa(smem_u32(total + c), static_cast<uint32_t>(k))) : total[c];
        const long long at = static_cast<long long>(block) * width + c % width;
        if (at < p.N) p.dbias[e * pitch + c / width * p.N + at] = s;
    }
    if (ctas > 1) cluster_sync();   // (the others have read this CTA's sums)
}

template <int KIND, bool GATED>
cudaError_t go(const LinearGradParams &p, cudaStream_t stream, bool overlap)
{
    const int64_t pieces = (p.N + 7) / 8, each = p.rows / p.experts;
    int tx = 32, ctas = 1;
    while (tx > 4 && tx / 2 >= pieces) tx /= 2;
    const auto grid = [&] { return p.experts * ((pieces + tx - 1) / tx) * ctas; };
    while (grid() < 4 * p.sms && ctas < kGradMaxCtas && each / (2 * ctas) >= kGradThreads / tx * kGradRows) ctas *= 2;
    while (grid() < 4 * p.sms && ctas == kGradMaxCtas && tx > 8) tx /= 2;
    if (grid() > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const size_t smem = (GATED ? 2 : 1) * (kGradThreads + tx) * 8 * sizeof(float);
    return launch_kernel(linear_grad_kernel<KIND, GATED>, dim3(static_cast<unsigned>(grid())), kGradThreads, smem, ctas, stream, overlap, p,
                         tx, ctas, static_cast<int>((pieces + tx - 1) / tx));
}

}  // namespace

cudaError_t launch_linear_grad(int kind, const LinearGradParams &p, cudaStream_t stream, bool overlap)
{
    if (p.act & ACT_GATED) return kind == 0 ? go<0, true>(p, stream, overlap) : go<1, true>(p, stream, overlap);
    return kind == 0 ? go<0, false>(p, stream, overlap) : go<1, false>(p, stream, overlap);
}

}  // namespace pts
