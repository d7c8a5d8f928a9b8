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
#include "ptx.cuh"

namespace pts {

namespace {

constexpr int kGradThreads = 256;      // of a CTA, or twice that
constexpr int kGradRows = 2;      // rows of a thread that are loaded together, while those before are computed
constexpr int kGradMaxCtas = 16;   // CTAs of a cluster: they share an expert's rows

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

template <int KIND, bool GATED>
cudaError_t go(const LinearGradParams &p, cudaStream_t stream, bool overlap)
{
    // Blocks of 64 columns, and as many CTAs of 512 threads (two to an SM; gated, with more
    // registers, one, and two of 256) to one as make a single wave, 8 at most; blocks of 32
    // where columns are few, then also 16 CTAs of 256 threads (us, gelu's tanh form, bf16:
    // 16384 rows of 8192 128 blocks by 2 133, by 4 of 256 threads 134, by 8 142; of 2048 32
    // by 8 38.5, 64 blocks of 32 columns by 4 44; of 1024 32 of 32 by 8 24.5, 16 of 64 by 16
    // 29.7; of 512 16 of 32 by 16 of 256 threads 17.2, by 8 19.1; 9115 gated of 1024 by 256
    // threads 21, by 512 33).  Rows that are no multiple of 32 bytes share those at a
    // block's edges: blocks of 128 columns (9115 rows of 7000 76, of 64 84).
    // Experts' rows are uneven: where there are many of them a block is shared although a
    // wave is full, so that the largest does not end last (16384 over 8 of 2048, uneven as
    // exp of half a normal / even: 54 / 41, not shared 67 / 37; gated 67 / 68, 76 / 61).
    // Few rows each and more blocks than five waves: wider ones (4000 over 64 of 4096 35 /
    // 20, of 64 columns 32 / 30; gated 44 / 33, 51 / 50).
    // Clusters need not be whole where nothing is added up.
    const int64_t pieces = p.N / 8, each = p.rows / p.experts, by8 = p.experts * ((pieces + 7) / 8);
    const bool many = p.experts > 1, fills = p.dbias && by8 > p.sms && by8 <= 2 * p.sms;   // (a wave without sharing)
    const bool wasteful = many && by8 * 3 <= 2 * p.sms && by8 * 80 > p.experts * pieces * 11;   // (more than a tenth of a block)
    int64_t tx = by8 * 8 <= p.sms || wasteful ? 4 : p.N % 16 && by8 >= 40 && !fills ? 16 : 8;
    while (tx < 64 && each < 512 && p.experts * ((pieces + tx - 1) / tx) > 5 * p.sms) tx *= 2;
    const int64_t blocks = (pieces + tx - 1) / tx, units = p.experts * blocks;
    int64_t ctas = 1;
    while (units * ctas * 2 <= 2 * p.sms && each >= 128 * ctas && (ctas < 8 || !p.dbias)) ctas *= 2;
    while (many && ctas < 8 && units * ctas < 512 && each >= 512 * ctas) ctas *= 2;
    int threads = !GATED ? (units <= 2 * p.sms ? 2 : 1) * kGradThreads
                  : (many && each >= 64 && ((ctas == 1 && units <= 2 * p.sms) || each >= 512 * ctas)) || (ctas == 1 && units <= p.sms) ? 2 * kGradThreads : kGradThreads;
    if (p.dbias && ctas == 8 && units * 16 <= 2 * p.sms && each >= 128 * 8) ctas = kGradMaxCtas, threads = kGradThreads;
    const int64_t grid = units * ctas;
    const size_t smem = (GATED ? 2 : 1) * (threads + tx) * 8 * sizeof(float);
    const auto kernel = linear_grad_kernel<KIND, GATED>;
    if (p.dbias && ctas > 8) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(kernel, dim3(static_cast<unsigned>(grid)), threads, smem, p.dbias ? static_cast<int>(ctas) : 1, stream, overlap, p,
                         static_cast<int>(tx), static_cast<int>(ctas), static_cast<int>(blocks));
}

}  // namespace

cudaError_t launch_linear_grad(int kind, const LinearGradParams &p, cudaStream_t stream, bool overlap)
{
    if (p.act & ACT_GATED) return kind == 0 ? go<0, true>(p, stream, overlap) : go<1, true>(p, stream, overlap);
    return kind == 0 ? go<0, false>(p, stream, overlap) : go<1, false>(p, stream, overlap);
}

}  // namespace pts
