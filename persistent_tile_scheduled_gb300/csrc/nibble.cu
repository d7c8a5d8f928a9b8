// Few rows times 4-bit weights with a scale (and a zero) per group:
//
//   C[r, n] = sum_k A[r, k] (q_e[n, k] - z_e[n, k / group]) s_e[n, k / group]
//
// for the rows r of expert e (offsets on the device), or of the one matrix.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_launch.h"
#include "ptx.cuh"

namespace pts {

namespace {

template <int KIND>
__device__ __forceinline__ float widen(uint16_t v)
{
    if constexpr (KIND == 0) return __half2float(*reinterpret_cast<const __half *>(&v));
    else return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(&v));
}

// A warp per (feature, expert); lane l takes 8 weights (a 32-bit word) of every
// 256 and 4 rows at a time.
template <int KIND>
__global__ void __launch_bounds__(256) nibble_kernel(const NibbleParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int n = static_cast<int>(blockIdx.x) * 8 + static_cast<int>(threadIdx.x >> 5);
    const int lane = static_cast<int>(lane_id());
    if (n >= p.N) return;
    for (int e = blockIdx.y; e < p.experts; e += gridDim.y) {
        int lo = 0, hi = p.rows;
        if (p.offsets) {
            lo = max(0, min(p.offsets[e], p.rows));
            hi = max(lo, min(p.offsets[e + 1], p.rows));
        }
        const long long wrow = static_cast<long long>(e) * p.N + n;
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p.b) + wrow * (p.K / 8);
        const uint16_t *s = static_cast<const uint16_t *>(p.scales) + wrow * p.groups;
        const uint8_t *z = p.zeros ? p.zeros + wrow * p.groups : nullptr;
        for (int r0 = lo; r0 < hi; r0 += 4) {
            float acc[4] = {};
            for (int w = lane; w < p.K / 8; w += 32) {
                const uint32_t v = q[w];
                const int g = w * 8 / p.group;
                const float sc = widen<KIND>(s[g]), zero = z ? static_cast<float>(z[g]) : 8.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = (static_cast<float>((v >> (4 * i)) & 15u) - zero) * sc;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (r0 + j < hi)
                            acc[j] = fmaf(x, widen<KIND>(static_cast<const uint16_t *>(p.a)[static_cast<long long>(r0 + j) * p.K + 8 * w + i]), acc[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], d);
                if (lane == 0 && r0 + j < hi) {
                    const long long at = static_cast<long long>(r0 + j) * p.N + n;
                    if constexpr (KIND == 0) static_cast<__half *>(p.c)[at] = __float2half_rn(acc[j]);
                    else static_cast<__nv_bfloat16 *>(p.c)[at] = __float2bfloat16_rn(acc[j]);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_nibble(int kind, const NibbleParams &p, int sms, cudaStream_t stream, bool overlap)
{
    (void)sms;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>((p.N + 7) / 8), static_cast<unsigned>(p.experts < 65535 ? p.experts : 65535), 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    if (overlap) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kind == 0 ? nibble_kernel<0> : nibble_kernel<1>, p);
}

}  // namespace pts
