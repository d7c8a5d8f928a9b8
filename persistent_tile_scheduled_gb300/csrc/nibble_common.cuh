// What the two forms of the product with 4-bit weights share: the weights' bits
// as exact 16-bit floats, and the blocks of rows of all experts.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_launch.h"
#include "ptx.cuh"

namespace pts {

namespace {

__device__ __forceinline__ uint32_t lds_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ float lds_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ void sts_f32(uint32_t addr, float v)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ void st_cluster_f32(uint32_t cluster_addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

// the low (0) or high (1) half of `pair`
template <int KIND>
__device__ __forceinline__ float widen(uint32_t pair, int half)
{
    if constexpr (KIND == 0) {
        const __half2 h = *reinterpret_cast<const __half2 *>(&pair);
        return half ? __high2float(h) : __low2float(h);
    } else {
        return __uint_as_float(half ? pair & 0xffff0000u : pair << 16);
    }
}

// (a & b) | c
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// 1024 + z (fp16) or 128 + z (bf16), twice, z being byte i of `zeros`
template <int KIND>
__device__ __forceinline__ uint32_t zero_bits(uint32_t zeros, int i)
{
    return __byte_perm(zeros, KIND == 0 ? 0x64u : 0x43u, 0x4040u + 0x101u * i);
}

template <int KIND>
__device__ __forceinline__ void nib_store(const NibbleParams &p, long long row, int n, float v)
{
    if constexpr (KIND == 0) static_cast<__half *>(p.c)[row * p.N + n] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p.c)[row * p.N + n] = __float2bfloat16_rn(v);
}

// A block of rows: its expert, its first row and how many.
struct NibBlock {
    int e, r0, cnt;
};

// Row blocks of all experts, at most as many as rows in that order make: offsets
// that go back and forth claim more, and are not followed that far.  Called by a
// whole warp.
template <int ROWS>
__device__ __forceinline__ int nib_blocks(const NibbleParams &p)
{
    if (!p.offsets) return (p.rows + ROWS - 1) / ROWS;
    uint32_t n = 0;
    const uint32_t most = static_cast<uint32_t>(p.max_blocks);
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
        const int i = e0 + static_cast<int>(lane_id());
        if (i < p.experts) {
            const int a = max(0, min(ld_global(p.offsets + i), p.rows)), b = max(a, min(ld_global(p.offsets + i + 1), p.rows));
            n = min(n + static_cast<uint32_t>((b - a + ROWS - 1) / ROWS), most);
        }
    }
    // (in two halves: 32 lanes' counts may pass 32 bits)
    const uint32_t low = __reduce_add_sync(0xffffffffu, n & 0xffffu), high = __reduce_add_sync(0xffffffffu, n >> 16);
    const unsigned long long all = (static_cast<unsigned long long>(high) << 16) + low;
    return static_cast<int>(all < most ? all : most);
}

// Expert and rows of a row block.  Called by a whole warp.
template <int ROWS>
__device__ __forceinline__ NibBlock nib_block(int block, const NibbleParams &p)
{
    const int lane = static_cast<int>(lane_id());
    int e = 0, lo = 0, hi = p.rows;
    uint32_t before = 0;   // row blocks before this one's expert, at most `block`
    if (p.offsets) {
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int i = e0 + lane;
            int a = 0, b = 0;
            if (i < p.experts) {
                a = max(0, min(ld_global(p.offsets + i), p.rows));
                b = max(a, min(ld_global(p.offsets + i + 1), p.rows));
            }
            // (saturating, for the offsets that claim too many)
            uint32_t incl = static_cast<uint32_t>((b - a + ROWS - 1) / ROWS);
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, incl, s);
                if (lane >= s) incl = min(incl + o, 0x7fffffffu);
            }
            const uint32_t past = __ballot_sync(0xffffffffu, before + incl > static_cast<uint32_t>(block));
            const int src = past ? __ffs(past) - 1 : 32;
            const uint32_t skipped = __shfl_sync(0xffffffffu, incl, (src - 1) & 31);
            if (src > 0) before += skipped;
            if (past) {
                e = e0 + src;
                lo = __shfl_sync(0xffffffffu, a, src);
                hi = __shfl_sync(0xffffffffu, b, src);
                break;
            }
        }
    }
    const int r0 = lo + (block - static_cast<int>(before)) * ROWS;
    return NibBlock{e, r0, min(hi - r0, ROWS)};
}

}  // namespace

}  // namespace pts
