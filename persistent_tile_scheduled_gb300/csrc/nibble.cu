// Few rows times 4-bit weights with a scale (and a zero) per group:
//
//   C[r, n] = sum_g s_e[n, g] sum_{k in g} A[r, k] (q_e[n, k] - z_e[n, g])
//
// for the rows r of expert e (offsets on the device), or of the one matrix.
//
// The weights' bytes bound it (half a byte per product and row), so it streams
// them once and keeps the arithmetic per weight small.  A weight becomes an
// exact 16-bit float without conversions: its 4 bits are put into the low
// mantissa bits of 1024 (fp16) or 128 (bf16) by one three-input logic
// operation for two weights, and 1024 + z (128 + z) is subtracted, which is
// exact too.  The products go to mma.sync m16n8k16 (16 features x up to 8
// rows, fp32 sums): one row uses an eighth of it, and still the tensor pipe is
// idle most of the time, where fp32 multiply-adds would need two conversions
// and two instructions more per pair of weights.  tcgen05 would want the
// expanded weights in shared memory, four times the bytes that arrive.  A
// group's sum is scaled in fp32, so no scaled weight is ever rounded.
//
// A CTA takes 32 features; its 8 warps share the contraction in whole stages
// of 256 and add their sums up in shared memory in a fixed order.  Each warp
// has a ring of 3 stages of its own, filled by TMA (4 KB a stage: 32 features x
// 128 contiguous bytes): the MMA wants thread t of a quad to hold the 8 weights
// that are word t of a 16-byte chunk, where a thread's own 16-byte load would
// hold 32 consecutive weights, whose quad spans 128 and so up to four groups.
// The 128-byte swizzle puts chunk c of row r at c ^ (r % 8): no bank conflicts.
// Two CTAs per SM keep the loads of one going while the other starts or adds up.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_launch.h"
#include "ptx.cuh"

namespace pts {

namespace {

constexpr int kNibWarps = 8;
constexpr int kNibRing = 3;             // stages per warp
constexpr int kNibStageK = 256;         // contraction per stage
constexpr int kNibStageBytes = kNibFeatures * kNibStageK / 2;

__device__ __forceinline__ uint32_t lds_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// (a & b) | c
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// The 8 weights of a word minus their zero, as pairs (0, 4), (1, 5), (2, 6),
// (3, 7); zero: from zero_bits().
template <int KIND>
__device__ __forceinline__ void expand(uint32_t w, uint32_t zero, uint32_t (&o)[4])
{
    if constexpr (KIND == 0) {
        // low halves of the bytes: 1024 + q; high halves: 1024 + 16 q, times
        // 1/16 minus 64 + z.  Both exact.
        const uint32_t w8 = w >> 8;
        const __half2 z = *reinterpret_cast<const __half2 *>(&zero);                       // 1024 + z
        const __half2 sixteenth = __float2half2_rn(0.0625f);
        const __half2 zh = __hfma2(z, __float2half2_rn(-1.0f), __float2half2_rn(960.0f));   // -(64 + z)
        const uint32_t m = 0x64006400u;
        const uint32_t a = and_or(w, 0x000f000fu, m), b = and_or(w, 0x00f000f0u, m);
        const uint32_t c = and_or(w8, 0x000f000fu, m), d = and_or(w8, 0x00f000f0u, m);
        const __half2 r0 = __hsub2(*reinterpret_cast<const __half2 *>(&a), z);
        const __half2 r1 = __hfma2(*reinterpret_cast<const __half2 *>(&b), sixteenth, zh);
        const __half2 r2 = __hsub2(*reinterpret_cast<const __half2 *>(&c), z);
        const __half2 r3 = __hfma2(*reinterpret_cast<const __half2 *>(&d), sixteenth, zh);
        o[0] = *reinterpret_cast<const uint32_t *>(&r0);
        o[1] = *reinterpret_cast<const uint32_t *>(&r1);
        o[2] = *reinterpret_cast<const uint32_t *>(&r2);
        o[3] = *reinterpret_cast<const uint32_t *>(&r3);
    } else {
        const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162 *>(&zero);   // 128 + z
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = and_or(w >> (4 * i), 0x000f000fu, 0x43004300u);
            const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), z);
            o[i] = *reinterpret_cast<const uint32_t *>(&r);
        }
    }
}

// 1024 + z (fp16) or 128 + z (bf16), twice, z being byte i of `zeros`
template <int KIND>
__device__ __forceinline__ uint32_t zero_bits(uint32_t zeros, int i)
{
    return __byte_perm(zeros, KIND == 0 ? 0x64u : 0x43u, 0x4040u + 0x101u * i);
}

template <int KIND>
__device__ __forceinline__ float widen(uint32_t bits)
{
    const uint16_t v = static_cast<uint16_t>(bits);
    if constexpr (KIND == 0) return __half2float(*reinterpret_cast<const __half *>(&v));
    else return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(&v));
}

// d = a . b + c, or a . b for FIRST
template <int KIND, bool FIRST>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
#define PTS_MMA(T_)                                                                                             \
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." T_ "." T_ ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "   \
                 "{%8, %9}, {%10, %11, %12, %13};"                                                               \
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])                                                \
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(FIRST ? 0.0f : c[0]),               \
                   "f"(FIRST ? 0.0f : c[1]), "f"(FIRST ? 0.0f : c[2]), "f"(FIRST ? 0.0f : c[3]))
    if constexpr (KIND == 0) PTS_MMA("f16");
    else PTS_MMA("bf16");
#undef PTS_MMA
}

// Wait for phase `parity` of `bar`, bounded: on time-out the handle's status
// block records it and the CTA goes on with what it has.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const NibbleParams &p)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 15u) == 0 && globaltimer_ns() - t0 > p.timeout_ns) {
            if (atomicCAS(p.status, 0, DEV_ERR_TIMEOUT) == 0) {
                p.status[1] = 2;   // (waiting for a loaded stage)
                p.status[2] = static_cast<int32_t>(blockIdx.x);
            }
            atomicAdd(p.status + 3, 1);
            return false;
        }
    }
}

// What a warp needs to work on its CTA's features.
struct NibWarp {
    uint32_t ring, bars;            // its stages and their barriers
    int s_begin, s_end;             // its stages of the contraction
    int n0, row_b;                  // first feature, and its row in the weights
    const uint16_t *scales;         // of feature n0 + lane
    const uint8_t *zeros;           // null: 8
    bool there, vec;                // that feature exists; whole stages of scales are aligned
    uint32_t phases;                // bit i: the parity of ring barrier i that comes next
};

// Chunks of 32 of the rows' values that are on their way while the ones before
// them are used: with 16 warps per SM, loads from L2 are otherwise waited for.
__host__ __device__ constexpr int ahead(int nt) { return nt == 4 ? 2 : 4; }

__device__ __forceinline__ uint4 ld_row(const uint16_t *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }

// The groups of one stage: acc += scale * (rows . (q - z)).  ALL: the stage has
// its 8 chunks of 32, x holds the first `ahead` of them and, on return, those
// at xn; else the contraction ends in it and it has `here` chunks.
template <int KIND, int NT, int GC, bool ALL>
__device__ __forceinline__ void stage_sums(float (&acc)[NT][2][4], uint32_t buf, int g, uint4 (&x)[ahead(NT)][NT],
                                           const uint16_t *const (&xp)[NT], const uint16_t *const (&xn)[NT],
                                           const uint32_t *sc, const uint32_t *zr, int here)
{
    constexpr int kGroups = kNibStageK / 32 / GC;
    constexpr int D = ahead(NT);
#pragma unroll
    for (int gi = 0; gi < kGroups; ++gi) {
        if (!ALL && gi * GC >= here) break;
        // the four features of this thread: g, g + 8, g + 16, g + 24
        uint32_t sv[4], zv[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            sv[q] = __shfl_sync(0xffffffffu, sc[gi / 2], g + 8 * q);
            zv[q] = zero_bits<KIND>(__shfl_sync(0xffffffffu, zr[gi / 4], g + 8 * q), gi & 3);
        }
        float part[NT][2][4];
#pragma unroll
        for (int ci = 0; ci < GC; ++ci) {
            const int c = gi * GC + ci;
            if (!ALL && ci > 0 && c >= here) break;
            const uint32_t at = buf + (static_cast<uint32_t>(c ^ g) << 4);
            uint32_t w[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) expand<KIND>(lds_u32(at + q * 1024), zv[q], w[q]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                uint4 v;
                if constexpr (ALL) {
                    v = x[c % D][j];
                    x[c % D][j] = ld_row(c + D < 8 ? xp[j] + (c + D) * 32 : xn[j] + (c + D - 8) * 32);
                } else {
                    v = ld_row(xp[j] + c * 32);
                }
                // pairs (0, 4), (1, 5), (2, 6), (3, 7), as expand() leaves the weights
                const uint32_t b0 = __byte_perm(v.x, v.z, 0x5410), b1 = __byte_perm(v.x, v.z, 0x7632);
                const uint32_t b2 = __byte_perm(v.y, v.w, 0x5410), b3 = __byte_perm(v.y, v.w, 0x7632);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    if (ci == 0)
                        mma16816<KIND, true>(part[j][m], w[2 * m][0], w[2 * m + 1][0], w[2 * m][1], w[2 * m + 1][1], b0, b1);
                    else
                        mma16816<KIND, false>(part[j][m], w[2 * m][0], w[2 * m + 1][0], w[2 * m][1], w[2 * m + 1][1], b0, b1);
                    mma16816<KIND, false>(part[j][m], w[2 * m][2], w[2 * m + 1][2], w[2 * m][3], w[2 * m + 1][3], b2, b3);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float f = widen<KIND>(sv[q] >> (16 * (gi & 1)));
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float *to = &acc[j][q >> 1][2 * (q & 1)];
                const float *from = &part[j][q >> 1][2 * (q & 1)];
                to[0] = fmaf(f, from[0], to[0]);
                to[1] = fmaf(f, from[1], to[1]);
            }
        }
    }
}

// Rows r0 .. r0 + cnt - 1 (cnt <= 8 NT) of the CTA's expert.  GC: chunks of 32
// per group (group / 32).
template <int KIND, int NT, int GC>
__device__ __forceinline__ void nibble_rows(const CUtensorMap &tmB, const NibbleParams &p, NibWarp &w, float *sums,
                                            int r0, int cnt)
{
    constexpr int kGroups = kNibStageK / 32 / GC;        // groups per stage: 8, 4 or 2
    constexpr int kS = kGroups / 2, kZ = (kGroups + 3) / 4;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id());
    const int g = lane >> 2, t = lane & 3;
    const uint32_t one = lane == 0 ? 1u : 0u;
    // rows that are not there read the last one's values: their sums are not stored
    const uint16_t *xp[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
        xp[j] = static_cast<const uint16_t *>(p.a) + static_cast<long long>(r0 + min(8 * j + g, cnt - 1)) * p.K
                + static_cast<long long>(w.s_begin) * kNibStageK + t * 8;
    auto load_stage = [&](int s, int i) {
        if (s < w.s_end) {
            mbar_arrive_expect_tx_if(one, w.bars + 8 * i, kNibStageBytes);
            tma_load_3d(one, w.ring + i * kNibStageBytes, &tmB, w.bars + 8 * i, s * 128, w.row_b, 0);
        }
    };
    // this lane's scales (pairs) and zeros (fours) of a stage's groups
    uint32_t sc[kS], zr[kZ];
    auto load_scales = [&](int s) {
#pragma unroll
        for (int j = 0; j < kS; ++j) sc[j] = 0u;
#pragma unroll
        for (int j = 0; j < kZ; ++j) zr[j] = 0x08080808u;
        if (!w.there || s >= w.s_end) return;
        const int gi = s * kGroups;
        const uint16_t *sp = w.scales + gi;
        const uint8_t *zp = w.zeros + gi;
        if (w.vec) {
            if constexpr (kGroups == 8) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(sp));
                sc[0] = v.x, sc[1] = v.y, sc[2] = v.z, sc[3] = v.w;
                if (w.zeros) {
                    const uint2 z = __ldg(reinterpret_cast<const uint2 *>(zp));
                    zr[0] = z.x, zr[1] = z.y;
                }
            } else if constexpr (kGroups == 4) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(sp));
                sc[0] = v.x, sc[1] = v.y;
                if (w.zeros) zr[0] = __ldg(reinterpret_cast<const uint32_t *>(zp));
            } else {
                sc[0] = __ldg(reinterpret_cast<const uint32_t *>(sp));
                if (w.zeros) zr[0] = __ldg(reinterpret_cast<const uint16_t *>(zp));
            }
        } else {
#pragma unroll
            for (int j = 0; j < kGroups; ++j)
                if (gi + j < p.groups) {
                    sc[j / 2] |= static_cast<uint32_t>(__ldg(sp + j)) << (16 * (j & 1));
                    if (w.zeros)
                        zr[j / 4] = (zr[j / 4] & ~(255u << (8 * (j & 3)))) | (static_cast<uint32_t>(__ldg(zp + j)) << (8 * (j & 3)));
                }
        }
    };
#pragma unroll
    for (int i = 0; i < kNibRing; ++i) load_stage(w.s_begin + i, i);
    load_scales(w.s_begin);

    const int full = p.K / kNibStageK;   // stages below this one are whole
    uint4 x[ahead(NT)][NT] = {};
    if (w.s_begin < min(full, w.s_end)) {
#pragma unroll
        for (int c = 0; c < ahead(NT); ++c)
#pragma unroll
            for (int j = 0; j < NT; ++j) x[c][j] = ld_row(xp[j] + c * 32);
    }
    float acc[NT][2][4] = {};
    int i = 0;   // ring slot of stage s
    for (int s = w.s_begin; s < w.s_end; ++s) {
        uint32_t nsc[kS], nzr[kZ];
#pragma unroll
        for (int j = 0; j < kS; ++j) nsc[j] = sc[j];
#pragma unroll
        for (int j = 0; j < kZ; ++j) nzr[j] = zr[j];
        load_scales(s + 1);
        if (!wait(w.bars + 8 * i, (w.phases >> i) & 1u, p)) break;
        w.phases ^= 1u << i;
        const uint32_t buf = w.ring + i * kNibStageBytes + g * 128 + t * 4;
        if (s < full) {
            // where no whole stage follows, what is fetched ahead is not used
            const uint16_t *xn[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) xn[j] = s + 1 < min(full, w.s_end) ? xp[j] + kNibStageK : xp[j];
            stage_sums<KIND, NT, GC, true>(acc, buf, g, x, xp, xn, nsc, nzr, 8);
        } else {
            stage_sums<KIND, NT, GC, false>(acc, buf, g, x, xp, xp, nsc, nzr, p.K / 32 - s * 8);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) xp[j] += kNibStageK;
        __syncwarp();   // every lane is done with the stage before its slot is loaded again
        load_stage(s + kNibRing, i);
        i = i + 1 == kNibRing ? 0 : i + 1;
    }
    __syncthreads();   // the ring's memory becomes the sums'
    constexpr int kPitch = 8 * NT + 1;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float *to = sums + (warp * kNibFeatures + g + 8 * q) * kPitch + 8 * j + 2 * t;
            to[0] = acc[j][q >> 1][2 * (q & 1)];
            to[1] = acc[j][q >> 1][2 * (q & 1) + 1];
        }
    __syncthreads();
    for (int o = threadIdx.x; o < cnt * kNibFeatures; o += 32 * kNibWarps) {
        const int r = o / kNibFeatures, f = o % kNibFeatures;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kNibWarps; ++k) v += sums[(k * kNibFeatures + f) * kPitch + r];
        if (w.n0 + f < p.N) {
            const long long to = static_cast<long long>(r0 + r) * p.N + w.n0 + f;
            if constexpr (KIND == 0) static_cast<__half *>(p.c)[to] = __float2half_rn(v);
            else static_cast<__nv_bfloat16 *>(p.c)[to] = __float2bfloat16_rn(v);
        }
    }
}

template <int KIND, int GC>
__global__ void __launch_bounds__(32 * kNibWarps, 2)
    nibble_kernel(const __grid_constant__ CUtensorMap tmB, const NibbleParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    float *sums = reinterpret_cast<float *>(smem_raw + (base - raw));   // after the loop: [warp][feature][8 NT + 1]
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id());
    const int tiles = (p.N + kNibFeatures - 1) / kNibFeatures;
    const int slot = static_cast<int>(blockIdx.x) / tiles;   // which of the experts that have rows
    const int stages = (p.K + kNibStageK - 1) / kNibStageK;
    NibWarp w;
    w.n0 = (static_cast<int>(blockIdx.x) - slot * tiles) * kNibFeatures;
    w.ring = base + warp * (kNibRing * kNibStageBytes);
    w.bars = base + kNibWarps * kNibRing * kNibStageBytes + warp * (8 * kNibRing);
    w.s_begin = stages * warp / kNibWarps;
    w.s_end = stages * (warp + 1) / kNibWarps;
    w.phases = 0;

    if (lane == 0) {
        for (int i = 0; i < kNibRing; ++i) mbar_init(w.bars + 8 * i, 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_launch_dependents();
    // one matrix: its place is known, so its first stages may come into L2
    // while the previous grid finishes (a prefetch changes no loaded value)
    if (!p.offsets)
        for (int s = w.s_begin; s < w.s_end && s < w.s_begin + kNibRing; ++s)
            tma_prefetch_3d(lane == 0 ? 1u : 0u, &tmB, s * 128, w.n0, 0);
    pdl_wait();

    // this CTA's expert: the slot-th that has rows
    int e = 0, lo = 0, hi = p.rows;
    if (p.offsets) {
        int seen = 0;
        bool found = false;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int i = e0 + lane;
            int a = 0, b = 0;
            if (i < p.experts) {
                a = max(0, min(__ldg(p.offsets + i), p.rows));
                b = max(a, min(__ldg(p.offsets + i + 1), p.rows));
            }
            const uint32_t some = __ballot_sync(0xffffffffu, b > a);
            // lane whose expert is the (slot - seen)-th set bit
            const bool mine = ((some >> lane) & 1u) && __popc(some & ((1u << lane) - 1u)) == slot - seen;
            const uint32_t at = __ballot_sync(0xffffffffu, mine);
            if (at) {
                const int src = __ffs(at) - 1;
                e = e0 + src;
                lo = __shfl_sync(0xffffffffu, a, src);
                hi = __shfl_sync(0xffffffffu, b, src);
                found = true;
                break;
            }
            seen += __popc(some);
        }
        if (!found) return;
    }
    w.row_b = e * p.N + w.n0;   // (experts * N < 2^31)
    w.there = w.n0 + lane < p.N;
    const long long feature = static_cast<long long>(w.row_b + lane) * p.groups;
    w.scales = static_cast<const uint16_t *>(p.scales) + feature;
    w.zeros = p.zeros ? p.zeros + feature : nullptr;
    w.vec = p.groups % (kNibStageK / 32 / GC) == 0;

    for (int r0 = lo; r0 < hi; r0 += 32) {
        const int cnt = min(hi - r0, 32);
        if (cnt <= 8)
            nibble_rows<KIND, 1, GC>(tmB, p, w, sums, r0, cnt);
        else if (cnt <= 16)
            nibble_rows<KIND, 2, GC>(tmB, p, w, sums, r0, cnt);
        else
            nibble_rows<KIND, 4, GC>(tmB, p, w, sums, r0, cnt);
        if (r0 + 32 < hi) {
            fence_proxy_async_smem();   // the sums' accesses before the next rows' TMA loads
            __syncthreads();
        }
    }
}

template <int KIND, int GC>
cudaError_t go(const CUtensorMap &b, const NibbleParams &p, cudaStream_t stream, bool overlap)
{
    constexpr int smem = 1024 + kNibWarps * kNibRing * (kNibStageBytes + 8);
    static_assert(kNibRing * kNibStageBytes >= kNibFeatures * (8 * 4 + 1) * 4, "the sums fit in the ring");
    cudaError_t e = cudaFuncSetAttribute(nibble_kernel<KIND, GC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    // at most `rows` experts have rows
    const int64_t experts = p.offsets ? (p.experts < p.rows ? p.experts : p.rows) : 1;
    const int64_t ctas = (static_cast<int64_t>(p.N) + kNibFeatures - 1) / kNibFeatures * experts;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(32 * kNibWarps, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (overlap) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, nibble_kernel<KIND, GC>, b, p);
}

template <int KIND>
cudaError_t by_group(const CUtensorMap &b, const NibbleParams &p, cudaStream_t stream, bool overlap)
{
    return p.group == 32 ? go<KIND, 1>(b, p, stream, overlap)
           : p.group == 64 ? go<KIND, 2>(b, p, stream, overlap)
                           : go<KIND, 4>(b, p, stream, overlap);
}

}  // namespace

cudaError_t launch_nibble(int kind, const CUtensorMap &b, const NibbleParams &p, cudaStream_t stream, bool overlap)
{
    return kind == 0 ? by_group<0>(b, p, stream, overlap) : by_group<1>(b, p, stream, overlap);
}

}  // namespace pts
