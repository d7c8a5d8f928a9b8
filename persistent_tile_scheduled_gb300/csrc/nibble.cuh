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
// group's sum is scaled in fp32, so no scaled weight is ever rounded.  (The
// 8-bit mma.sync would take the four bits as e4m3 subnormals, q * 2^-9, and
// the rows cut into e4m3 digits; that is exact too, but the instruction first
// unpacks both operands to fp16: 71 us where this form took 41.)
//
// A CTA takes 32 features of one expert (or the one matrix); its 8 warps share
// the contraction in whole units of 256 and add their sums up in shared memory
// in a fixed order.  Each warp has a ring of units of its own, filled by TMA
// (4 KB: 32 features x 128 contiguous bytes): the MMA wants thread t of a quad
// to hold the 8 weights that are word t of a 16-byte chunk, where a thread's
// own 16-byte load would hold 32 consecutive weights, whose quad spans 128 and
// so up to four groups.  The 128-byte swizzle puts chunk c of row r at
// c ^ (r % 8): no bank conflicts.  Two CTAs per SM keep the loads of one going
// while the other starts or adds up.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_launch.h"
#include "ptx.cuh"

namespace pts {

namespace {

constexpr int kNibWarps = 8;
constexpr int kNibRing = 3;             // units in flight per warp
constexpr int kNibStageBytes = kNibFeatures * kNibStageK / 2;
constexpr int kNibRows = 16;            // rows at a time

__device__ __forceinline__ uint32_t lds_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

template <int KIND>
__device__ __forceinline__ float widen(uint32_t bits)
{
    const uint16_t v = static_cast<uint16_t>(bits);
    if constexpr (KIND == 0) return __half2float(*reinterpret_cast<const __half *>(&v));
    else return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(&v));
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
        const __half2 zh = __hsub2(__float2half2_rn(960.0f), z);                            // -(64 + z)
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

// d = a . b + c, or a . b for FIRST
template <int KIND, bool FIRST>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
#define PTS_MMA(T_)                                                                                             \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." T_ "." T_ ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "            \
        "{%8, %9}, {%10, %11, %12, %13};"                                                                        \
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])                                                         \
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(FIRST ? 0.0f : c[0]),                        \
          "f"(FIRST ? 0.0f : c[1]), "f"(FIRST ? 0.0f : c[2]), "f"(FIRST ? 0.0f : c[3]))
    if constexpr (KIND == 0) PTS_MMA("f16");
    else PTS_MMA("bf16");
#undef PTS_MMA
}

// Wait for phase `parity` of `bar`, bounded: on time-out the handle's status
// block records it and the CTA goes on with what it has.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const NibbleParams &p)
{
    uint64_t t0 = 0;   // (the timer is slow to read: first after some tries)
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 255u) != 0) continue;
        if (t0 == 0) t0 = globaltimer_ns();
        if (globaltimer_ns() - t0 > p.timeout_ns) {
            if (atomicCAS(p.status, 0, DEV_ERR_TIMEOUT) == 0) {
                p.status[1] = 2;   // (waiting for a loaded stage)
                p.status[2] = static_cast<int32_t>(blockIdx.x);
            }
            atomicAdd(p.status + 3, 1);
            return false;
        }
    }
}

template <int KIND>
__device__ __forceinline__ void nib_store(const NibbleParams &p, long long row, int n, float v)
{
    if constexpr (KIND == 0) static_cast<__half *>(p.c)[row * p.N + n] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p.c)[row * p.N + n] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ uint4 ld_row(const uint16_t *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }

// Scales (pairs) and zeros (fours) of a unit's groups for one feature.
template <int GC>
struct NibScales {
    static constexpr int kGroups = kNibStageK / 32 / GC;   // groups per unit: 8, 4 or 2
    uint32_t s[kGroups / 2], z[(kGroups + 3) / 4];
};

// VEC: whole units of them, aligned.  Else one at a time, the last one again
// behind the end.  (No branches around the loads: a value that meets another
// at the end of a branch would be waited for there.)
template <int GC, bool VEC, bool ZEROS>
__device__ __forceinline__ NibScales<GC> ld_scales(const uint16_t *sp, const uint8_t *zp, int first, int groups)
{
    constexpr int kGroups = NibScales<GC>::kGroups;
    NibScales<GC> r;
    if constexpr (VEC && kGroups == 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(sp + first));
        r.s[0] = v.x, r.s[1] = v.y, r.s[2] = v.z, r.s[3] = v.w;
        if constexpr (ZEROS) {
            const uint2 z = __ldg(reinterpret_cast<const uint2 *>(zp + first));
            r.z[0] = z.x, r.z[1] = z.y;
        }
    } else if constexpr (VEC && kGroups == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(sp + first));
        r.s[0] = v.x, r.s[1] = v.y;
        if constexpr (ZEROS) r.z[0] = __ldg(reinterpret_cast<const uint32_t *>(zp + first));
    } else if constexpr (VEC) {
        r.s[0] = __ldg(reinterpret_cast<const uint32_t *>(sp + first));
        if constexpr (ZEROS) r.z[0] = __ldg(reinterpret_cast<const uint16_t *>(zp + first));
    } else {
        uint32_t s[kGroups], z[kGroups];
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            const int i = min(first + j, groups - 1);
            s[j] = __ldg(sp + i);
            z[j] = ZEROS ? __ldg(zp + i) : 0;
        }
#pragma unroll
        for (int j = 0; j < kGroups / 2; ++j) r.s[j] = s[2 * j] | s[2 * j + 1] << 16;
#pragma unroll
        for (int j = 0; j < (kGroups + 3) / 4; ++j) {
            r.z[j] = 0;
#pragma unroll
            for (int i = 0; i < 4 && 4 * j + i < kGroups; ++i) r.z[j] |= z[4 * j + i] << (8 * i);
        }
    }
    return r;
}

// Chunks of 32 of the rows' values that are on their way while the ones before
// them are used.
constexpr int kAhead = 2;

// The groups of half a unit (4 chunks of 32), times the rows:
// acc += scale * (rows . (q - z)).  ALL: it has its 4 chunks, x holds the first
// of them and, on return, those at xn; else the contraction ends in it and it
// has `here`.  buf: chunk c of this thread's row is at buf ^ (c << 4).  xp: this
// lane's row per block of 8.
template <int KIND, int NT, int GC, bool ZEROS, bool ALL>
__device__ __forceinline__ void half_sums(float (&acc)[NT][2][4], uint32_t buf, int g, uint4 (&x)[kAhead][NT],
                                          const uint16_t *const (&xp)[NT], const uint16_t *const (&xn)[NT],
                                          const NibScales<GC> &sc, int here)
{
#pragma unroll
    for (int gi = 0; gi < 4 / GC; ++gi) {
        if (!ALL && gi * GC >= here) break;
        // the four features of this thread: g, g + 8, g + 16, g + 24
        float f[4];
        uint32_t zv[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f[q] = widen<KIND>(__shfl_sync(0xffffffffu, sc.s[gi / 2], g + 8 * q) >> (16 * (gi & 1)));
            zv[q] = zero_bits<KIND>(0x08080808u, 0);
            if constexpr (ZEROS) zv[q] = zero_bits<KIND>(__shfl_sync(0xffffffffu, sc.z[0], g + 8 * q), gi);
        }
        float part[NT][2][4];
#pragma unroll
        for (int ci = 0; ci < GC; ++ci) {
            const int c = gi * GC + ci;
            if (!ALL && ci > 0 && c >= here) break;
            const uint32_t from = buf ^ (static_cast<uint32_t>(c) << 4);
            uint32_t w[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) expand<KIND>(lds_u32(from + q * 1024), zv[q], w[q]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                uint4 v;
                if constexpr (ALL) {
                    v = x[c % kAhead][j];
                    x[c % kAhead][j] = ld_row(c + kAhead < 4 ? xp[j] + (c + kAhead) * 32 : xn[j] + (c + kAhead - 4) * 32);
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
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float &to = acc[j][q >> 1][2 * (q & 1) + k];
                    to = fmaf(f[q], part[j][q >> 1][2 * (q & 1) + k], to);
                }
    }
}

// Rows r0 .. r0 + cnt - 1 of the expert at rows row_b .. of the weights, cnt at
// most 8 NT.  GC: chunks of 32 per group (group / 32).
template <int KIND, int NT, int GC, bool VEC, bool ZEROS>
__device__ __forceinline__ void nib_rows(const CUtensorMap &tmB, const NibbleParams &p, uint32_t ring, uint32_t bars,
                                         uint32_t &phases, float *sums, int n0, int row_b, int r0, int cnt)
{
    constexpr int kGroups = NibScales<GC>::kGroups;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id()), g = lane >> 2;
    const uint32_t one = lane == 0 ? 1u : 0u;
    const int units = (p.K + kNibStageK - 1) / kNibStageK;
    const int s0 = units * warp / kNibWarps, s1 = units * (warp + 1) / kNibWarps;
    auto load = [&](int s, int i) {
        if (s < s1) {
            mbar_arrive_expect_tx_if(one, bars + 8 * i, kNibStageBytes);
            tma_load_3d(one, ring + i * kNibStageBytes, &tmB, bars + 8 * i, s * 128, row_b, 0);
        }
    };
#pragma unroll
    for (int i = 0; i < kNibRing; ++i) load(s0 + i, i);

    float acc[NT][2][4] = {};
    if (s0 < s1) {
        // rows that are not there read the last one's values: their sums are not stored
        const uint16_t *xp[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
            xp[j] = static_cast<const uint16_t *>(p.a) + static_cast<long long>(r0 + min(8 * j + g, cnt - 1)) * p.K
                    + static_cast<long long>(s0) * kNibStageK + (lane & 3) * 8;
        // scales of this lane's feature (of the last one, where there is none)
        const long long at = static_cast<long long>(row_b + min(lane, p.N - 1 - n0)) * p.groups;
        const uint16_t *sp = static_cast<const uint16_t *>(p.scales) + at;
        const uint8_t *zp = p.zeros + at;
        NibScales<GC> next = ld_scales<GC, VEC, ZEROS>(sp, zp, s0 * kGroups, p.groups);
        const int full = min(p.K / kNibStageK, s1);   // whole units end here
        uint4 x[kAhead][NT] = {};
        if (s0 < full) {
#pragma unroll
            for (int c = 0; c < kAhead; ++c)
#pragma unroll
                for (int j = 0; j < NT; ++j) x[c][j] = ld_row(xp[j] + c * 32);
        }
        int i = 0;
#pragma unroll 1
        for (int s = s0; s < s1; ++s) {
            NibScales<GC> sc = next;
            next = ld_scales<GC, VEC, ZEROS>(sp, zp, min(s + 1, s1 - 1) * kGroups, p.groups);
            if (!wait(bars + 8 * i, (phases >> i) & 1u, p)) break;
            phases ^= 1u << i;
            uint32_t buf = ring + i * kNibStageBytes + g * 144 + (lane & 3) * 4;
            // two halves, in a loop: half the code to fetch where a warp has but a unit or two
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (s < full) {
                    // where no whole unit follows, what is fetched ahead is not used
                    const uint16_t *xn[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) xn[j] = h == 0 || s + 1 < full ? xp[j] + kNibStageK / 2 : xp[j];
                    half_sums<KIND, NT, GC, ZEROS, true>(acc, buf, g, x, xp, xn, sc, 4);
                } else {
                    half_sums<KIND, NT, GC, ZEROS, false>(acc, buf, g, x, xp, xp, sc, p.K / 32 - s * 8 - h * 4);
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) xp[j] += kNibStageK / 2;
                buf ^= 4u << 4;
                // the second half's groups
                if constexpr (GC == 1) sc.s[0] = sc.s[2], sc.s[1] = sc.s[3], sc.z[0] = sc.z[1];
                if constexpr (GC == 2) sc.s[0] = sc.s[1], sc.z[0] >>= 16;
                if constexpr (GC == 4) sc.s[0] >>= 16, sc.z[0] >>= 8;
            }
            __syncwarp();   // every lane is done with the unit before its slot is loaded again
            load(s + kNibRing, i);
            i = i + 1 == kNibRing ? 0 : i + 1;
        }
    }
    __syncthreads();   // the ring's memory becomes the sums'
    constexpr int kPitch = 8 * NT + 1;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float *to = sums + (warp * kNibFeatures + g + 8 * q) * kPitch + 8 * j + 2 * (lane & 3);
            to[0] = acc[j][q >> 1][2 * (q & 1)];
            to[1] = acc[j][q >> 1][2 * (q & 1) + 1];
        }
    __syncthreads();
    for (int o = threadIdx.x; o < cnt * kNibFeatures; o += 32 * kNibWarps) {
        const int r = o / kNibFeatures, f = o % kNibFeatures;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kNibWarps; ++k) v += sums[(k * kNibFeatures + f) * kPitch + r];
        if (n0 + f < p.N) nib_store<KIND>(p, r0 + r, n0 + f, v);
    }
}

template <int KIND, int GC, bool VEC, bool ZEROS>
__global__ void __launch_bounds__(32 * kNibWarps, 2)
    nibble_kernel(const __grid_constant__ CUtensorMap tmB, const NibbleParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    float *sums = reinterpret_cast<float *>(smem_raw + (base - raw));   // after the loop: [warp][feature][8 NT + 1]
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id());
    const int tiles = (p.N + kNibFeatures - 1) / kNibFeatures;
    const int slot = static_cast<int>(blockIdx.x) / tiles;   // which of the experts that have rows
    const int n0 = (static_cast<int>(blockIdx.x) - slot * tiles) * kNibFeatures;
    const uint32_t ring = base + warp * (kNibRing * kNibStageBytes);
    const uint32_t bars = base + kNibWarps * kNibRing * kNibStageBytes + warp * (8 * kNibRing);
    uint32_t phases = 0;   // bit i: the parity of ring barrier i that comes next

    if (lane == 0) {
        for (int i = 0; i < kNibRing; ++i) mbar_init(bars + 8 * i, 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_launch_dependents();
    // one matrix: its place is known, so its first units may come into L2
    // while the previous grid finishes (a prefetch changes no loaded value)
    if (!p.offsets) {
        const int units = (p.K + kNibStageK - 1) / kNibStageK, end = units * (warp + 1) / kNibWarps;
        for (int s = units * warp / kNibWarps, i = 0; s < end && i < kNibRing; ++s, ++i)
            tma_prefetch_3d(lane == 0 ? 1u : 0u, &tmB, s * 128, n0, 0);
    }
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
    const int row_b = e * p.N + n0;   // (experts * N < 2^31)

    for (int r0 = lo; r0 < hi; r0 += kNibRows) {
        const int cnt = min(hi - r0, kNibRows);
        if (cnt <= 8)
            nib_rows<KIND, 1, GC, VEC, ZEROS>(tmB, p, ring, bars, phases, sums, n0, row_b, r0, cnt);
        else
            nib_rows<KIND, 2, GC, VEC, ZEROS>(tmB, p, ring, bars, phases, sums, n0, row_b, r0, cnt);
        if (r0 + kNibRows < hi) {
            fence_proxy_async_smem();   // the sums' accesses before the next rows' TMA loads
            __syncthreads();
        }
    }
}

template <class... P, class... A>
cudaError_t go(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream, bool overlap, A... args)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (overlap) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int KIND, int GC, bool VEC>
cudaError_t run(const CUtensorMap &b, const NibbleParams &p, uint32_t *prepared, cudaStream_t stream, bool overlap)
{
    constexpr int smem = 1024 + kNibWarps * kNibRing * (kNibStageBytes + 8);
    static_assert(kNibRing * kNibStageBytes >= kNibFeatures * (kNibRows + 1) * 4, "the sums fit in the ring");
    const auto kernel = p.zeros ? nibble_kernel<KIND, GC, VEC, true> : nibble_kernel<KIND, GC, VEC, false>;
    const uint32_t bit = 1u << (((KIND * 3 + GC / 2) * 2 + VEC) * 2 + (p.zeros ? 1 : 0));   // (GC / 2: 0, 1, 2)
    if (!(*prepared & bit)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        *prepared |= bit;
    }
    // at most `rows` experts have rows
    const int64_t experts = p.offsets ? (p.experts < p.rows ? p.experts : p.rows) : 1;
    const int64_t ctas = (static_cast<int64_t>(p.N) + kNibFeatures - 1) / kNibFeatures * experts;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    return go(kernel, static_cast<unsigned>(ctas), 32 * kNibWarps, smem, stream, overlap, b, p);
}

template <int KIND, int GC>
cudaError_t by_alignment(const CUtensorMap &b, const NibbleParams &p, uint32_t *prepared, cudaStream_t stream, bool overlap)
{
    return p.groups % NibScales<GC>::kGroups == 0 ? run<KIND, GC, true>(b, p, prepared, stream, overlap)
                                                  : run<KIND, GC, false>(b, p, prepared, stream, overlap);
}

}  // namespace

// (one translation unit per kind: expert_launch.h names the two)
cudaError_t PTS_NIBBLE_LAUNCH(const CUtensorMap &b, const NibbleParams &p, uint32_t *prepared, cudaStream_t stream, bool overlap)
{
    return p.group == 32 ? by_alignment<PTS_NIBBLE_KIND, 1>(b, p, prepared, stream, overlap)
           : p.group == 64 ? by_alignment<PTS_NIBBLE_KIND, 2>(b, p, prepared, stream, overlap)
                           : by_alignment<PTS_NIBBLE_KIND, 4>(b, p, prepared, stream, overlap);
}

}  // namespace pts
