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
// The grid is one CTA of 16 warps per SM, and stays: features rarely divide
// into 152 equal parts (16384 of them, 32 at a time, leave 16 % of the SMs idle
// in the last round), so each taker gets an equal stretch of blocks of 16
// features, which it walks 32 at a time.  The warps of a taker share the
// contraction, a unit of 256 each: a warp then meets the same values of the
// rows tile after tile and holds them in registers, where loading them for
// every tile cost as many bytes from L2 as the weights.  A taker is a cluster
// of 1, 2 or 4 CTAs, so that K up to 16384 has a warp per unit; for K below 4096
// a CTA holds several takers.  (A CTA per 32 features and 8 warps, with the
// rows loaded as they are needed: 35.2 us where this takes 25.8; 8 rows, 16384 x
// 8192, groups of 32 with zeros, bf16.)
// Weights arrive by TMA, 32 features x 128 contiguous bytes per unit: the MMA
// wants thread t of a quad to hold the 8 weights that are word t of a 16-byte
// chunk, where a thread's own 16-byte load would hold 32 consecutive weights,
// whose quad spans 128 and so up to four groups.  The 128-byte swizzle puts
// chunk c of row r at c ^ (r % 8): no bank conflicts.  The warps' sums of a tile
// meet in shared memory, those of a cluster's CTAs in the first one's, in a
// fixed order.
#pragma once
#include "nibble_common.cuh"

namespace pts {

namespace {

constexpr int kNibWarps = 16;
constexpr int kNibRing = 2;             // units in flight per warp
constexpr int kNibRows = 8;             // rows at a time: one MMA's
constexpr int kNibStageBytes = kNibFeatures * kNibStageK / 2;
constexpr int kNibSlots = 8;            // tiles whose sums a cluster gathers before they are stored
constexpr int kNibPitch = kNibFeatures + 4;           // floats between rows of a tile's sums: no bank conflicts
constexpr int kNibSums = kNibRows * kNibPitch;

__device__ __forceinline__ void bar_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
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
        if (mbar_try_wait_cta(bar, parity)) return true;
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

__device__ __forceinline__ uint4 ld_row(const uint16_t *p) { return ld_global(reinterpret_cast<const uint4 *>(p)); }

// Scales (pairs) and zeros (fours) of a unit's groups for one feature.
template <int GC>
struct NibScales {
    static constexpr int kGroups = kNibStageK / 32 / GC;   // groups per unit: 8, 4 or 2
    uint32_t s[kGroups / 2], z[(kGroups + 3) / 4];
};

// VEC: whole units of them, aligned.  Else one at a time, zeros behind the end.  (No branches around the loads: a value that meets another
// at the end of a branch would be waited for there.)
template <int GC, bool VEC, bool ZEROS>
__device__ __forceinline__ NibScales<GC> ld_scales(const uint16_t *sp, const uint8_t *zp, int first, int groups)
{
    constexpr int kGroups = NibScales<GC>::kGroups;
    NibScales<GC> r;
    if constexpr (VEC && kGroups == 8) {
        const uint4 v = ld_global(reinterpret_cast<const uint4 *>(sp + first));
        r.s[0] = v.x, r.s[1] = v.y, r.s[2] = v.z, r.s[3] = v.w;
        if constexpr (ZEROS) {
            const uint2 z = ld_global(reinterpret_cast<const uint2 *>(zp + first));
            r.z[0] = z.x, r.z[1] = z.y;
        }
    } else if constexpr (VEC && kGroups == 4) {
        const uint2 v = ld_global(reinterpret_cast<const uint2 *>(sp + first));
        r.s[0] = v.x, r.s[1] = v.y;
        if constexpr (ZEROS) r.z[0] = ld_global(reinterpret_cast<const uint32_t *>(zp + first));
    } else if constexpr (VEC) {
        r.s[0] = ld_global(reinterpret_cast<const uint32_t *>(sp + first));
        if constexpr (ZEROS) r.z[0] = ld_global(reinterpret_cast<const uint16_t *>(zp + first));
    } else {
        uint32_t s[kGroups], z[kGroups];
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            const int i = min(first + j, groups - 1);
            s[j] = ld_global(sp + i);
            if (first + j >= groups) s[j] = 0;   // (an infinite scale times the sum of nothing would be NaN)
            z[j] = ZEROS ? ld_global(zp + i) : 0;
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

// A tile whose sums wait to be stored.
struct NibTile {
    int n0, features, r0, cnt;
};

// A unit times the rows: acc += sum over its groups of scale * (rows . (q - z)).
// x: the rows' values, as the MMA takes them, zeros behind the contraction.
// buf: chunk c of this thread's first feature is at buf ^ (c << 4).
template <int KIND, int GC, bool ZEROS>
__device__ __forceinline__ void unit_sums(float (&acc)[2][4], uint32_t buf, int g, const uint4 (&x)[8], const NibScales<GC> &sc)
{
    constexpr int kGroups = NibScales<GC>::kGroups;
#pragma unroll
    for (int gi = 0; gi < kGroups; ++gi) {
        // the four features of this thread: g, g + 8, g + 16, g + 24
        float f[4];
        uint32_t zv[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f[q] = widen<KIND>(__shfl_sync(0xffffffffu, sc.s[gi / 2], g + 8 * q), gi & 1);
            zv[q] = zero_bits<KIND>(0x08080808u, 0);
            if constexpr (ZEROS) zv[q] = zero_bits<KIND>(__shfl_sync(0xffffffffu, sc.z[gi / 4], g + 8 * q), gi & 3);
        }
        float part[2][4];
#pragma unroll
        for (int ci = 0; ci < GC; ++ci) {
            const int c = gi * GC + ci;
            const uint32_t from = buf ^ (static_cast<uint32_t>(c) << 4);
            uint32_t w[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) expand<KIND>(lds_u32(from + q * 1024), zv[q], w[q]);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (ci == 0)
                    mma16816<KIND, true>(part[m], w[2 * m][0], w[2 * m + 1][0], w[2 * m][1], w[2 * m + 1][1], x[c].x, x[c].y);
                else
                    mma16816<KIND, false>(part[m], w[2 * m][0], w[2 * m + 1][0], w[2 * m][1], w[2 * m + 1][1], x[c].x, x[c].y);
                mma16816<KIND, false>(part[m], w[2 * m][2], w[2 * m + 1][2], w[2 * m][3], w[2 * m + 1][3], x[c].z, x[c].w);
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                acc[q >> 1][2 * (q & 1) + k] = fmaf(f[q], part[q >> 1][2 * (q & 1) + k], acc[q >> 1][2 * (q & 1) + k]);
    }
}

template <int KIND, int GC, bool VEC, bool ZEROS>
__global__ void __launch_bounds__(32 * kNibWarps, 1)
    nibble_kernel(const __grid_constant__ CUtensorMap tmB, const NibbleParams p)
{
    constexpr int kGroups = NibScales<GC>::kGroups;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sums0 = base + kNibWarps * kNibRing * kNibStageBytes;   // [2][warp][row][feature]
    const uint32_t gather = sums0 + 2 * kNibWarps * kNibSums * 4;          // [slot][CTA][row][feature], in the first CTA
    const uint32_t bars = gather + kNibSlots * kNibMaxCtas * kNibSums * 4;
    __shared__ NibTile gathered[kNibSlots];
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id());
    const int g = lane >> 2, t = lane & 3;
    const uint32_t one = lane == 0 ? 1u : 0u;
    const uint32_t ring = base + warp * (kNibRing * kNibStageBytes), my_bars = bars + warp * (8 * kNibRing);
    const int ctas = p.cluster;
    const int rank = ctas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    // takers of this CTA (several only in clusters of one) and this warp's place in its own
    const int kw = p.k_warps, group = warp / kw, takers = kNibWarps / kw;
    const int first_unit = rank * kw + warp % kw, unit_step = ctas * kw;
    const int units = (p.K + kNibStageK - 1) / kNibStageK;
    const int mine = units > first_unit ? (units - first_unit + unit_step - 1) / unit_step : 0;   // this warp's units of a tile
    const int all = (p.N + 15) / 16;

    if (lane == 0) {
        for (int i = 0; i < kNibRing; ++i) mbar_init(my_bars + 8 * i, 1);
        fence_mbar_init();
    }
    __syncwarp();
    if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // (this CTA has started)
    pdl_launch_dependents();
    auto begin_of = [&](int blocks, int part) -> int {
        const int parts = static_cast<int>(gridDim.x) / ctas * takers;
        return static_cast<int>(static_cast<long long>(blocks) * all * part / parts);
    };
    const int part = static_cast<int>(blockIdx.x) / ctas * takers + group;
    if (!p.offsets && mine > 0) {
        // one matrix: its place is known, so this warp's first unit may come
        // into L2 while the previous grid finishes (a prefetch changes no
        // loaded value)
        const int blocks = (p.rows + kNibRows - 1) / kNibRows, h = begin_of(blocks, part);
        if (h < begin_of(blocks, part + 1)) tma_prefetch_3d(one, &tmB, first_unit * 128, h % all * 16, 0);
    }
    pdl_wait();

    const int blocks = nib_blocks<kNibRows>(p);   // (blocks * all < 2^31: checked by the host)
    // blocks of 16 features are counted through the row blocks of all experts; a
    // taker's stretch of them is walked row block by row block
    int h = begin_of(blocks, part);
    const int h_end = begin_of(blocks, part + 1);
    int slot = 0, parity = 0, filled = 0;
    uint32_t phases = 0;   // bit i: the parity of ring barrier i that comes next
    bool ok = true;        // false: a load did not come; this warp asks for no more and adds what it has
    if (ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // (the others have started)

    while (h < h_end) {
        // the part of one row block that is this taker's: features n_begin .. n_end - 1
        const int block = h / all, n16 = h - block * all, count = min(h_end - h, all - n16);
        h += count;
        const NibBlock rows = nib_block<kNibRows>(block, p);
        const int n_begin = n16 * 16, n_end = min((n16 + count) * 16, p.N);
        const int row_b = rows.e * p.N;   // (experts * N < 2^31)
        // ask for the next unit
        int ld_n = n_begin, ld_unit = first_unit;
        auto load = [&](int i) {
            if (ld_n >= n_end || mine == 0 || !ok) return;
            mbar_arrive_expect_tx_if(one, my_bars + 8 * i, kNibStageBytes);
            tma_load_3d(one, ring + i * kNibStageBytes, &tmB, my_bars + 8 * i, ld_unit * 128, row_b + ld_n, 0);
            ld_unit += unit_step;
            if (ld_unit >= units) ld_unit = first_unit, ld_n += kNibFeatures;
        };
        for (int i = 0; i < kNibRing; ++i) load(slot ^ i);

        uint4 x[8];
        auto load_rows = [&](int unit) {
            // rows that are not there read the last one's values: their sums are not stored
            const uint16_t *xp = static_cast<const uint16_t *>(p.a) + static_cast<long long>(rows.r0 + min(g, rows.cnt - 1)) * p.K
                                 + unit * kNibStageK + t * 8;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                x[c] = make_uint4(0, 0, 0, 0);
                if (unit * kNibStageK + c * 32 < p.K) x[c] = ld_row(xp + c * 32);
            }
#pragma unroll
            for (int c = 0; c < 8; ++c)   // pairs (0, 4), (1, 5), (2, 6), (3, 7), as expand() leaves the weights
                x[c] = make_uint4(__byte_perm(x[c].x, x[c].z, 0x5410), __byte_perm(x[c].x, x[c].z, 0x7632),
                                  __byte_perm(x[c].y, x[c].w, 0x5410), __byte_perm(x[c].y, x[c].w, 0x7632));
        };
        // scales of this lane's feature (of the last one, where there is none)
        auto scales = [&](int n, int unit) {
            const long long f = static_cast<long long>(row_b + min(n + lane, p.N - 1)) * p.groups;
            return ld_scales<GC, VEC, ZEROS>(static_cast<const uint16_t *>(p.scales) + f, p.zeros + f, unit * kGroups, p.groups);
        };
        NibScales<GC> next = {};
        if (mine > 0) {
            next = scales(n_begin, first_unit);
            if (mine == 1) load_rows(first_unit);
        }

        for (int n = n_begin; n < n_end; n += kNibFeatures) {
            float acc[2][4] = {};
            for (int unit = first_unit; unit < units; unit += unit_step) {
                const NibScales<GC> sc = next;
                // (behind the last one its own again)
                const bool more = unit + unit_step < units;
                next = scales(more || n + kNibFeatures >= n_end ? n : n + kNibFeatures, more ? unit + unit_step : first_unit);
                if (mine > 1) load_rows(unit);
                ok = ok && __all_sync(0xffffffffu, wait(my_bars + 8 * slot, (phases >> slot) & 1u, p));
                if (!ok) break;
                phases ^= 1u << slot;
                unit_sums<KIND, GC, ZEROS>(acc, ring + slot * kNibStageBytes + g * 144 + t * 4, g, x, sc);
                __syncwarp();   // every lane is done with the unit before its slot is loaded again
                load(slot);
                slot ^= 1;
            }
            // the taker's warps add up; two sets of sums, so that one barrier per tile does
            const uint32_t to = sums0 + ((parity * kNibWarps + warp) * kNibSums + 2 * t * kNibPitch + g) * 4;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int k = 0; k < 2; ++k) sts_f32(to + (k * kNibPitch + 8 * q) * 4, acc[q >> 1][2 * (q & 1) + k]);
            if (kw > 1) bar_sync(1 + group, 32 * kw);   // (at most 8 takers then: 9 of the 16 barriers)
            else __syncwarp();
            const int r = warp - group * kw;
            for (int rr = r; rr < rows.cnt; rr += kw) {   // a warp per row, a lane per feature
                const uint32_t from = sums0 + ((parity * kNibWarps + group * kw) * kNibSums + rr * kNibPitch + lane) * 4;
                float v = 0.0f;
#pragma unroll 4
                for (int k = 0; k < kw; ++k) v += lds_f32(from + k * kNibSums * 4);
                if (ctas > 1)
                    st_cluster_f32(mapa(gather + ((filled * ctas + rank) * kNibSums + rr * kNibPitch + lane) * 4, 0u), v);
                else if (n + lane < n_end)
                    nib_store<KIND>(p, rows.r0 + rr, n + lane, v);
            }
            parity ^= 1;
            if (ctas == 1) continue;
            if (threadIdx.x == 0) gathered[filled] = NibTile{n, min(kNibFeatures, n_end - n), rows.r0, rows.cnt};
            const bool end = h == h_end && n + kNibFeatures >= n_end;
            if (++filled == kNibSlots || end) {
                cluster_sync();
                if (rank == 0)
                    for (int o = warp; o < filled * kNibRows; o += kNibWarps) {
                        const int s = o / kNibRows, i = o % kNibRows;
                        const NibTile w = gathered[s];
                        const uint32_t from = gather + (s * ctas * kNibSums + i * kNibPitch + lane) * 4;
                        float v = 0.0f;
                        for (int c = 0; c < ctas; ++c) v += lds_f32(from + c * kNibSums * 4);
                        if (i < w.cnt && lane < w.features) nib_store<KIND>(p, w.r0 + i, w.n0 + lane, v);
                    }
                filled = 0;
                if (!end) cluster_sync();   // the sums are read before the next ones come
            }
        }
    }
    if (!ok) {   // let what was asked for land before shared memory goes away (bounded)
        const uint64_t t0 = globaltimer_ns();
        for (int i = 0; i < kNibRing; ++i)
            while (!mbar_try_wait(my_bars + 8 * i, (phases >> i) & 1u) && globaltimer_ns() - t0 < 10000000ull) {
            }
    }
}

template <int KIND, int GC, bool VEC, bool ZEROS>
cudaError_t run(const CUtensorMap &b, NibbleParams p, NibPrepared *prepared, cudaStream_t stream, bool overlap)
{
    constexpr int smem = 1024 + kNibWarps * kNibRing * (kNibStageBytes + 8) + (2 * kNibWarps + kNibSlots * kNibMaxCtas) * kNibSums * 4;
    const auto kernel = nibble_kernel<KIND, GC, VEC, ZEROS>;
    const uint32_t bit = 1u << ((GC / 2 * 2 + VEC) * 2 + ZEROS);   // (GC / 2: 0, 1, 2)
    if (!(prepared->kernels & bit)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        prepared->kernels |= bit;
    }
    // Takers: of all ways to have a warp per unit, or several units per warp
    // (which then loads the rows' values for each: taken as a third more), the
    // one that leaves the fewest idle.
    const int units = (p.K + kNibStageK - 1) / kNibStageK;
    double least = 1e30;
    for (int c = 1; c <= kNibMaxCtas; c *= 2)
        for (int k = c == 1 ? 1 : kNibWarps; k <= kNibWarps; k *= 2) {
            const int each = units > 0 ? (units + c * k - 1) / (c * k) : 1;
            const double cost = static_cast<double>(each) * c * k * (each > 1 ? 1.33 : 1.0);
            if (cost <= least) least = cost, p.cluster = c, p.k_warps = k;
        }
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.blockDim = dim3(32 * kNibWarps, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (p.cluster > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
        int &resident = prepared->clusters[p.cluster / 2 - 1];
        if (resident == 0) {   // as many as the device holds at once (a GPC's SMs need not divide by 4)
            cfg.gridDim = dim3(static_cast<unsigned>(p.cluster), 1, 1);
            cudaError_t e = cudaOccupancyMaxActiveClusters(&resident, kernel, &cfg);
            if (e != cudaSuccess) return e;
            if (resident < 1) return cudaErrorInvalidConfiguration;
        }
        cfg.gridDim = dim3(static_cast<unsigned>(resident * p.cluster), 1, 1);
    } else {
        cfg.gridDim = dim3(static_cast<unsigned>(p.ctas), 1, 1);
    }
    if (overlap) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kernel, b, p);
}

template <int KIND, int GC>
cudaError_t by_alignment(const CUtensorMap &b, const NibbleParams &p, NibPrepared *prepared, cudaStream_t stream, bool overlap)
{
    if (p.groups % NibScales<GC>::kGroups == 0)
        return p.zeros ? run<KIND, GC, true, true>(b, p, prepared, stream, overlap)
                       : run<KIND, GC, true, false>(b, p, prepared, stream, overlap);
    return p.zeros ? run<KIND, GC, false, true>(b, p, prepared, stream, overlap)
                   : run<KIND, GC, false, false>(b, p, prepared, stream, overlap);
}

}  // namespace

// (one translation unit per kind: expert_launch.h names the two)
cudaError_t PTS_NIBBLE_LAUNCH(const CUtensorMap &b, const NibbleParams &p, NibPrepared *prepared, cudaStream_t stream,
                              bool overlap)
{
    return p.group == 32 ? by_alignment<PTS_NIBBLE_KIND, 1>(b, p, prepared, stream, overlap)
           : p.group == 64 ? by_alignment<PTS_NIBBLE_KIND, 2>(b, p, prepared, stream, overlap)
                           : by_alignment<PTS_NIBBLE_KIND, 4>(b, p, prepared, stream, overlap);
}

}  // namespace pts
