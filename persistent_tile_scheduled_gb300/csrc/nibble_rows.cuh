// More rows times 4-bit weights: the same product as nibble.cuh, for blocks of
// up to 32 or 64 rows, on tcgen05.
//
// With a row block of 8 the weights are made into 16-bit floats once for every
// 8 rows, and that is where the time goes.  Here they are expanded once per
// block, into shared memory as an operand of 128 features x 64 (128-byte
// swizzle), exactly as there: q - z is a small integer.  A tcgen05.mma has 128
// features on its M side and the rows on its N side.  Every scale group is a sum
// of its own in TMEM, read back by the warp that holds these features and added
// with its scale in fp32, so that no scaled weight is rounded here either: in
// TMEM a lane is a feature, which has one scale per group.
//
// Warp roles: TMA producer (a stage: 256 of the contraction, the packed weights
// of 128 features and the rows), MMA, warps that scale and sum (4 per 32 rows),
// warps that expand.  They hand on units of 256 or 128 of the contraction, two
// of each in flight: the expanded weights and the sums of their groups.
// A tile is 128 features x one row block.  Either a CTA takes one tile after
// another, the loads and the expanding running ahead into the next; or a cluster
// of 2 or 4 CTAs shares a tile's contraction and adds up through distributed
// shared memory, every CTA its part of the rows, in order.  The latter is for
// fewer tiles than SMs, but also for a few more, whose last round would leave most
// SMs idle (64 rows of 20480 x 16384, 160 tiles: 4 CTAs to each, in several
// rounds, 147 us, 2 CTAs 155, one 184): the caller reckons which.
//
// What bounds it (bf16, groups of 64): 32 rows of 8192^2 take 19.4 us, 8 at a time
// 37; 64 rows 29.3 and 69; 512 rows of 4096^2 49.7 and 121.  A CTA spends 0.95 us on
// 256 of its contraction (1.5 for 64 rows), mostly in the expanding warps: loads,
// barriers and scales alone 0.45, the MMAs 0.3, the expanding 0.5; start and end
// take 5 us, so that few weights are better off in nibble.cuh.  One elected lane
// issues the MMAs: under a predicate of its own each took some 200 cycles (49 us
// where the rest took 31).
#pragma once
#include "gemm_kernel.cuh"
#include "nibble_common.cuh"

namespace pts {

namespace {

constexpr int kNrScaleWarp0 = 2;
constexpr int kNrPackedBytes = kNibWideFeatures * kNibStageK / 2;
constexpr int kNrBlockBytes = kNibWideFeatures * 128;      // an expanded block: 128 features x 64 of the contraction

template <int RB>
struct NibRowsShape {
    static constexpr int kUnit = RB == 32 ? 4 : 2;         // blocks of 64 of a unit
    static constexpr int kUnits = 2;                       // in flight
    static constexpr int kStages = 3;
    static constexpr int kScaleWarps = RB / 8;
    static constexpr int kTeams = RB == 32 ? 2 : 1;        // of 8 expanding warps, each every kTeams-th unit
    static constexpr int kExpandWarps = 8 * kTeams;
    static constexpr int kExpandWarp0 = kNrScaleWarp0 + kScaleWarps;
    static constexpr int kThreads = 32 * (kExpandWarp0 + kExpandWarps);
    static constexpr int kStageBytes = kNrPackedBytes + 4 * RB * 128;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kUnits * kUnit * kNrBlockBytes
                                 + 8 * (2 * kStages + 4 * kUnits + 1) + 16;
};

// The 8 weights of a word minus their zero, in order: (0, 1), (2, 3), (4, 5), (6, 7).
template <int KIND>
__device__ __forceinline__ void expand_in_order(uint32_t w, uint32_t zero, uint32_t (&o)[4])
{
    const uint32_t magic = KIND == 0 ? 0x64u : 0x43u;
    const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
    // bytes: weights 0 .. 3, 4 .. 7
    const uint32_t lo = __byte_perm(even, odd, 0x5140), hi = __byte_perm(even, odd, 0x7362);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = __byte_perm(i < 2 ? lo : hi, magic, i & 1 ? 0x4342 : 0x4140);       // 1024 + q or 128 + q
        if constexpr (KIND == 0) {
            const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&zero));
            o[i] = *reinterpret_cast<const uint32_t *>(&r);
        } else {
            const __nv_bfloat162 r =
                __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&zero));
            o[i] = *reinterpret_cast<const uint32_t *>(&r);
        }
    }
}

// The scales of N groups of a feature, `first` the first, two to a register; and
// their zeros, four to a register, left as they are where `given` is 0.  VEC: all
// there and aligned, one load; else one by one, the last one again behind the end.
// A lane has a feature, so every load touches 32 lines: one load per group took a
// third of the time (31 us where the rest took 20.6).  There is no branch around a
// load, since it would be waited for at the branch's end.
template <int N, bool VEC>
__device__ __forceinline__ void load_group_scales(const uint16_t *p, int first, int groups, uint32_t (&v)[(N + 1) / 2])
{
    if constexpr (VEC && N == 8) {
        const uint4 x = ld_global(reinterpret_cast<const uint4 *>(p + first));
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else if constexpr (VEC && N == 4) {
        const uint2 x = ld_global(reinterpret_cast<const uint2 *>(p + first));
        v[0] = x.x, v[1] = x.y;
    } else if constexpr (VEC && N == 2) {
        v[0] = ld_global(reinterpret_cast<const uint32_t *>(p + first));
    } else {
        uint32_t one[N];
#pragma unroll
        for (int i = 0; i < N; ++i) one[i] = ld_global(p + min(first + i, groups - 1));
#pragma unroll
        for (int i = 0; i < (N + 1) / 2; ++i) {
            v[i] = one[2 * i];
            if constexpr (N > 1) v[i] |= one[2 * i + 1] << 16;
        }
    }
}

template <int N, bool VEC>
__device__ __forceinline__ void load_group_zeros(uint32_t given, const uint8_t *p, int first, int groups,
                                                 uint32_t (&v)[(N + 3) / 4])
{
    if constexpr (VEC && N == 8) {
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q ld.global.v2.b32 {%0, %1}, [%3];\n\t}"
                     : "+r"(v[0]), "+r"(v[1]) : "r"(given), "l"(p + first));
    } else if constexpr (VEC && N == 4) {
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q ld.global.b32 %0, [%2];\n\t}"
                     : "+r"(v[0]) : "r"(given), "l"(p + first));
    } else if constexpr (VEC && N == 2) {
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q ld.global.u16 %0, [%2];\n\t}"
                     : "+r"(v[0]) : "r"(given), "l"(p + first));
    } else {
        uint32_t one[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            one[i] = 8;
            asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q ld.global.u8 %0, [%2];\n\t}"
                         : "+r"(one[i]) : "r"(given), "l"(p + min(first + i, groups - 1)));
        }
#pragma unroll
        for (int j = 0; j < (N + 3) / 4; ++j) {
            v[j] = 0;
#pragma unroll
            for (int i = 0; i < 4 && 4 * j + i < N; ++i) v[j] |= one[4 * j + i] << (8 * i);
        }
    }
}

template <int KIND, int RB, int GC, bool VEC>
__global__ void __launch_bounds__(NibRowsShape<RB>::kThreads, 1)
    nibble_rows_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmX,
                       const NibbleParams p)
{
    using Shape = NibRowsShape<RB>;
    constexpr int S = Shape::kStages, NU = Shape::kUnits, U = Shape::kUnit;
    constexpr int kPerStage = 4 / U;                        // units of a stage
    constexpr int kGroups = 2 * U / GC;                     // groups of a unit
    constexpr int kSet = kGroups * RB;                      // TMEM columns of a unit's sums
    constexpr int kUnitK = 64 * U, kTeams = Shape::kTeams;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t blocks0 = base + S * Shape::kStageBytes;
    const uint32_t full0 = blocks0 + NU * U * kNrBlockBytes;   // + 8*s: a stage is loaded
    const uint32_t empty0 = full0 + 8 * S;                  // + 8*s: and used up
    const uint32_t ready0 = empty0 + 8 * S;                 // + 8*u: a unit is expanded
    const uint32_t used0 = ready0 + 8 * NU;                 // + 8*u: its MMAs are through: expand the next
    const uint32_t sum0 = used0 + 8 * NU;                   // + 8*u: and read the sums
    const uint32_t taken0 = sum0 + 8 * NU;                  // + 8*u: they are read
    const uint32_t done = taken0 + 8 * NU;                  // every MMA is through
    const uint32_t tmem_slot = done + 8, abort_flag = tmem_slot + 4;

    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id());
    const uint32_t one = lane == 0 ? 1u : 0u;
    const int ctas = p.cluster, rank = ctas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int tiles_n = (p.N + kNibWideFeatures - 1) / kNibWideFeatures;
    // this CTA's stages of the contraction
    const int stages = (p.K + kNibStageK - 1) / kNibStageK;
    const int first = static_cast<int>(static_cast<long long>(stages) * rank / ctas);
    const int last = static_cast<int>(static_cast<long long>(stages) * (rank + 1) / ctas);

    WaitCtl ctl;
    ctl.abort_addr = abort_flag;
    ctl.peer_abort = 0;
    ctl.timeout_ns = p.timeout_ns;
    ctl.status = p.status;
    // (as WaitCtl::wait_all, but that the timer, slow to read, is left alone for 256 tries)
    auto wait_all = [&](uint32_t bar, uint32_t parity, int32_t where) -> bool {
        bool mine = false;
        for (int n = 0; n < 256 && !mine; ++n) mine = mbar_try_wait_cta(bar, parity);
        return __all_sync(0xffffffffu, mine) || ctl.wait_all(bar, parity, where);
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 8 * (kTeams < kPerStage ? kTeams : kPerStage) + 1);
        }
        for (int u = 0; u < NU; ++u) {
            mbar_init(ready0 + 8 * u, 8);
            mbar_init(used0 + 8 * u, 1);
            mbar_init(sum0 + 8 * u, 1);
            mbar_init(taken0 + 8 * u, Shape::kScaleWarps);
        }
        mbar_init(done, 1);
        st_shared_u32(abort_flag, 0u);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc<1>(tmem_slot, NU * kSet);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ld_shared_u32(tmem_slot);
    pdl_launch_dependents();
    pdl_wait();

    const int units_end = (p.K + kUnitK - 1) / kUnitK;   // units of the whole contraction
    const int u_first = first * kPerStage, u_last = min(last * kPerStage, units_end);
    // tiles of this CTA: row block by row block, the features of one next to one another (a cluster has one at most)
    const int tiles = nib_blocks<RB>(p) * tiles_n, stride = static_cast<int>(gridDim.x) / ctas;
    const int tile0 = static_cast<int>(blockIdx.x) / ctas;
    struct Tile {
        NibBlock rows;
        int n0, row_b;   // first feature; rows of the weights before the expert's (experts * N < 2^31)
    };
    auto tile_at = [&](int tile) -> Tile {
        const int block = tile / tiles_n;
        const NibBlock rows = nib_block<RB>(block, p);
        return Tile{rows, (tile - block * tiles_n) * kNibWideFeatures, rows.e * p.N};
    };
    float acc[32];

    if (warp == 0) {
        // =============================== producer ==============================
        bool ok = true;
        int issued = 0, s = 0;
        uint32_t phase = 0;
        for (int tile = tile0; ok && tile < tiles; tile += stride) {
            const Tile t = tile_at(tile);
            for (int st = first; st < last; ++st) {
                ok = wait_all(empty0 + 8 * s, phase ^ 1u, WHERE_EMPTY);
                if (!ok) break;
                const uint32_t at = base + s * Shape::kStageBytes;
                const int k0 = st * kNibStageK;
                if (elect_one()) {   // (a box behind the end of the contraction is zeros)
                    // (test hook: more bytes than come, so that a bounded wait on this stage runs out)
                    mbar_arrive_expect_tx_if(1u, full0 + 8 * s, kNrPackedBytes + 4 * (RB * 128) + (issued == p.fault_load ? 16u : 0u));
                    tma_load_3d(1u, at, &tmB, full0 + 8 * s, k0 / 2, t.row_b + t.n0, 0);
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        tma_load_3d(1u, at + kNrPackedBytes + b * (RB * 128), &tmX, full0 + 8 * s, k0 + b * 64, t.rows.r0, 0);
                }
                __syncwarp();
                ++issued;
                if (++s == S) s = 0, phase ^= 1u;
            }
        }
        // Every load that was issued lands before the CTA can exit (bounded), also where
        // another warp gave up on a stage after the last load was issued.
        for (int j = max(0, issued - S); j < issued; ++j) ctl.drain(full0 + 8 * (j % S), (j / S) & 1, 10000000ull);
    } else if (warp == 1) {
        // ================================ MMA ==================================
        constexpr uint32_t idesc = make_idesc<KIND, 1>(RB);
        bool ok = true;
        int s = 0, u = 0;
        uint32_t s_phase = 0, u_phase = 0;
        for (int tile = tile0; ok && tile < tiles; tile += stride) {
            for (int i = u_first; i < u_last; ++i) {
                const int part = (i - u_first) % kPerStage;   // of its stage
                if (part == 0) ok = wait_all(full0 + 8 * s, s_phase, WHERE_FULL);
                ok = ok && wait_all(taken0 + 8 * u, u_phase ^ 1u, WHERE_ACC_EMPTY)
                     && wait_all(ready0 + 8 * u, u_phase, WHERE_FULL);
                if (!ok) break;
                tc_fence_after();
                const int steps = (p.K - i * kUnitK) / 16;   // left (K is a multiple of 32)
                const bool stage_ends = part == kPerStage - 1 || i + 1 == u_last;
                if (elect_one()) {
                    const uint64_t ad = smem_desc_sw128(blocks0 + u * (U * kNrBlockBytes));
                    const uint64_t xd = smem_desc_sw128(base + s * Shape::kStageBytes + kNrPackedBytes + part * (U * RB * 128));
                    const uint32_t d = tmem_base + u * kSet;
#pragma unroll
                    for (int k = 0; k < 4 * U; ++k) {
                        if (k >= steps) break;
                        umma<KIND, 1>(1u, d + k / (2 * GC) * RB, ad + (k / 4) * (kNrBlockBytes / 16) + 2 * (k % 4),
                                      xd + (k / 4) * (RB * 128 / 16) + 2 * (k % 4), idesc, k % (2 * GC) == 0 ? 0u : 1u);
                    }
                    umma_commit<1>(1u, used0 + 8 * u, 0);
                    umma_commit<1>(1u, sum0 + 8 * u, 0);
                    if (stage_ends) umma_commit<1>(1u, empty0 + 8 * s, 0);
                }
                __syncwarp();
                if (++u == NU) u = 0, u_phase ^= 1u;
                if (stage_ends && ++s == S) s = 0, s_phase ^= 1u;
            }
        }
        if (elect_one()) umma_commit<1>(1u, done, 0);
        __syncwarp();
        ctl.drain(done, 0, 10000000ull);
    } else if (warp < Shape::kExpandWarp0) {
        // ========================== scale and sum ==============================
        // This lane's feature, its scales a unit ahead; acc[r]: the sum of row
        // 32 * half + r.
        const int quarter = warp & 3, half = (warp - kNrScaleWarp0) >> 2;
        int u = 0;
        uint32_t u_phase = 0;
        bool ok = true;
        for (int tile = tile0; ok && tile < tiles; tile += stride) {
            const Tile t = tile_at(tile);
            const int f = t.n0 + quarter * 32 + lane;
            const uint16_t *sp = static_cast<const uint16_t *>(p.scales) + static_cast<long long>(t.row_b + min(f, p.N - 1)) * p.groups;
            uint32_t next[(kGroups + 1) / 2] = {};
            if (u_first < u_last) load_group_scales<kGroups, VEC>(sp, u_first * kGroups, p.groups, next);
#pragma unroll
            for (int r = 0; r < 32; ++r) acc[r] = 0.0f;
            for (int i = u_first; i < u_last; ++i) {
                uint32_t scale[(kGroups + 1) / 2];
#pragma unroll
                for (int j = 0; j < (kGroups + 1) / 2; ++j) scale[j] = next[j];
                load_group_scales<kGroups, VEC>(sp, (i + 1 < u_last ? i + 1 : i) * kGroups, p.groups, next);
                ok = wait_all(sum0 + 8 * u, u_phase, WHERE_ACC_FULL);
                if (!ok) break;
                tc_fence_after();
                const uint32_t from = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + u * kSet + 32 * half;
                const int groups = p.groups - i * kGroups;   // left
#pragma unroll
                for (int j = 0; j < kGroups; ++j) {
                    if (j >= groups) break;
                    const float c = widen<KIND>(scale[j / 2], j & 1);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(from + j * RB + 16 * h, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[16 * h + r] = fmaf(c, __uint_as_float(v[r]), acc[16 * h + r]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                mbar_arrive_if(one, taken0 + 8 * u);
                if (++u == NU) u = 0, u_phase ^= 1u;
            }
            if (ok && ctas == 1 && f < p.N)
#pragma unroll
                for (int r = 0; r < 32; ++r)
                    if (32 * half + r < t.rows.cnt) nib_store<KIND>(p, t.rows.r0 + 32 * half + r, f, acc[r]);
        }
    } else {
        // =============================== expand ================================
        // A thread has 32 weights of every block of a unit: feature f, half of its
        // 64.  Teams of 8 warps take units in turn, so that one's waits and fence
        // go with the other's arithmetic.
        const int thread = static_cast<int>(threadIdx.x) - 32 * Shape::kExpandWarp0;
        const int f = thread & 127, half = (thread >> 7) & 1, team = thread >> 8;
        const uint32_t given = p.zeros ? 1u : 0u;
        int before_u = 0, before_s = 0;   // units and stages of the tiles before this one
        bool ok = true;
        for (int tile = tile0; ok && tile < tiles; tile += stride) {
            const Tile t = tile_at(tile);
            const uint8_t *zp = p.zeros + static_cast<long long>(t.row_b + min(t.n0 + f, p.N - 1)) * p.groups;
            uint32_t next[(kGroups + 3) / 4];   // (a unit of this team ahead)
#pragma unroll
            for (int j = 0; j < (kGroups + 3) / 4; ++j) next[j] = 0x08080808u;
            if (u_first + team < u_last) load_group_zeros<kGroups, VEC>(given, zp, (u_first + team) * kGroups, p.groups, next);
            for (int i = u_first + team; i < u_last; i += kTeams) {
                uint32_t zero[U];   // of this thread's weights in each block
#pragma unroll
                for (int b = 0; b < U; ++b) {
                    if constexpr (GC == 1) zero[b] = zero_bits<KIND>(next[b / 2] >> (8 * half), 2 * (b & 1));
                    else zero[b] = zero_bits<KIND>(next[0], GC == 2 ? b : b / 2);
                }
                load_group_zeros<kGroups, VEC>(given, zp, (i + kTeams < u_last ? i + kTeams : i) * kGroups, p.groups, next);
                const int at = i - u_first, part = at % kPerStage;
                const uint32_t unit = before_u + at, stage = before_s + at / kPerStage, u = unit % NU, s = stage % S;
                ok = wait_all(full0 + 8 * s, (stage / S) & 1, WHERE_FULL)
                     && wait_all(used0 + 8 * u, ((unit / NU) & 1) ^ 1, WHERE_EMPTY);
                if (!ok) break;
                const uint32_t from = base + s * Shape::kStageBytes + f * 128;
                const uint32_t to = blocks0 + u * (U * kNrBlockBytes) + f * 128;
                uint4 w[U];
#pragma unroll
                for (int b = 0; b < U; ++b) w[b] = ld_shared_v4(from + (((2 * (part * U + b) + half) ^ (f & 7)) << 4));
#pragma unroll
                for (int b = 0; b < U; ++b) {
                    const uint32_t words[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t o[4];
                        expand_in_order<KIND>(words[j], zero[b], o);
                        st_shared_v4(to + b * kNrBlockBytes + (((4 * half + j) ^ (f & 7)) << 4), o[0], o[1], o[2], o[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                mbar_arrive_if(one, ready0 + 8 * u);
                if (kTeams >= kPerStage || part == kPerStage - 1 || i + 1 == u_last) mbar_arrive_if(one, empty0 + 8 * s);
            }
            before_u += u_last - u_first;
            before_s += last - first;
        }
    }
    __syncwarp();

    // ---- a cluster's sums ------------------------------------------------------
    if (ctas > 1) {
        // CTA j adds up rows j * part ..: [CTA][row][feature], where the stages were
        const int part = RB / ctas, shift = __ffs(part) - 1;   // (2 or 4 CTAs)
        const bool there = tile0 < tiles;
        const Tile t = there ? tile_at(tile0) : Tile{};
        __syncthreads();
        cluster_sync();   // (every CTA is through with its stages)
        if (there && warp >= kNrScaleWarp0 && warp < Shape::kExpandWarp0) {
            const int f = ((warp & 3) << 5) + lane, row0 = ((warp - kNrScaleWarp0) >> 2) * 32;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int r = row0 + i, to = r >> shift;
                st_cluster_f32(mapa(base + ((rank * part + (r & (part - 1))) * kNibWideFeatures + f) * 4, static_cast<uint32_t>(to)), acc[i]);
            }
        }
        cluster_sync();
        if (there)
            for (int i = static_cast<int>(threadIdx.x); i < part * kNibWideFeatures; i += Shape::kThreads) {
                const int r = i / kNibWideFeatures, n = i % kNibWideFeatures;
                float v = 0.0f;
                for (int c = 0; c < ctas; ++c) v += lds_f32(base + ((c * part + r) * kNibWideFeatures + n) * 4);
                if (rank * part + r < t.rows.cnt && t.n0 + n < p.N) nib_store<KIND>(p, t.rows.r0 + rank * part + r, t.n0 + n, v);
            }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<1>(tmem_base, NU * kSet);
    }
}

template <int KIND, int RB, int GC, bool VEC>
cudaError_t run_rows(const CUtensorMap &b, const CUtensorMap &x, const NibbleParams &p, NibPrepared *prepared,
                     cudaStream_t stream, bool overlap)
{
    constexpr int smem = NibRowsShape<RB>::kSmem;
    const auto kernel = nibble_rows_kernel<KIND, RB, GC, VEC>;
    const uint32_t bit = 1u << (12 + (RB == 32 ? 0 : 6) + 2 * (GC / 2) + VEC);   // (GC / 2: 0, 1, 2)
    if (!(prepared->kernels & bit)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        prepared->kernels |= bit;
    }
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    const unsigned tiles = static_cast<unsigned>(p.max_blocks) * ((p.N + kNibWideFeatures - 1) / kNibWideFeatures);
    cfg.gridDim = dim3(p.cluster > 1 || tiles < static_cast<unsigned>(p.ctas) ? tiles * p.cluster : static_cast<unsigned>(p.ctas), 1, 1);
    cfg.blockDim = dim3(NibRowsShape<RB>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (p.cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(p.cluster);
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (overlap) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kernel, b, x, p);
}

template <int KIND, int RB, int GC>
cudaError_t rows_by_alignment(const CUtensorMap &b, const CUtensorMap &x, const NibbleParams &p, NibPrepared *prepared,
                              cudaStream_t stream, bool overlap)
{
    constexpr int kGroups = 2 * NibRowsShape<RB>::kUnit / GC;
    if constexpr (kGroups > 1)
        if (p.groups % kGroups == 0) return run_rows<KIND, RB, GC, true>(b, x, p, prepared, stream, overlap);
    return run_rows<KIND, RB, GC, false>(b, x, p, prepared, stream, overlap);
}

template <int KIND, int RB>
cudaError_t rows_by_group(const CUtensorMap &b, const CUtensorMap &x, const NibbleParams &p, NibPrepared *prepared,
                          cudaStream_t stream, bool overlap)
{
    return p.group == 32 ? rows_by_alignment<KIND, RB, 1>(b, x, p, prepared, stream, overlap)
           : p.group == 64 ? rows_by_alignment<KIND, RB, 2>(b, x, p, prepared, stream, overlap)
                           : rows_by_alignment<KIND, RB, 4>(b, x, p, prepared, stream, overlap);
}

}  // namespace

// (one translation unit per kind: expert_launch.h names the two)
cudaError_t PTS_NIBBLE_ROWS_LAUNCH(const CUtensorMap &b, const CUtensorMap &x, const NibbleParams &p, NibPrepared *prepared,
                                   cudaStream_t stream, bool overlap)
{
    return p.block_rows == 32 ? rows_by_group<PTS_NIBBLE_KIND, 32>(b, x, p, prepared, stream, overlap)
                              : rows_by_group<PTS_NIBBLE_KIND, 64>(b, x, p, prepared, stream, overlap);
}

}  // namespace pts
