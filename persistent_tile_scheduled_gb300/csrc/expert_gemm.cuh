// The products of a layer of experts: rows sorted by expert, the row counts on
// the device, one launch for all experts.
//
//   EXPERT_FWD     out[r, f] = sum_k X[r, k] W_e[f, k]     rows r of expert e
//   EXPERT_DGRAD   out[r, f] = sum_c X[r, c] W_e[c, f]     (X = dC, f over K)
//   EXPERT_WGRAD   out_e[n, f] = sum_r X[r, n] W[r, f]     (X = dC, W = A, r over expert e's rows)
//
// In all three the accumulator holds D[f, row]: the features f, contiguous in
// the output, are the M side of the tensor-core instruction (128 per CTA) and
// the output rows are its N side.  The row count of an expert is arbitrary, and
// N may be any multiple of 16 (32 for a CTA pair) up to 256 while M is fixed,
// so a tile wastes at most 15 (31) rows instead of up to 255; an expert's rows
// are cut into tiles of equal size.  The epilogue reads the accumulator in
// fragment layout and transposes it on its way to shared memory
// (stmatrix .trans), so the rows leave contiguous.
//
// Operand layouts, read by TMA with the 128-byte swizzle from the arrays as
// the user holds them, without a transposed copy:
//   contraction contiguous (K-major): FWD's X and W, DGRAD's X.
//   contraction strided (MN-major): DGRAD's W, WGRAD's X and W.  A box of
//     64 features x a ring stage's contraction rows (128 for a pair) is one
//     block; blocks of 64 features follow one another (leading byte offset),
//     groups of 8 contraction rows are 1024 bytes apart (stride byte offset).
//     One box per 64 rows instead, twice the TMA instructions, took 371 us for
//     16384 rows over 8 experts of 4096 x 4096 where this takes 325.
// An operand row that belongs to another expert (a box that runs past the
// expert's last row) only feeds accumulator columns that are not stored.  In
// WGRAD the rows are the contraction, so there the last 16-row step is cleared
// in shared memory behind the expert's last row, in both operands (a NaN or
// infinity there times zero would not be zero), before the MMA reads it.
//
// What bounds it (GB300, bf16).  Many rows: the tensor pipe, 85 % busy over 16384
// rows spread unevenly over 8 experts of 8192 x 4096 (580 us alone; back to back
// under the power cap 660 to 690 us, one dense gemm_run of that size 647).  An expert whose rows do not fill its tiles costs the weights' loads of a
// full one: a pair's stage is 64 KB per SM for 1024 cycles of MMA, the most an SM
// takes in, so a tile of 200 rows runs hardly faster than one of 256 (8192 rows
// over 16 experts: 232 us uneven, 213 even).  Few rows: the weights' bytes, 6.2
// TB/s, with tiles of 64 rows and 8 stages (45.1 us for 40 rows over 8 experts of
// 4096^2 when each MMA was issued under a predicate, 43.3 by one elected lane).  The weights' gradient loses about
// 0.5 us per tile to the cleared step where rows are no multiple of 16 (2047 and
// 2049 per expert 325 us, 2048 312).
// Tiles for less than half the SMs (one token): 2, 4 or 8 CTAs share a tile's
// contraction and add up through distributed shared memory, each its part of the
// rows, in order (one row of 4096^2 11.3 us instead of 18.6).
//
// Warp roles as in gemm_kernel.cuh: producer, MMA, 4 epilogue warps, scheduler
// (a static stride over the tiles of all experts, which it counts from the
// offsets as it walks them), and in WGRAD a warp that clears.  Waits are
// bounded in the same way.
#pragma once
#include "expert_launch.h"
#include "gemm_kernel.cuh"

namespace pts {

// One output tile, decoded by the scheduler warp.
struct ExpertItem {
    int e, f0, row0, row_end;   // expert, first feature, first output row (WGRAD: within the expert), its rows' end
    int n_len;                  // accumulator columns (a multiple of 16 * CG)
    int nkb;                    // k-blocks
    int c0, c_rows;             // WGRAD: first contraction row, contraction rows
};

// Shared-memory descriptor of an MN-major operand: 64-feature blocks `rows`
// contraction rows of 128 bytes apart, groups of 8 contraction rows 1024 bytes
// apart, version 1, 128-byte swizzle.
template <int ROWS>
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t addr)
{
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(ROWS * 128 / 16) << 16) | (64ull << 32)
           | (1ull << 46) | (2ull << 61);
}

template <int KIND, int MODE, int CG, int BN>
__global__ void __launch_bounds__(expert_threads(MODE), 1)
    expert_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                  const __grid_constant__ CUtensorMap tmXs, const __grid_constant__ CUtensorMap tmO,
                  const ExpertParams p)
{
    // tmW: boxes of 128 features x one k-block (MN-major: 64 features x a stage); tmX: boxes
    // of BN / CG rows x one k-block, tmXs: of 16 rows (MN-major: both as tmW);
    // tmO: the store box, 32 features x 64 rows
    constexpr bool kWmn = MODE != EXPERT_FWD;     // the operand's features are contiguous, the contraction is not
    constexpr bool kXmn = MODE == EXPERT_WGRAD;
    constexpr int KBS = kb_per_stage(CG);
    constexpr int SA = KBS * kRowsPerCta * kKBlockBytes;
    constexpr int SB = KBS * (BN / CG) * kKBlockBytes;
    constexpr int KELEMS = (KIND == 2) ? kKBlockBytes : kKBlockBytes / 2;
    constexpr int kXRows = BN / CG;               // this CTA's share of a tile's accumulator columns
    constexpr int kGran = 16 * CG;
    constexpr uint32_t kBlock = KBS * 64 * 128;   // an MN-major block: a stage's contraction rows of 128 bytes
    constexpr uint32_t kAccCols = 2 * BN;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const int S = p.stages;
    const uint32_t sA = base;
    const uint32_t sB = sA + S * SA;
    const uint32_t sEpi = sB + S * SB;
    const uint32_t bar0 = sEpi + epi_bytes();
    const uint32_t full0 = bar0;                             // + 8*s
    const uint32_t empty0 = bar0 + 8 * kMaxStages;           // + 8*s
    const uint32_t fix0 = bar0 + 16 * kMaxStages;            // + 8*s (WGRAD)
    const uint32_t acc_full0 = bar0 + 24 * kMaxStages;       // + 8*b
    const uint32_t acc_empty0 = acc_full0 + 16;              // + 8*b
    const uint32_t ring_full0 = acc_empty0 + 16;             // + 8*r
    const uint32_t ring_empty0 = ring_full0 + 8 * kRing;     // + 8*r
    const uint32_t ring0 = (ring_empty0 + 8 * kRing + 15) & ~15u;   // + 4*kRingWords*r
    const uint32_t tmem_slot = ring0 + 4 * kRingWords * kRing;
    const uint32_t abort_flag = tmem_slot + 4;

    const uint32_t warp = threadIdx.x >> 5;
    const uint32_t lane = lane_id();
    const uint32_t rank = (CG == 2) ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    // few tiles: `split` CTAs share one's contraction, and have no other
    constexpr bool kSplit = MODE == EXPERT_FWD && CG == 1 && BN == kExpertTileNFew;
    const int split = kSplit ? p.split : 1;
    const int share = kSplit && split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cluster_id = static_cast<int>(blockIdx.x) / (CG * split);
    const int num_clusters = static_cast<int>(gridDim.x) / (CG * split);

    WaitCtl ctl;
    ctl.abort_addr = abort_flag;
    ctl.peer_abort = (CG == 2) ? mapa(abort_flag, rank ^ 1u) : 0u;
    ctl.timeout_ns = p.timeout_ns;
    ctl.status = p.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            // (of a pair in WGRAD: both CTAs' clearing warps, or the leader's producer twice)
            mbar_init(full0 + 8 * s, MODE == EXPERT_WGRAD ? CG : 1);
            mbar_init(empty0 + 8 * s, 1);
            if (MODE == EXPERT_WGRAD) mbar_init(fix0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full0 + 8 * b, 1);
            mbar_init(acc_empty0 + 8 * b, kEpiWarps * CG);
        }
        // readers of the ring: every CTA's producer, epilogue (and clearing) warps, the leader's MMA warp
        constexpr uint32_t readers = 1 + CG * (1 + kEpiWarps + (MODE == EXPERT_WGRAD ? 1 : 0));
        for (int r = 0; r < kRing; ++r) {
            mbar_init(ring_full0 + 8 * r, 1);
            mbar_init(ring_empty0 + 8 * r, readers);
        }
        st_shared_u32(abort_flag, 0u);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
        prefetch_tmap(&tmXs);
        prefetch_tmap(&tmO);
    }
    if (warp == 1) {
        tmem_alloc<CG>(tmem_slot, kAccCols);
        tmem_relinquish<CG>();
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = ld_shared_u32(tmem_slot);
    const uint32_t one = lane == 0 ? 1u : 0u;

    pdl_launch_dependents();
    pdl_wait();   // the offsets and operands may be the previous grid's outputs

    // ---- work-item broadcast ring (as in gemm_kernel.cuh) ---------------------
    auto publish = [&](int i, bool valid, const ExpertItem &t) -> bool {
        const int slot = i % kRing;
        if (i >= kRing && !ctl.wait_all(ring_empty0 + 8 * slot, ((i / kRing) & 1) ^ 1, WHERE_RING_EMPTY))
            return false;
        if (lane == 0) {
            const uint32_t a = ring0 + 4 * kRingWords * slot;
            const uint32_t v[12] = {valid ? 1u : 0u,
                                    static_cast<uint32_t>(t.e),
                                    static_cast<uint32_t>(t.f0),
                                    static_cast<uint32_t>(t.row0),
                                    static_cast<uint32_t>(t.row_end),
                                    static_cast<uint32_t>(t.n_len),
                                    static_cast<uint32_t>(t.nkb),
                                    static_cast<uint32_t>(t.c0),
                                    static_cast<uint32_t>(t.c_rows),
                                    0u,
                                    0u,
                                    0u};
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                st_shared_v4(a + 16 * q, v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                if constexpr (CG == 2)
                    st_cluster_v4(mapa(a + 16 * q, 1u), v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            }
            if constexpr (CG == 2) mbar_arrive_cluster(mapa(ring_full0 + 8 * slot, 1u));
            mbar_arrive(ring_full0 + 8 * slot);
        }
        __syncwarp();
        return true;
    };
    // Called by a whole converged warp.  1: an item, 0: no more, -1: stopped.
    auto ring_read = [&](int i, ExpertItem &t) -> int {
        const int slot = i % kRing;
        if (!ctl.wait_all(ring_full0 + 8 * slot, (i / kRing) & 1, WHERE_RING_FULL)) return -1;
        const uint32_t a = ring0 + 4 * kRingWords * slot;
        const uint4 v0 = ld_shared_v4(a), v1 = ld_shared_v4(a + 16), v2 = ld_shared_v4(a + 32);
        t.e = static_cast<int>(v0.y);
        t.f0 = static_cast<int>(v0.z);
        t.row0 = static_cast<int>(v0.w);
        t.row_end = static_cast<int>(v1.x);
        t.n_len = static_cast<int>(v1.y);
        t.nkb = static_cast<int>(v1.z);
        t.c0 = static_cast<int>(v1.w);
        t.c_rows = static_cast<int>(v2.x);
        __syncwarp();   // every lane has read the slot before lane 0 hands it back
        if (CG == 2 && !leader)
            mbar_arrive_cluster_if(one, mapa(ring_empty0 + 8 * slot, 0u));
        else
            mbar_arrive_if(one, ring_empty0 + 8 * slot);
        return v0.x != 0 ? 1 : 0;
    };

    if (warp == 0) {
        // =============================== producer ==============================
        int stage = 0;
        uint32_t phase = 0;
        long long issued = 0;
        bool ok = true;
        for (int i = 0;; ++i) {
            ExpertItem t;
            if (ring_read(i, t) <= 0) break;
            const int xr = t.n_len / CG;   // this CTA's accumulator columns
            const int wf = t.f0 + static_cast<int>(rank) * kRowsPerCta;
            const int xrow = t.row0 + static_cast<int>(rank) * xr;
            // K-major X: one large box when it holds mostly wanted rows, else boxes of 16
            const bool big = 2 * xr > kXRows;
            const int xloads = kXmn ? (xr + 63) / 64 : (big ? 1 : xr / 16);
            const uint32_t xbox = kXmn ? kBlock : static_cast<uint32_t>((big ? kXRows : 16) * kKBlockBytes);
            const CUtensorMap *mx = (kXmn || big) ? &tmX : &tmXs;
            for (int kb = 0; kb < t.nkb; kb += KBS) {
                if (!ctl.wait_all(empty0 + 8 * stage, phase ^ 1u, WHERE_EMPTY)) {
                    ok = false;
                    break;
                }
                const int nk = t.nkb - kb < KBS ? t.nkb - kb : KBS;
                // (an MN-major box always spans the stage; rows behind the contraction are not read)
                const uint32_t tx = (kWmn ? SA : static_cast<uint32_t>(nk) * (SA / KBS))
                                    + static_cast<uint32_t>(kXmn ? xloads : nk * xloads) * xbox;
                // a stage that ends inside a 16-row step first goes to the clearing warp of this CTA
                const bool fix = kXmn && kb + KBS >= t.nkb && (t.c_rows & 15) != 0;
                const uint32_t fb = (fix ? fix0 : full0) + 8 * stage;
                const bool pair = CG == 2 && !fix;
                const uint32_t fbc = pair ? mapa(fb, 0u) : fb;
                // (test hook: more bytes than come, so that the bounded wait on this stage runs out)
                const uint32_t withheld = issued == p.fault_load ? 16u : 0u;
                // a pair's leader announces both CTAs' bytes (each announcing its own, the
                // peer through a remote arrival, took 862 us for 16384 rows of 8192 x 4096
                // where this takes 607); a stage that is cleared first is announced by
                // each CTA to itself
                if (elect_one()) {
                    if (!pair || leader) mbar_arrive_expect_tx_if(1u, fb, (pair ? CG * tx : tx) + withheld);
                    if (MODE == EXPERT_WGRAD && pair && leader) mbar_arrive_if(1u, fb);
                    auto load = [&](uint32_t dst, const CUtensorMap *m, int x, int y, int z) {
                        if (pair)
                            tma_load_3d_pair(1u, dst, m, fbc, x, y, z);
                        else
                            tma_load_3d(1u, dst, m, fbc, x, y, z);
                    };
                    const uint32_t da = sA + stage * SA, db = sB + stage * SB;
                    const int c = (kSplit ? t.c0 + kb : kb) * KELEMS;
                    if constexpr (kWmn) {
#pragma unroll
                        for (int b = 0; b < kRowsPerCta / 64; ++b)
                            load(da + b * kBlock, &tmW, wf + 64 * b, t.c0 + c, MODE == EXPERT_DGRAD ? t.e : 0);
                    } else {
                        for (int j = 0; j < nk; ++j) load(da + j * (SA / KBS), &tmW, c + j * KELEMS, wf, t.e);
                    }
                    if constexpr (kXmn) {
                        for (int b = 0; b < xloads; ++b) load(db + b * kBlock, mx, xrow + 64 * b, t.c0 + c, 0);
                    } else {
                        for (int j = 0; j < nk; ++j)
                            for (int b = 0; b < xloads; ++b)
                                load(db + j * (SB / KBS) + b * xbox, mx, c + j * KELEMS, xrow + 16 * b, 0);
                    }
                }
                __syncwarp();
                ++issued;
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
        }
        // Every load that was issued lands before the CTA can exit (bounded), also
        // where another warp gave up on a stage after the last load was issued.  A
        // leader's barriers count both CTAs' bytes; a load of its peer's that it did
        // not announce is given time at the teardown.
        if (CG == 1 || leader) {
            const long long n = issued < S ? issued : S;
            for (long long j = 0; j < n; ++j) {
                const long long g = issued - 1 - j;
                ctl.drain(full0 + 8 * static_cast<int>(g % S), static_cast<uint32_t>((g / S) & 1), 10000000ull);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================================ MMA ==================================
        if (leader) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            int last_stage = -1;
            uint32_t last_phase = 0;
            for (int i = 0;; ++i) {
                ExpertItem t;
                if (ring_read(i, t) <= 0) break;
                if (!ctl.wait_all(acc_empty0 + 8 * acc, acc_phase ^ 1u, WHERE_ACC_EMPTY)) break;
                tc_fence_after();
                // operand majorness: bit 15 for the M side (W), bit 16 for the N side (X)
                const uint32_t idesc = make_idesc<KIND, CG>(static_cast<uint32_t>(t.n_len)) | (kWmn ? 1u << 15 : 0u)
                                       | (kXmn ? 1u << 16 : 0u);
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
                bool ok = true;
                for (int kb = 0; kb < t.nkb; kb += KBS) {
                    if (!ctl.wait_all(full0 + 8 * stage, phase, WHERE_FULL)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int nk = t.nkb - kb < KBS ? t.nkb - kb : KBS;
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < KBS; ++j) {
                            if (j >= nk) break;
                            // (the next k-block of an MN-major stage: 64 rows on in every block)
                            const uint32_t aa = sA + stage * SA + j * (kWmn ? 64 * 128 : SA / KBS);
                            const uint32_t ab = sB + stage * SB + j * (kXmn ? 64 * 128 : SB / KBS);
                            const uint64_t ad = kWmn ? smem_desc_mn_sw128<64 * KBS>(aa) : smem_desc_sw128(aa);
                            const uint64_t bd = kXmn ? smem_desc_mn_sw128<64 * KBS>(ab) : smem_desc_sw128(ab);
                            // an instruction takes 32 bytes of a K-major row, or 16 contraction rows of 128 bytes
                            constexpr uint64_t da = kWmn ? 128 : 2, db = kXmn ? 128 : 2;
                            int steps = 4;
                            if constexpr (kXmn) {
                                const int left = t.c_rows - (kb + j) * KELEMS;
                                steps = left >= KELEMS ? 4 : (left + 15) / 16;
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k < steps) umma<KIND, CG>(1u, d, ad + da * k, bd + db * k, idesc,
                                               (kb + j != 0 || k != 0) ? 1u : 0u);
                        }
                        umma_commit<CG>(1u, empty0 + 8 * stage, 0x3);
                    }
                    __syncwarp();
                    last_stage = stage;
                    last_phase = phase;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if (elect_one()) umma_commit<CG>(1u, acc_full0 + 8 * acc, 0x3);
                __syncwarp();
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            if (last_stage >= 0) ctl.drain(empty0 + 8 * last_stage, last_phase, 10000000ull);
        }
        __syncwarp();
    } else if (warp < 2 + kEpiWarps) {
        // ============================== epilogue ===============================
        // A warp owns 32 features (TMEM lanes) of the tile.  Per chunk of 64
        // output rows it packs the fragments, stores them transposed into a
        // staging buffer of 64 rows x 64 bytes (64-byte swizzle) and hands
        // that to one TMA store; a chunk that ends inside an expert's last
        // rows is copied out 16 bytes at a time instead.
        const uint32_t q = warp & 3u;
        const uint32_t stage_base = sEpi + (warp - 2) * (kEpiBufsPerWarp * kEpiBufBytes);
        // stmatrix: this lane's address is that of row (lane % 8) of the 8 x 8
        // matrix of features 8 (lane / 8) .. + 7
        const uint32_t st_row = lane & 7u, st_chunk = lane >> 3;
        int acc = 0;
        uint32_t acc_phase = 0;
        uint32_t nstore = 0;
        for (int i = 0;; ++i) {
            ExpertItem t;
            if (ring_read(i, t) <= 0) break;
            const bool empty_sum = t.nkb == 0;
            if (!ctl.wait_all(acc_full0 + 8 * acc, acc_phase, WHERE_ACC_FULL)) break;
            tc_fence_after();
            if (kSplit && split > 1) break;   // (the only tile; added up below)
            const uint32_t tbase = tmem_base + ((q * 32u) << 16) + static_cast<uint32_t>(acc * BN);
            const int chunks = (t.n_len + 63) / 64;
            const int f = t.f0 + static_cast<int>(rank) * kRowsPerCta + static_cast<int>(q) * 32;
            for (int c = 0; c < chunks; ++c) {
                uint32_t lo[32], hi[32];
                tmem_ld_16x256b_x8(tbase + c * 64, lo);
                tmem_ld_16x256b_x8(tbase + (16u << 16) + c * 64, hi);
                tmem_wait_ld();
                if (empty_sum) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) lo[j] = hi[j] = 0u;
                }
                if (c + 1 == chunks) {
                    tc_fence_before();
                    __syncwarp();
                    if (CG == 2 && !leader)
                        mbar_arrive_cluster_if(one, mapa(acc_empty0 + 8 * acc, 0u));
                    else
                        mbar_arrive_if(one, acc_empty0 + 8 * acc);
                }
                const uint32_t buf = stage_base + (nstore & 1u) * kEpiBufBytes;
                bulk_wait_read<1>();   // the store that used this buffer has read it
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t row = 8 * j + st_row;
                    stmatrix_x4_trans(buf + row * 64 + ((st_chunk ^ ((row >> 1) & 3u)) << 4),
                                      pack2<KIND>(lo[4 * j], lo[4 * j + 1], p.out_scale),
                                      pack2<KIND>(lo[4 * j + 2], lo[4 * j + 3], p.out_scale),
                                      pack2<KIND>(hi[4 * j], hi[4 * j + 1], p.out_scale),
                                      pack2<KIND>(hi[4 * j + 2], hi[4 * j + 3], p.out_scale));
                }
                const int row0 = t.row0 + c * 64;
                if (MODE == EXPERT_WGRAD || row0 + 64 <= t.row_end) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    tma_store_3d_if((f < p.features && row0 < t.row_end) ? one : 0u, &tmO, buf, f, row0,
                                    MODE == EXPERT_WGRAD ? t.e : 0);
                } else {
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t r = 8 * j + (lane >> 2), ch = lane & 3u;
                        const uint4 v = ld_shared_v4(buf + r * 64 + ((ch ^ ((r >> 1) & 3u)) << 4));
                        const long long row = row0 + static_cast<long long>(r);
                        if (row < t.row_end && f + 8 * static_cast<int>(ch) < p.features)
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + row * p.features + f + 8 * ch) = v;
                    }
                }
                bulk_commit();
                ++nstore;
            }
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        bulk_wait_read<0>();
        __syncwarp();
    } else if (warp == kSchedWarp) {
        // ============================== scheduler ==============================
        // Tile w of all experts' tiles in order, w = cluster, cluster + grid, ...
        if (leader) {
            const int tiles_f = (p.features + kRowsPerCta * CG - 1) / (kRowsPerCta * CG);
            bool ok = true;
            int i = 0;
            auto offset = [&](int e) -> int {   // clamped, so that no offsets lead outside the arrays
                const int v = ld_global(p.offsets + e);
                return v < 0 ? 0 : (v > p.rows ? p.rows : v);
            };
            if constexpr (MODE == EXPERT_WGRAD) {
                const int tiles_n = (p.out_rows + BN - 1) / BN;
                const long long per = static_cast<long long>(tiles_f) * tiles_n;
                const long long tiles = per * p.experts;
                for (long long w = cluster_id; ok && w < tiles; w += num_clusters) {
                    ExpertItem t;
                    t.e = static_cast<int>(w / per);
                    int tn, tf;
                    tile_of(static_cast<int>(w - t.e * per), tiles_n, tiles_f, p.group_m, tn, tf);
                    t.f0 = tf * (kRowsPerCta * CG);
                    t.row0 = tn * BN;
                    t.row_end = p.out_rows;
                    const int left = p.out_rows - t.row0;
                    t.n_len = left >= BN ? BN : (left + kGran - 1) / kGran * kGran;
                    const int lo = offset(t.e), hi = offset(t.e + 1);
                    t.c0 = lo;
                    t.c_rows = hi > lo ? hi - lo : 0;
                    t.nkb = (t.c_rows + KELEMS - 1) / KELEMS;
                    ok = publish(i, true, t);
                    ++i;
                }
            } else {
                const int nkb = (p.contraction + KELEMS - 1) / KELEMS;
                // 32 experts at a time: lane l holds expert e0 + l, its rows and
                // the tiles of the experts before it
                long long w = cluster_id, before = 0;
                for (int e0 = 0; ok && e0 < p.experts; e0 += 32) {
                    const int e = e0 + static_cast<int>(lane);
                    int lo = 0, cnt = 0;
                    if (e < p.experts) {
                        lo = offset(e);
                        cnt = offset(e + 1) - lo;
                        cnt = cnt > 0 ? cnt : 0;
                    }
                    const int tn = (cnt + BN - 1) / BN;
                    long long incl = static_cast<long long>(tn) * tiles_f;
#pragma unroll
                    for (int s = 1; s < 32; s <<= 1) {
                        const long long o = __shfl_up_sync(0xffffffffu, incl, s);
                        if (static_cast<int>(lane) >= s) incl += o;
                    }
                    const long long total = __shfl_sync(0xffffffffu, incl, 31);
                    for (; ok && w < before + total; w += num_clusters) {
                        const int src = __ffs(__ballot_sync(0xffffffffu, before + incl > w)) - 1;
                        const int elo = __shfl_sync(0xffffffffu, lo, src);
                        const int ecnt = __shfl_sync(0xffffffffu, cnt, src);
                        const int etn = __shfl_sync(0xffffffffu, tn, src);
                        const long long eincl = __shfl_sync(0xffffffffu, incl, src);
                        const int local = static_cast<int>(w - before - (eincl - static_cast<long long>(etn) * tiles_f));
                        int it, itf;
                        tile_of(local, etn, tiles_f, p.group_m, it, itf);
                        // equal tiles: ecnt rows in etn tiles, each a multiple of the MMA's granularity
                        const int size = ((ecnt - 1) / etn + kGran) / kGran * kGran;
                        ExpertItem t;
                        t.e = e0 + src;
                        t.f0 = itf * (kRowsPerCta * CG);
                        t.row0 = elo + it * size;
                        t.row_end = elo + ((it + 1) * size < ecnt ? (it + 1) * size : ecnt);
                        const int rows = t.row_end - t.row0;
                        t.n_len = (rows + kGran - 1) / kGran * kGran;
                        t.c0 = kSplit ? nkb * share / split : 0;
                        t.nkb = (kSplit ? nkb * (share + 1) / split : nkb) - t.c0;
                        t.c_rows = 0;
                        if (rows > 0) {   // (rounding the tile size up may leave the last tile nothing)
                            ok = publish(i, true, t);
                            ++i;
                        }
                        if (kSplit && split > 1) w = 1ll << 62;   // (the one tile; offsets that go back and forth claim more)
                    }
                    before += total;
                }
            }
            if (ok) publish(i, false, ExpertItem{});
        }
        __syncwarp();
    } else if (MODE == EXPERT_WGRAD) {
        // =============================== clearing ==============================
        // The last stage of an item whose rows end inside a 16-row step: wait
        // for this CTA's loads of it, clear the rows behind the end in both
        // operands, and hand the stage to the MMA warp.
        int stage = 0;
        uint32_t phases = 0;   // bit s: the parity of fix barrier s that comes next
        for (int i = 0;; ++i) {
            ExpertItem t;
            if (ring_read(i, t) <= 0) break;
            const int stages_used = (t.nkb + KBS - 1) / KBS;
            if ((t.c_rows & 15) == 0) {
                stage = (stage + stages_used) % S;
                continue;
            }
            const int s = (stage + stages_used - 1) % S;
            if (!ctl.wait_all(fix0 + 8 * s, (phases >> s) & 1u, WHERE_FULL)) break;
            // rows of the stage that are the expert's, up to the end of their last step
            const uint32_t rem = static_cast<uint32_t>(t.c_rows - (stages_used - 1) * KBS * KELEMS);
            const uint32_t end = (rem + 15u) & ~15u;
            const int xblocks = (t.n_len / CG + 63) / 64;
            for (int b = 0; b < kRowsPerCta / 64 + xblocks; ++b) {
                const uint32_t blk = b < kRowsPerCta / 64 ? sA + s * SA + b * kBlock
                                                          : sB + s * SB + (b - kRowsPerCta / 64) * kBlock;
                // rows of 128 bytes: 8 lanes to a row, 4 rows at a time
                for (uint32_t r = rem + (lane >> 3); r < end; r += 4)
                    st_shared_v4(blk + r * 128 + (lane & 7u) * 16, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (CG == 2 && !leader) mbar_arrive_cluster_if(one, mapa(full0 + 8 * s, 0u));
            else mbar_arrive_if(one, full0 + 8 * s);
            phases ^= 1u << s;
            stage = (stage + stages_used) % S;
        }
        __syncwarp();
    }

    // ---- a tile whose contraction is shared ------------------------------------
    if (kSplit && split > 1) {
        // CTA j of the cluster adds up rows j * part ..: [CTA][row][feature], where the
        // stages were; the tile is the ring's first item
        const int part = BN / split, shift = __ffs(part) - 1;   // (split is 2, 4 or 8)
        __syncthreads();
        cluster_sync();   // (every CTA is through with its stages)
        const bool published = mbar_try_wait(ring_full0, 0);
        const uint4 v0 = ld_shared_v4(ring0), v1 = ld_shared_v4(ring0 + 16);
        const bool there = published && v0.x != 0;
        if (there && warp >= 2 && warp < 2 + kEpiWarps) {
            const uint32_t q = warp & 3u;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem_base + ((q * 32u) << 16) + 32 * c, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int row = 32 * c + i, to = row >> shift;
                    st_cluster_u32(mapa(base + ((share * part + (row & (part - 1))) * kRowsPerCta + q * 32 + lane) * 4,
                                        static_cast<uint32_t>(to)), v[i]);
                }
            }
        }
        cluster_sync();
        if (there)
            for (int i = static_cast<int>(threadIdx.x); i < part * kRowsPerCta / 2; i += static_cast<int>(blockDim.x)) {
                const int row = i / (kRowsPerCta / 2), n = 2 * (i % (kRowsPerCta / 2));
                float lo = 0.0f, hi = 0.0f;
                for (int c = 0; c < split; ++c) {
                    const uint32_t from = base + ((c * part + row) * kRowsPerCta + n) * 4;
                    lo += __uint_as_float(ld_shared_u32(from));
                    hi += __uint_as_float(ld_shared_u32(from + 4));
                }
                const long long out_row = static_cast<long long>(v0.w) + share * part + row;
                const int f = static_cast<int>(v0.z) + n;
                if (out_row < static_cast<int>(v1.x) && f < p.features)
                    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + out_row * p.features + f) =
                        pack2<KIND>(__float_as_uint(lo), __float_as_uint(hi), p.out_scale);
            }
    }

    // ---- teardown ------------------------------------------------------------
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) {
        // stopped early: a load of this CTA that the leader did not announce
        // completes on a phase that cannot finish; let 1 ms pass, far longer than
        // any load takes
        if (!leader && warp == 0 && ld_shared_u32(abort_flag)) {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 1000000ull) {
            }
            __syncwarp();
        }
        cluster_sync();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<CG>(tmem_base, kAccCols);
    }
}

template <int KIND, int MODE, int CG, int BN>
struct ExpertInst {
    static void config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, int grid, int cluster, int smem,
                       cudaStream_t stream, bool overlap)
    {
        cfg = cudaLaunchConfig_t{};
        cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
        cfg.blockDim = dim3(expert_threads(MODE), 1, 1);
        cfg.dynamicSmemBytes = static_cast<size_t>(smem);
        cfg.stream = stream;
        cfg.attrs = attr;
        int n = 0;
        if (overlap) {
            attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[n].val.programmaticStreamSerializationAllowed = 1;
            ++n;
        }
        if (cluster > 1) {
            attr[n].id = cudaLaunchAttributeClusterDimension;
            attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
            attr[n].val.clusterDim.y = 1;
            attr[n].val.clusterDim.z = 1;
            ++n;
        }
        cfg.numAttrs = static_cast<unsigned>(n);
    }

    // Raise the shared-memory limit and report how many clusters the device
    // holds (single CTAs: one per SM, see Inst::max_active_clusters on why the
    // occupancy query is not asked there).
    static cudaError_t prepare(int smem, int sms, int *clusters)
    {
        cudaError_t e = cudaFuncSetAttribute(expert_kernel<KIND, MODE, CG, BN>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        *clusters = sms;
        if (CG == 1) return cudaSuccess;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        config(cfg, attr, 2, CG, smem, nullptr, false);
        return cudaOccupancyMaxActiveClusters(clusters, expert_kernel<KIND, MODE, CG, BN>, &cfg);
    }

    static cudaError_t launch(const CUtensorMap &w, const CUtensorMap &x, const CUtensorMap &xs, const CUtensorMap &o,
                              const ExpertParams &p, int grid, int smem, cudaStream_t stream, bool overlap)
    {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        config(cfg, attr, grid, CG * p.split, smem, stream, overlap);
        return cudaLaunchKernelEx(&cfg, expert_kernel<KIND, MODE, CG, BN>, w, x, xs, o, p);
    }

    static ExpertOps ops() { return ExpertOps{&prepare, &launch}; }
};

}  // namespace pts
