// Parameters and launch entry points of the expert layer's kernels (host and
// device).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gemm_params.h"

namespace pts {

enum : int { EXPERT_FWD = 0, EXPERT_DGRAD = 1, EXPERT_WGRAD = 2 };

// ---- the experts' products (expert_gemm.cuh) --------------------------------

// The epilogue: none; bias, activation and residual (EPI_LINEAR); the same with a
// gate's features and those it multiplies side by side (EPI_GATED).
enum : int { EPI_NONE = 0, EPI_LINEAR = 1, EPI_GATED = 2 };

struct ExpertParams {
    int32_t rows;          // rows of X (the offsets are clamped to it)
    int32_t experts;
    int32_t features;      // contiguous extent of the output (M side)
    int32_t contraction;   // K (FWD), N (DGRAD); unused in WGRAD, where it is an expert's rows
    int32_t out_rows;      // WGRAD: output rows per expert
    int32_t stages;
    int32_t split;                    // CTAs that share a tile's contraction
    int32_t group_m;       // row tiles per group of the tile order
    float out_scale;
    const int32_t *offsets;   // experts + 1, device
    void *out;
    int32_t fault_load;       // test hook: the stage load of a producer that announces too many bytes (-1: none)
    uint64_t timeout_ns;
    int32_t *status;
    // of an epilogue (offsets may then be null: one matrix has all rows)
    int32_t act;              // gemm_act_t
    const void *bias, *residual;   // experts x N', rows x N, or null
    void *z;                  // rows x N', or null
    int32_t tile0, tiles_f;   // first tile of features and tiles of this launch
    int32_t chain;            // 1: another launch takes the other tiles, 2: this is it
};

// Tensor maps of a product, and of one with an epilogue.
struct ExpertMaps {
    CUtensorMap w, x, xs, o;
};
struct LinearMaps : ExpertMaps {
    CUtensorMap r, z;   // residual, Z: boxes as o's
};

// Epilogue warps.  One with activations computes some 25 instructions per element, which
// 4 warps, one to a scheduler, take too long for (bf16 4096^2, K = 512, gated silu, chunks
// of 16 rows: 42 us with 4, 37 with 8).
__host__ __device__ constexpr int expert_epi_warps(int epi) { return epi == EPI_NONE ? kEpiWarps : 2 * kEpiWarps; }

// producer, MMA, epilogue warps, scheduler; WGRAD has a clearing warp too
__host__ __device__ constexpr int expert_threads(int mode, int epi = EPI_NONE)
{
    return 96 + 32 * expert_epi_warps(epi) + (mode == EXPERT_WGRAD ? 32 : 0);
}
static_assert(expert_threads(EXPERT_FWD) == kThreads, "");

// Barriers that only some kernels use: WGRAD's cleared stages, an epilogue's residual.
__host__ __device__ constexpr int expert_fix_barriers(int epi) { return epi == EPI_NONE ? kMaxStages : expert_epi_warps(epi); }

// Dynamic shared memory for `stages` stages of a tile of bn rows (plus 1 KB
// for aligning the base to the swizzle period).
__host__ __device__ constexpr int expert_smem_bytes(int cg, int bn, int stages, int epi = EPI_NONE)
{
    return 1024 + stages * kb_per_stage(cg) * (kRowsPerCta + bn / cg) * kKBlockBytes + epi_bytes()
           + 8 * (2 * kMaxStages + expert_fix_barriers(epi) + 4 + 2 * kRing) + 16   // mbarriers, alignment
           + 4 * kRingWords * kRing + 16;                // ring payload, TMEM base, abort flag
}

constexpr int kExpertTileN = 256;       // rows of a tile
constexpr int kExpertTileNFew = 64;     // rows of a tile when the experts have few:
constexpr int64_t kExpertFewRows = 32;  // at most so many on average

struct ExpertOps {
    cudaError_t (*prepare)(int smem, int sms, int *clusters);
    cudaError_t (*launch)(const LinearMaps &maps, const ExpertParams &p, int grid, int smem, cudaStream_t stream, bool overlap);
    cudaError_t (*fit)(int cluster, int smem, int *clusters);
};

// kind: 0 fp16, 1 bf16, 2 e4m3 (forward only); bn: kExpertTileN, or
// kExpertTileNFew (forward, single CTAs)
ExpertOps expert_ops_fwd(int kind, int cg, int bn);
ExpertOps expert_ops_dgrad(int kind, int cg);
ExpertOps expert_ops_wgrad(int kind, int cg);
// the forward product with an epilogue
ExpertOps linear_ops_f16(bool gated, int cg, int bn);
ExpertOps linear_ops_bf16(bool gated, int cg, int bn);
ExpertOps linear_ops_e4m3(bool gated, int cg, int bn);
// Output rows per box of an epilogue with more to do than to round.  What a chunk costs
// whatever its size, waits, fence and store, is some 500 cycles of a warp (bf16 4096^2, K =
// 256, chunks of 16 / 32 rows: nothing in the epilogue 18 / 14 us, gated silu with Z 41 /
// 30); of 64 rows a warp's 4 KB hold no second box.
constexpr int kLinearChunk = 32;

// The same for few rows (linear_rows.cu): fp16 and bf16.
struct LinearRowsParams {
    int32_t rows, experts, N, K;
    int32_t act;                // gemm_act_t
    const void *x, *w, *bias, *residual;
    const int32_t *offsets;     // or null (one matrix)
    void *c, *z;                // z: or null
};
constexpr int kLinearRowsMax = 1024;   // rows, and experts: tables in shared memory

// Clusters of 1, 2, 4 or 8 of these kernels' CTAs (two to an SM) that the device holds at once:
// fewer CTAs than there is room for, since its parts are no multiples of a cluster.
struct RowsRoom {
    int clusters[9];   // [CTAs of a cluster]; [1] 0: not asked yet
};
void ask_rows_room(RowsRoom &room, int sms);

cudaError_t launch_linear_rows(int kind, const LinearRowsParams &p, const RowsRoom &room, cudaStream_t stream, bool overlap);

// ---- rows to the experts and back (expert_route.cu) ---------------------------

constexpr int kMaxExpertsSorted = 1024;   // the sort keeps a count per warp and expert in shared memory

// chunks: 16-byte pieces of a row; prepared: whether the handle has raised the sort's shared-memory limit (its two kernels)
cudaError_t launch_expert_sort(const int32_t *ids, int64_t n, int experts, int32_t *offsets, int32_t *row_of,
                               int32_t *src_of, bool *prepared, cudaStream_t stream, bool overlap);
cudaError_t launch_expert_gather(const void *x, const int32_t *row_of, void *xs, int tokens, int top_k, int chunks,
                                 cudaStream_t stream, bool overlap);
cudaError_t launch_expert_combine(int kind, const void *ys, const int32_t *row_of, const float *w, void *y, int tokens,
                                  int top_k, int chunks, cudaStream_t stream, bool overlap);
cudaError_t launch_expert_combine_grad(int kind, const void *dy, const void *ys, const int32_t *row_of, const float *w,
                                       void *dys, float *dw, int tokens, int top_k, int chunks, cudaStream_t stream,
                                       bool overlap);

// ---- rows times 4-bit weights (nibble.cuh: a few, nibble_rows.cuh: more) ---------------------------------

struct NibbleParams {
    int32_t rows, experts, N, K, group, groups;
    const void *a;            // rows x K, 16-bit
    const uint8_t *b;         // experts x N x K / 2
    const void *scales;       // experts x N x groups, 16-bit
    const uint8_t *zeros;     // experts x N x groups, or null (8)
    const int32_t *offsets;   // experts + 1, or null (one expert has every row)
    void *c;                  // rows x N, 16-bit
    int32_t block_rows;       // rows of a block: 8 (nibble.cuh), 32 or 64 (nibble_rows.cuh)
    int32_t max_blocks;       // blocks that ascending offsets can make
    int32_t ctas;             // SMs
    int32_t cluster, k_warps; // CTAs and warps of a CTA that share a contraction (nibble.cuh: set by the launch)
    int32_t fault_load;       // as above (nibble_rows.cuh)
    uint64_t timeout_ns;
    int32_t *status;
};

constexpr int kNibFeatures = 32;   // features of a tile, rows of the weights' TMA box (128 bytes wide)
constexpr int kNibStageK = 256;    // contraction per unit of work
constexpr int kNibMaxCtas = 4;     // CTAs of a cluster
constexpr int kNibWideFeatures = 128;   // features of a tile where rows are more

// What a handle keeps per dtype: the kernels whose shared-memory limit is
// raised (a bit each), and the clusters of 2 and 4 CTAs the device holds.
struct NibPrepared {
    uint32_t kernels;
    int clusters[2];
};

cudaError_t launch_nibble_f16(const CUtensorMap &b, const NibbleParams &p, NibPrepared *prepared, cudaStream_t stream,
                              bool overlap);
cudaError_t launch_nibble_bf16(const CUtensorMap &b, const NibbleParams &p, NibPrepared *prepared, cudaStream_t stream,
                               bool overlap);
cudaError_t launch_nibble_rows_f16(const CUtensorMap &b, const CUtensorMap &x, const NibbleParams &p, NibPrepared *prepared,
                                   cudaStream_t stream, bool overlap);
cudaError_t launch_nibble_rows_bf16(const CUtensorMap &b, const CUtensorMap &x, const NibbleParams &p, NibPrepared *prepared,
                                    cudaStream_t stream, bool overlap);

}  // namespace pts
