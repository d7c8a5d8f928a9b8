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
};

// producer, MMA, 4 epilogue warps, scheduler; WGRAD has a clearing warp too
__host__ __device__ constexpr int expert_threads(int mode) { return kThreads + (mode == EXPERT_WGRAD ? 32 : 0); }

// Dynamic shared memory for `stages` stages of a tile of bn rows (plus 1 KB
// for aligning the base to the swizzle period).
__host__ __device__ constexpr int expert_smem_bytes(int cg, int bn, int stages)
{
    return 1024 + stages * kb_per_stage(cg) * (kRowsPerCta + bn / cg) * kKBlockBytes + epi_bytes()
           + 8 * (3 * kMaxStages + 4 + 2 * kRing) + 16   // mbarriers, alignment
           + 4 * kRingWords * kRing + 16;                // ring payload, TMEM base, abort flag
}

constexpr int kExpertTileN = 256;       // rows of a tile
constexpr int kExpertTileNFew = 64;     // rows of a tile when the experts have few:
constexpr int64_t kExpertFewRows = 32;  // at most so many on average

struct ExpertOps {
    cudaError_t (*prepare)(int smem, int sms, int *clusters);
    cudaError_t (*launch)(const CUtensorMap &w, const CUtensorMap &x, const CUtensorMap &xs, const CUtensorMap &o,
                          const ExpertParams &p, int grid, int smem, cudaStream_t stream, bool overlap);
};

// kind: 0 fp16, 1 bf16, 2 e4m3 (forward only); bn: kExpertTileN, or
// kExpertTileNFew (forward, single CTAs)
ExpertOps expert_ops_fwd(int kind, int cg, int bn);
ExpertOps expert_ops_dgrad(int kind, int cg);
ExpertOps expert_ops_wgrad(int kind, int cg);

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
