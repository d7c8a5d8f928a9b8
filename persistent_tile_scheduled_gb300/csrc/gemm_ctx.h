// The handle's state and the helpers every entry point shares: error mapping
// and the cache of TMA tensor maps.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/pts_gemm.h"
#include "expert_launch.h"
#include "gemm_params.h"

namespace pts {

constexpr int kBatchSlots = 6;   // gemm_run_host_batch staging depth
constexpr int kGroupSlots = 2;   // gemm_run_grouped problem tables in flight
constexpr int kMapCache = 1024;   // direct-mapped; a K sweep's A, B, C maps rarely collide
constexpr unsigned long long kDefaultTimeoutNs = 1000000000ull;   // 1 s per wait

struct MapEntry {
    const void *ptr = nullptr;
    uint64_t rows = 0, cols = 0;
    int dtype = -1;
    uint32_t box_rows = 0, box_cols = 0;
    CUtensorMap map;
};

inline int elem_bytes(gemm_dtype_t d) { return d == GEMM_E4M3 ? 1 : 2; }

}  // namespace pts

struct gemm_ctx {
    int device = 0;
    int sm_count = 0;
    int max_smem_optin = 0;
    gemm_opts_t opts{};
    int32_t *d_status = nullptr;              // 4 ints
    pts::TileRecord *d_records = nullptr;
    int64_t records_cap = 0;                  // in work items
    int64_t last_work = 0;
    int last_cta_group = 1;
    int64_t last_sk_tiles = 0, last_sk_units = 0, last_num_kb = 0;   // which record slots are pieces
    void *d_host_bufs = nullptr;              // gemm_run_host staging (A | B | C)
    size_t host_bufs_cap = 0;
    float *d_ws_partial = nullptr;            // stream-K fixup workspace
    size_t ws_partial_cap = 0;                // bytes
    uint32_t *d_ws_sync = nullptr;            // stream-K claim counters / ready flags (zero between launches)
    size_t ws_sync_cap = 0;                   // bytes
    // gemm_run_host_batch: staging slots (A | B | C each), copy streams and events
    void *d_slot[pts::kBatchSlots] = {};
    size_t slot_cap = 0;
    cudaStream_t s_h2d = nullptr, s_d2h[2] = {nullptr, nullptr};   // copy-out alternates between two
                                                                    // streams: one reaches ~146 GB/s of
                                                                    // the ~190 two reach (GB300)
    cudaEvent_t ev_entry = nullptr, ev_in[pts::kBatchSlots] = {}, ev_comp[pts::kBatchSlots] = {}, ev_free[pts::kBatchSlots] = {};
    // gemm_run_grouped: problem tables (GroupDesc[count] then int32 group_start[count + 1]),
    // each as uploaded (pinned host copy) and on the device, and the event after the
    // last launch that read it
    void *tab_host[pts::kGroupSlots] = {};
    void *tab_dev[pts::kGroupSlots] = {};
    size_t tab_cap[pts::kGroupSlots] = {};
    size_t tab_bytes[pts::kGroupSlots] = {};   // bytes of the table the slot holds (0 = none)
    cudaEvent_t ev_tab[pts::kGroupSlots] = {};
    int tab_cur = 0;
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    // per dtype, kernel variant (0: wide tile, single CTAs; 1: wide, pairs; 2: narrow tile,
    // single CTAs; 3: narrow tile, pairs) and build (0: the common launch's kernel, 1: full)
    bool smem_set[3][4][2] = {};
    int occ_smem[3][4][2] = {};               // smem the cached occupancy was computed for
    int occ_clusters[3][4][2] = {};
    pts::MapEntry maps[pts::kMapCache];
    // experts' products: resident clusters per dtype, mode and variant (0: single CTAs, 1: pairs,
    // 2: single CTAs with the short row tile); 0 = not asked yet
    int expert_clusters[3][3][3] = {};
    int linear_clusters[3][2][3] = {};        // gemm_run_linear: the same per dtype, plain or gated, and variant
    int linear_shared[3][2][3] = {};          // and clusters of 2, 4 and 8 CTAs that share a tile
    pts::RowsRoom rows_room = {};             // the kernels for few rows
    int grad_clusters[2][2] = {};             // gemm_linear_grad's largest, per dtype, plain or gated; -1: none
    bool sort_smem[2] = {};                   // gemm_expert_sort: limits raised, per kernel
    pts::NibPrepared nibble[2] = {};          // gemm_run_nibble, per dtype
};

namespace pts {

inline gemm_status_t cuda_fail(cudaError_t e)
{
    (void)cudaGetLastError();   // clear a non-sticky error so the next call starts clean
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// Encode (or find) a 2-D row-major tensor map over rows x cols elements.
inline const CUtensorMap *get_map(gemm_ctx *h, const void *ptr, uint64_t rows, uint64_t cols, int dtype,
                           uint32_t box_rows, uint32_t box_cols)
{
    // direct-mapped cache keyed by every field of the map
    uint64_t key = reinterpret_cast<uintptr_t>(ptr) ^ (rows * 0x9E3779B97F4A7C15ull) ^ (cols * 0xC2B2AE3D27D4EB4Full)
                   ^ (uint64_t(dtype) << 7) ^ (uint64_t(box_rows) << 17) ^ (uint64_t(box_cols) << 29);
    key ^= key >> 31;
    key *= 0x94D049BB133111EBull;
    key ^= key >> 29;
    MapEntry &m = h->maps[key % kMapCache];
    if (m.ptr == ptr && m.rows == rows && m.cols == cols && m.dtype == dtype && m.box_rows == box_rows
        && m.box_cols == box_cols)
        return &m.map;
    m.ptr = nullptr;
    CUtensorMapDataType t = dtype == GEMM_F16    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                            : dtype == GEMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int es = dtype == GEMM_E4M3 ? 1 : 2;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols * static_cast<cuuint64_t>(es)};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = h->encode(&m.map, t, 2, const_cast<void *>(ptr), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return nullptr;
    m.ptr = ptr;
    m.rows = rows;
    m.cols = cols;
    m.dtype = dtype;
    m.box_rows = box_rows;
    m.box_cols = box_cols;
    return &m.map;
}

// Encode the tensor map of a depth x rows x cols array of 2-byte or e4m3
// elements (cols contiguous), box box_rows x box_cols of one depth slice.
// box_cols fills the swizzle's width (128, 64 or 32 bytes).
inline bool encode_map3(const gemm_ctx *h, CUtensorMap *out, const void *ptr, uint64_t depth, uint64_t rows,
                        uint64_t cols, int dtype, uint32_t box_rows, uint32_t box_cols)
{
    const int es = dtype == GEMM_E4M3 ? 1 : 2;
    const CUtensorMapDataType t = dtype == GEMM_F16    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                  : dtype == GEMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    cuuint64_t dims[3] = {cols, rows, depth};
    cuuint64_t strides[2] = {cols * static_cast<cuuint64_t>(es), rows * cols * static_cast<cuuint64_t>(es)};
    cuuint32_t box[3] = {box_cols, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return h->encode(out, t, 3, const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     box_cols * es == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
                     : box_cols * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                           : CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE)
           == CUDA_SUCCESS;
}

inline CUtensorMapDataType map_type(int dtype)
{
    return dtype == GEMM_F16    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
           : dtype == GEMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                : CU_TENSOR_MAP_DATA_TYPE_UINT8;
}

// The matrices of a gated product, depth x (n gate rows, then n others) x cols, as
// 8 gate rows, the 8 others of the same features, the next 8 gate rows, ...: a box
// of 128 rows holds 64 features of both.  n is a multiple of 8.
inline bool encode_map_gated(const gemm_ctx *h, CUtensorMap *out, const void *ptr, uint64_t depth, uint64_t n, uint64_t cols,
                             int dtype, uint32_t box_cols)
{
    const cuuint64_t row = cols * (dtype == GEMM_E4M3 ? 1 : 2);
    cuuint64_t dims[5] = {cols, 8, 2, n / 8, depth};
    cuuint64_t strides[4] = {row, n * row, 8 * row, 2 * n * row};
    cuuint32_t box[5] = {box_cols, 8, 2, 8, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return h->encode(out, map_type(dtype), 5, const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE)
           == CUDA_SUCCESS;
}

// Rows of n gate values and n others (2-byte) as n x 2 x rows, so that a box of
// either half ends at its last feature: box_rows x 16 of one half.
inline bool encode_map_halves(const gemm_ctx *h, CUtensorMap *out, const void *ptr, uint64_t rows, uint64_t n, int dtype, uint32_t box_rows)
{
    cuuint64_t dims[3] = {n, 2, rows};
    cuuint64_t strides[2] = {2 * n, 4 * n};
    cuuint32_t box[3] = {16, 1, box_rows};
    cuuint32_t estr[3] = {1, 1, 1};
    return h->encode(out, map_type(dtype), 3, const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE)
           == CUDA_SUCCESS;
}

}  // namespace pts
