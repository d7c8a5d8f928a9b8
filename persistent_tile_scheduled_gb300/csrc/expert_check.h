// Checks and small helpers that the entry points on rows and experts share.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "gemm_ctx.h"

namespace pts {

constexpr int64_t kIntMax = (int64_t(1) << 31) - 1;
// Sizes of the products: the kernels count in 32 bits, and go up to a tile or a stage past the end.
constexpr int64_t kMaxSize = GEMM_EXPERT_MAX_SIZE;

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool is16(gemm_dtype_t d) { return d == GEMM_F16 || d == GEMM_BF16; }

inline bool is_act(int act)
{
    return act >= 0 && (act & ~GEMM_ACT_GATED) >= GEMM_ACT_NONE && (act & ~GEMM_ACT_GATED) <= GEMM_ACT_SILU;
}

inline gemm_status_t launched(cudaError_t e)
{
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? GEMM_OK : cuda_fail(e);
}

inline gemm_status_t on_device(const gemm_ctx *h)
{
    return cudaSetDevice(h->device) == cudaSuccess ? GEMM_OK : cuda_fail(cudaErrorInvalidDevice);
}

inline const RowsRoom &rows_room(gemm_ctx *h)
{
    if (h->rows_room.clusters[1] == 0) ask_rows_room(h->rows_room, h->sm_count);
    return h->rows_room;
}

inline bool overlap(const gemm_ctx *h) { return h->opts.overlap_launch >= 0; }

}  // namespace pts
