// Launch entry points of what stands around the products: routing, the
// epilogue's gradient, a layer of experts for a few tokens.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace pts {

// ---- routing (route.cu); kind: 0 fp16, 1 bf16, 3 fp32 -----------------------------
struct RouteParams {
    int64_t tokens;
    int32_t top_k, experts;
    int32_t mode;             // gemm_route_t
    const void *logits;
    int32_t *ids;             // (the gradient reads them)
    float *weights;
    const float *dweights;
    void *dlogits;
};

cudaError_t launch_route(int kind, const RouteParams &p, cudaStream_t stream, bool overlap);
cudaError_t launch_route_grad(int kind, const RouteParams &p, cudaStream_t stream, bool overlap);

// ---- the epilogue's gradient (linear_grad.cu) ---------------------------------------
struct LinearGradParams {
    int64_t rows;
    int32_t experts, N;
    int32_t act;              // gemm_act_t
    const void *dc, *z;
    const int32_t *offsets;   // or null (one matrix)
    void *dz;
    float *dbias;             // or null
    int32_t sms;
};

// Clusters of the most CTAs that share an expert's rows, as many as the device holds at once.
int ask_linear_grad_room(int kind, bool gated);
cudaError_t launch_linear_grad(int kind, const LinearGradParams &p, int room, cudaStream_t stream, bool overlap);

// ---- a layer of experts for a few tokens (expert_layer.cuh) -------------------------
constexpr int kLayerMaxTokens = 64;         // a mask of an expert's tokens is 64 bits
constexpr int kLayerMaxAssignments = 512;   // tables in shared memory
constexpr int kLayerMaxExperts = 1024;

struct LayerParams {
    int32_t tokens, top_k, experts, dim, hidden;
    int32_t act;
    const void *x;
    const int32_t *ids;
    const float *weights;
    const void *up, *up_bias, *down, *down_bias, *residual;
    void *hs, *y;
};

struct RowsRoom;   // expert_launch.h
cudaError_t launch_layer_f16(const LayerParams &p, const RowsRoom &room, cudaStream_t stream, bool overlap);
cudaError_t launch_layer_bf16(const LayerParams &p, const RowsRoom &room, cudaStream_t stream, bool overlap);

}  // namespace pts
