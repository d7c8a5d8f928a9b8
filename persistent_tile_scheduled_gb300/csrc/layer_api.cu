// C ABI of what stands around the products (routing, the epilogue's gradient, a
// layer of experts for a few tokens): argument checks and launches.  Declared in
// pts_gemm.h.
#include "expert_check.h"
#include "layer_launch.h"

using namespace pts;

namespace {

gemm_status_t check_route(const gemm_ctx *h, int64_t tokens, int64_t top_k, int64_t experts, const void *logits,
                          gemm_route_t mode, gemm_dtype_t dtype)
{
    if (h == nullptr || tokens < 0 || tokens > kIntMax) return GEMM_ERR_INVALID_ARG;
    if (mode < GEMM_ROUTE_SELECTED || mode > GEMM_ROUTE_SIGMOID || (!is16(dtype) && dtype != GEMM_F32)) return GEMM_ERR_INVALID_ARG;
    if (experts < 1 || experts > GEMM_EXPERT_SORT_MAX_EXPERTS || top_k < 1 || top_k > experts || top_k > GEMM_EXPERT_ROUTE_MAX_TOP_K)
        return GEMM_ERR_INVALID_ARG;
    const uintptr_t mask = dtype == GEMM_F32 ? 3 : 1;
    if (tokens > 0 && (logits == nullptr || (reinterpret_cast<uintptr_t>(logits) & mask))) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

RouteParams route_params(int64_t tokens, int64_t top_k, int64_t experts, const void *logits, gemm_route_t mode)
{
    RouteParams p{};
    p.tokens = tokens;
    p.top_k = static_cast<int32_t>(top_k);
    p.experts = static_cast<int32_t>(experts);
    p.mode = static_cast<int32_t>(mode);
    p.logits = logits;
    return p;
}

}  // namespace

extern "C" {

gemm_status_t gemm_expert_route(gemm_handle_t h, int64_t tokens, int64_t top_k, int64_t experts, const void *logits,
                                int32_t *expert_ids, float *weights, gemm_route_t mode, gemm_dtype_t dtype, void *stream)
{
    gemm_status_t st = check_route(h, tokens, top_k, experts, logits, mode, dtype);
    if (st != GEMM_OK) return st;
    if (tokens == 0) return GEMM_OK;
    if (expert_ids == nullptr || weights == nullptr || !aligned4(expert_ids) || !aligned4(weights)) return GEMM_ERR_INVALID_ARG;
    if ((st = on_device(h)) != GEMM_OK) return st;
    RouteParams p = route_params(tokens, top_k, experts, logits, mode);
    p.ids = expert_ids;
    p.weights = weights;
    return launched(launch_route(static_cast<int>(dtype), p, static_cast<cudaStream_t>(stream), overlap(h)));
}

gemm_status_t gemm_expert_route_grad(gemm_handle_t h, int64_t tokens, int64_t top_k, int64_t experts, const void *logits,
                                     const int32_t *expert_ids, const float *dweights, void *dlogits, gemm_route_t mode,
                                     gemm_dtype_t dtype, void *stream)
{
    gemm_status_t st = check_route(h, tokens, top_k, experts, logits, mode, dtype);
    if (st != GEMM_OK) return st;
    if (tokens == 0) return GEMM_OK;
    if (expert_ids == nullptr || dweights == nullptr || dlogits == nullptr || !aligned4(expert_ids) || !aligned4(dweights)) return GEMM_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(dlogits) & (dtype == GEMM_F32 ? 3 : 1)) return GEMM_ERR_INVALID_ARG;
    if ((st = on_device(h)) != GEMM_OK) return st;
    RouteParams p = route_params(tokens, top_k, experts, logits, mode);
    p.ids = const_cast<int32_t *>(expert_ids);
    p.dweights = dweights;
    p.dlogits = dlogits;
    return launched(launch_route_grad(static_cast<int>(dtype), p, static_cast<cudaStream_t>(stream), overlap(h)));
}

gemm_status_t gemm_linear_grad(gemm_handle_t h, int64_t rows, int64_t experts, int64_t N, const void *dC, const void *Z,
                               const int32_t *offsets, void *dZ, float *dbias, int act, gemm_dtype_t dtype, void *stream)
{
    if (h == nullptr || !is16(dtype) || !is_act(act) || rows < 0 || experts < 0 || N < 0) return GEMM_ERR_INVALID_ARG;
    if (rows > kMaxSize || experts > kMaxSize || N > kMaxSize || N % 8 != 0) return GEMM_ERR_INVALID_ARG;
    if (experts > 0 && ((offsets == nullptr && experts != 1) || !aligned4(offsets))) return GEMM_ERR_INVALID_ARG;
    if (experts == 0 || N == 0 || (rows == 0 && dbias == nullptr)) return GEMM_OK;
    if (rows > 0 && (dC == nullptr || Z == nullptr || dZ == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(dC) || !aligned16(Z) || !aligned16(dZ) || !aligned4(dbias)) return GEMM_ERR_INVALID_ARG;
    if (experts * ((N + 31) / 32) * 8 > kIntMax || ((act & GEMM_ACT_GATED) && N > kMaxSize / 2)) return GEMM_ERR_INVALID_ARG;   // CTAs
    gemm_status_t st = on_device(h);
    if (st != GEMM_OK) return st;
    LinearGradParams p{};
    p.rows = rows;
    p.experts = static_cast<int32_t>(experts);
    p.N = static_cast<int32_t>(N);
    p.act = act;
    p.dc = dC;
    p.z = Z;
    p.offsets = offsets;
    p.dz = dZ;
    p.dbias = dbias;
    p.sms = h->sm_count;
    int &room = h->grad_clusters[dtype][(act & GEMM_ACT_GATED) != 0];
    if (room == 0 && dbias != nullptr) {
        room = ask_linear_grad_room(static_cast<int>(dtype), act & GEMM_ACT_GATED);
        if (room < 1) room = -1;
    }
    return launched(launch_linear_grad(static_cast<int>(dtype), p, room, static_cast<cudaStream_t>(stream), overlap(h)));
}

gemm_status_t gemm_expert_layer(gemm_handle_t h, int64_t tokens, int64_t top_k, int64_t experts, int64_t dim,
                                int64_t hidden, const void *X, const int32_t *expert_ids, const float *weights,
                                const void *up, const void *up_bias, const void *down, const void *down_bias,
                                const void *residual, void *Hs, void *Y, int act, gemm_dtype_t dtype, void *stream)
{
    static_assert(GEMM_EXPERT_LAYER_MAX_TOKENS == kLayerMaxTokens && GEMM_EXPERT_LAYER_MAX_ASSIGNMENTS == kLayerMaxAssignments
                  && GEMM_EXPERT_SORT_MAX_EXPERTS == kLayerMaxExperts, "");
    if (h == nullptr || !is16(dtype) || !is_act(act)) return GEMM_ERR_INVALID_ARG;
    if (tokens < 0 || tokens > kLayerMaxTokens || top_k < 1 || top_k > kLayerMaxAssignments || tokens * top_k > kLayerMaxAssignments)
        return GEMM_ERR_INVALID_ARG;
    if (experts < 0 || experts > kLayerMaxExperts || dim < 0 || dim > kMaxSize || hidden < 0 || hidden > kMaxSize) return GEMM_ERR_INVALID_ARG;
    if (dim % 8 != 0 || hidden % 8 != 0) return GEMM_ERR_INVALID_ARG;
    // the kernels count items in 32 bits, blocks times tiles of 8 features, and go up to a stride of the grid past
    // the last: a block has a token at least, so there are no more of them than assignments
    if (static_cast<int64_t>(kLayerMaxAssignments + kLayerMaxAssignments / 16) * ((hidden + 7) / 8) > kIntMax) return GEMM_ERR_INVALID_ARG;
    if (tokens == 0 || dim == 0) return GEMM_OK;
    if (Y == nullptr || expert_ids == nullptr || weights == nullptr) return GEMM_ERR_INVALID_ARG;
    if (experts > 0 && (X == nullptr || (hidden > 0 && (up == nullptr || down == nullptr || Hs == nullptr)))) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(up) || !aligned16(up_bias) || !aligned16(down) || !aligned16(down_bias) || !aligned16(residual)
        || !aligned16(Hs) || !aligned16(Y) || !aligned4(expert_ids) || !aligned4(weights))
        return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = on_device(h);
    if (st != GEMM_OK) return st;
    LayerParams p{};
    p.tokens = static_cast<int32_t>(tokens);
    p.top_k = static_cast<int32_t>(top_k);
    p.experts = static_cast<int32_t>(experts);
    p.dim = static_cast<int32_t>(dim);
    p.hidden = static_cast<int32_t>(experts > 0 ? hidden : 0);
    p.act = act;
    p.x = X;
    p.ids = expert_ids;
    p.weights = weights;
    p.up = up;
    p.up_bias = up_bias;
    p.down = down;
    p.down_bias = down_bias;
    p.residual = residual;
    p.hs = Hs;
    p.y = Y;
    return launched((dtype == GEMM_F16 ? launch_layer_f16 : launch_layer_bf16)(p, rows_room(h), static_cast<cudaStream_t>(stream), overlap(h)));
}

}  // extern "C"
