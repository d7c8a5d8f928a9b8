// C ABI of the expert layer's operators: argument checks, tensor maps and
// launches.  Declared in pts_gemm.h.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "expert_launch.h"
#include "gemm_ctx.h"
#include "gemm_plan.h"

using namespace pts;

namespace {

constexpr int64_t kLim = (int64_t(1) << 31) - 1;
// Sizes of the products: the kernels count in 32 bits, and go up to a tile or a stage past the end.
constexpr int64_t kMaxSize = GEMM_EXPERT_MAX_SIZE;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool is16(gemm_dtype_t d) { return d == GEMM_F16 || d == GEMM_BF16; }

gemm_status_t launched(cudaError_t e)
{
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? GEMM_OK : cuda_fail(e);
}

gemm_status_t on_device(const gemm_ctx *h)
{
    return cudaSetDevice(h->device) == cudaSuccess ? GEMM_OK : cuda_fail(cudaErrorInvalidDevice);
}

// The stage load that announces too many bytes (GEMM_DEBUG_FAULT_SKIP_TMA), or -1.
int32_t fault_load(const gemm_ctx *h) { return h->opts.debug_flags & GEMM_DEBUG_FAULT_SKIP_TMA ? h->opts.fault_arg : -1; }

bool overlap(const gemm_ctx *h) { return h->opts.overlap_launch >= 0; }

// Common checks of the row kernels: tokens x top_k assignments, rows of dim elements.
gemm_status_t check_rows(gemm_ctx *h, int64_t tokens, int64_t top_k, int64_t dim, int es)
{
    if (h == nullptr || tokens < 0 || top_k < 1 || dim < 0 || dim > kLim) return GEMM_ERR_INVALID_ARG;
    if (top_k > kLim || tokens > kLim || tokens * top_k > kLim) return GEMM_ERR_INVALID_ARG;
    if ((dim * es) % 16 != 0) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

// One product of the experts.  features / contraction / out_rows as in
// ExpertParams; W and X as in expert_gemm.cuh.
gemm_status_t run_product(gemm_ctx *h, int mode, int64_t rows, int64_t experts, int64_t N, int64_t K, const void *W,
                          const void *X, const int32_t *offsets, void *out, gemm_dtype_t dtype, float out_scale,
                          cudaStream_t stream)
{
    const int64_t features = mode == EXPERT_FWD ? N : K;
    const int64_t contraction = mode == EXPERT_FWD ? K : N;   // (WGRAD: an expert's rows)
    const int kelems = dtype == GEMM_E4M3 ? 128 : 64;
    // Variant (cta_group 0).  Few rows per expert: the weights' bytes count, and
    // tiles of 64 rows leave room for 8 stages of them (us on GB300, this / pairs:
    // 64 rows over 8 experts of 4096^2 44.9 / 47.6, 256 45.5 / 48.4, 2048 over 64 of
    // 2048^2 85.3 / 90.3; but 512 over 8 53.1 / 49.9, an expert's rows then being
    // several tiles).  Else pairs from 14 k-blocks per tile, as in gemm_run: 16384
    // over 32, K = 1024, 103 / 111 for singles, 300 over 19, K = 560, 6.6 / 5.5.  The
    // weights' gradient counts the k-blocks of an average expert's rows: 4096 over
    // 4 33.5 / 33.1, 6000 over 24 42.2 / 36.7, 64 over 8 86 / 43.
    int cg = h->opts.cta_group;
    int bn = kExpertTileN;
    const int64_t length = mode == EXPERT_WGRAD ? rows / experts : contraction;
    if (cg == 0) cg = choose_cta_group((length + kelems - 1) / kelems);
    if (mode == EXPERT_FWD && h->opts.cta_group != 2 && rows <= kExpertFewRows * experts) {
        cg = 1;
        bn = kExpertTileNFew;
    }
    int stages = kMaxStages;
    while (stages > 2 && expert_smem_bytes(cg, bn, stages) > h->max_smem_optin) --stages;
    const int smem = expert_smem_bytes(cg, bn, stages);
    const int kind = static_cast<int>(dtype);
    const ExpertOps ops = mode == EXPERT_FWD ? expert_ops_fwd(kind, cg, bn)
                          : mode == EXPERT_DGRAD ? expert_ops_dgrad(kind, cg)
                                                 : expert_ops_wgrad(kind, cg);
    int &resident = h->expert_clusters[kind][mode][bn == kExpertTileNFew ? 2 : cg - 1];
    if (resident == 0) {
        int n = 0;
        if (ops.prepare(smem, h->sm_count, &n) != cudaSuccess) return cuda_fail(cudaErrorInvalidValue);
        if (n < 1) return GEMM_ERR_CUDA;
        resident = n;
    }
    // tiles: at most one short one per expert on top of the rows' own
    const int64_t tf = (features + kRowsPerCta * cg - 1) / (kRowsPerCta * cg);
    const int64_t used = rows < experts ? rows : experts;
    const int64_t tiles = mode == EXPERT_WGRAD ? experts * tf * ((N + bn - 1) / bn) : (rows / bn + used) * tf;
    if (tiles > (int64_t(1) << 30)) return GEMM_ERR_INVALID_ARG;
    int64_t clusters = h->opts.max_clusters > 0 && h->opts.max_clusters < resident ? h->opts.max_clusters : resident;
    if (clusters > tiles) clusters = tiles;
    // Tiles for less than half the SMs: CTAs share a tile's contraction, 0.2 us per
    // k-block saved for 2.8 us of joining (us, this / one CTA per tile: one row of 1024 x
    // 8192 10.0 / 32.7, of 2048^2 8.4 / 10.8, of 8192^2, 2 CTAs, 27.6 / 34.1; but of 512 x
    // 1024 7.2 / 6.8 and of 8192 x 1024 8.5 / 7.1).  Few clusters of 8 find room at once:
    // 16 tiles of that contraction take 20.7 by 8 CTAs each, 14.6 by 4.
    int split = 1;
    const int64_t length_kb = (contraction + kelems - 1) / kelems;
    if (mode == EXPERT_FWD && bn == kExpertTileNFew && h->opts.cta_group == 0 && h->opts.max_clusters == 0 && length_kb >= 24) {
        while (split < 4 && tiles * split * 2 <= h->sm_count) split *= 2;
        if (split == 4 && length_kb >= 64 && tiles * 16 <= h->sm_count) split = 8;
        if (split == 2 && length_kb < 32) split = 1;
    }

    CUtensorMap mw, mx, mxs, mo;
    std::memset(&mw, 0, sizeof(mw));
    mx = mxs = mo = mw;
    bool ok = true;
    const uint32_t stage_rows = static_cast<uint32_t>(64 * kb_per_stage(cg));   // contraction rows of a stage
    if (mode == EXPERT_WGRAD) {
        ok = encode_map3(h, &mw, W, 1, rows, K, dtype, stage_rows, 64) && encode_map3(h, &mx, X, 1, rows, N, dtype, stage_rows, 64);
        mxs = mx;
        ok = ok && encode_map3(h, &mo, out, experts, N, K, dtype, 64, 32);
    } else {
        if (contraction > 0) {
            ok = mode == EXPERT_FWD ? encode_map3(h, &mw, W, experts, N, K, dtype, kRowsPerCta, kelems)
                                    : encode_map3(h, &mw, W, experts, N, K, dtype, stage_rows, 64);
            ok = ok && encode_map3(h, &mx, X, 1, rows, contraction, dtype, static_cast<uint32_t>(bn / cg), kelems)
                 && encode_map3(h, &mxs, X, 1, rows, contraction, dtype, 16, kelems);
        }
        ok = ok
             && encode_map3(h, &mo, out, 1, rows, features, dtype == GEMM_E4M3 ? GEMM_BF16 : dtype, 64, 32);
    }
    if (!ok) return GEMM_ERR_INVALID_ARG;

    ExpertParams p{};
    p.rows = static_cast<int32_t>(rows);
    p.experts = static_cast<int32_t>(experts);
    p.features = static_cast<int32_t>(features);
    p.contraction = static_cast<int32_t>(contraction);
    p.out_rows = static_cast<int32_t>(N);
    p.stages = stages;
    p.group_m = h->opts.group_size_m;
    p.split = split;
    p.out_scale = out_scale;
    p.offsets = offsets;
    p.out = out;
    p.fault_load = fault_load(h);
    p.timeout_ns = h->opts.timeout_ns;
    p.status = h->d_status;
    return launched(ops.launch(mw, mx, mxs, mo, p, static_cast<int>(clusters) * cg * split, smem, stream, overlap(h)));
}

// How the product with 4-bit weights is done: rows of a block (8: nibble.cuh, 32
// or 64: nibble_rows.cuh, there with `cluster` CTAs to a tile's contraction).
struct NibbleForm {
    int block_rows, cluster;
};

// The form that should take the least time, each by what it takes (GB300, us; the
// groups' size and the zeros change it little).  By 8: 3.4 and 1 per 8.2 million
// weights of each row block.  By 32 or 64: 5.2 and, of a CTA, 0.95 or 1.5 per 256
// of the contraction of a tile of 128 features.  Measured / so reckoned:
//   rows of 8192^2         8: 13.4 / 11.6    16: 20.3 / 19.8, by 32 19.3 / 20.4
//                          24: 30.6 / 28, by 32 19.4 / 20.4    64: 69 / 69, by 64 29.2 / 29
//   64 rows of 20480 x 16384 by 64 with 1, 2, 4 CTAs to a tile 184 / 197, 155 / 160, 147 / 146
//   16 rows of 1000 x 2048 4.3 / 3.9, by 32 7.4 / 7.1
//   32 experts, 2048 x 4096, 10 rows each 66 / 59, by 32 63 / 66; 16 experts, 24 rows each
//   50 / 60, by 32 32.6 / 51
// The rows of each expert are device data: an expert's last block is taken as 0.45 full.
NibbleForm nibble_form(const gemm_ctx *h, int64_t rows, int64_t experts, int64_t N, int64_t K, bool spread)
{
    if (h->opts.debug_flags & GEMM_DEBUG_NIBBLE_FORM(0xff, 0))
        return NibbleForm{static_cast<int>(h->opts.debug_flags >> 8 & 0xff), static_cast<int>(h->opts.debug_flags >> 16 & 0xf)};
    auto blocks = [&](int of) -> double {
        if (!spread) return static_cast<double>((rows + of - 1) / of);
        const double n = static_cast<double>(rows) / of + 0.45 * static_cast<double>(experts), used = static_cast<double>(rows < experts ? rows : experts);
        return n > used ? n : used;
    };
    NibbleForm best{8, 1};
    double least = 3.4 + blocks(8) * static_cast<double>(N) * static_cast<double>(K) / 8.2e6;
    const double features = static_cast<double>((N + kNibWideFeatures - 1) / kNibWideFeatures);
    const double stages = static_cast<double>((K + kNibStageK - 1) / kNibStageK);
    for (int of = 32; of <= 64; of += 32)
        for (int c = 1; c <= kNibMaxCtas; c *= 2) {
            const double rounds = std::ceil(blocks(of) * features * c / h->sm_count), each = std::ceil(stages / c);
            const double time = (c == 1 ? 5.2 : 5.2 * rounds) + rounds * each * (of == 32 ? 0.95 : 1.5);
            if (time < least) least = time, best = NibbleForm{of, c};
        }
    return best;
}

gemm_status_t check_product(gemm_ctx *h, int64_t rows, int64_t experts, int64_t N, int64_t K, const int32_t *offsets)
{
    if (h == nullptr || rows < 0 || experts < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (rows > kMaxSize || experts > kMaxSize || N > kMaxSize || K > kMaxSize) return GEMM_ERR_INVALID_ARG;
    if (experts > 0 && (offsets == nullptr || !aligned4(offsets))) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t gemm_expert_sort(gemm_handle_t h, int64_t tokens, int64_t top_k, int64_t experts,
                               const int32_t *expert_ids, int32_t *offsets, int32_t *row_of, int32_t *src_of,
                               void *stream)
{
    gemm_status_t st = check_rows(h, tokens, top_k, 0, 2);
    if (st != GEMM_OK) return st;
    if (experts < 1 || experts > kMaxExpertsSorted || offsets == nullptr || !aligned4(offsets)) return GEMM_ERR_INVALID_ARG;
    const int64_t n = tokens * top_k;
    if (n > 0 && (expert_ids == nullptr || row_of == nullptr || src_of == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (!aligned4(expert_ids) || !aligned4(row_of) || !aligned4(src_of)) return GEMM_ERR_INVALID_ARG;
    if ((st = on_device(h)) != GEMM_OK) return st;
    return launched(launch_expert_sort(expert_ids, n, static_cast<int>(experts), offsets, row_of, src_of,
                                       h->sort_smem, static_cast<cudaStream_t>(stream), overlap(h)));
}

gemm_status_t gemm_expert_gather(gemm_handle_t h, int64_t tokens, int64_t top_k, int64_t dim, const void *X,
                                 const int32_t *row_of, void *Xs, gemm_dtype_t dtype, void *stream)
{
    if (dtype < GEMM_F16 || dtype > GEMM_E4M3) return GEMM_ERR_INVALID_ARG;
    const int es = elem_bytes(dtype);
    gemm_status_t st = check_rows(h, tokens, top_k, dim, es);
    if (st != GEMM_OK) return st;
    if (tokens == 0 || dim == 0) return GEMM_OK;
    if (X == nullptr || Xs == nullptr || row_of == nullptr) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(Xs) || !aligned4(row_of)) return GEMM_ERR_INVALID_ARG;
    if ((st = on_device(h)) != GEMM_OK) return st;
    return launched(launch_expert_gather(X, row_of, Xs, static_cast<int>(tokens), static_cast<int>(top_k),
                                         static_cast<int>(dim * es / 16), static_cast<cudaStream_t>(stream), overlap(h)));
}

gemm_status_t gemm_expert_combine(gemm_handle_t h, int64_t tokens, int64_t top_k, int64_t dim, const void *Ys,
                                  const int32_t *row_of, const float *weights, void *Y, gemm_dtype_t dtype,
                                  void *stream)
{
    if (!is16(dtype)) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_rows(h, tokens, top_k, dim, 2);
    if (st != GEMM_OK) return st;
    if (tokens == 0 || dim == 0) return GEMM_OK;
    if (Ys == nullptr || Y == nullptr || row_of == nullptr) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(Ys) || !aligned16(Y) || !aligned4(row_of) || !aligned4(weights)) return GEMM_ERR_INVALID_ARG;
    if ((st = on_device(h)) != GEMM_OK) return st;
    return launched(launch_expert_combine(static_cast<int>(dtype), Ys, row_of, weights, Y, static_cast<int>(tokens),
                                          static_cast<int>(top_k), static_cast<int>(dim / 8),
                                          static_cast<cudaStream_t>(stream), overlap(h)));
}

gemm_status_t gemm_expert_combine_grad(gemm_handle_t h, int64_t tokens, int64_t top_k, int64_t dim, const void *dY,
                                       const void *Ys, const int32_t *row_of, const float *weights, void *dYs,
                                       float *dweights, gemm_dtype_t dtype, void *stream)
{
    if (!is16(dtype)) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_rows(h, tokens, top_k, dim, 2);
    if (st != GEMM_OK) return st;
    if (tokens == 0) return GEMM_OK;
    if (row_of == nullptr || weights == nullptr || dweights == nullptr) return GEMM_ERR_INVALID_ARG;
    if (dim > 0 && (dY == nullptr || Ys == nullptr || dYs == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(dY) || !aligned16(Ys) || !aligned16(dYs) || !aligned4(row_of) || !aligned4(weights)
        || !aligned4(dweights))
        return GEMM_ERR_INVALID_ARG;
    if ((st = on_device(h)) != GEMM_OK) return st;
    return launched(launch_expert_combine_grad(static_cast<int>(dtype), dY, Ys, row_of, weights, dYs, dweights,
                                               static_cast<int>(tokens), static_cast<int>(top_k),
                                               static_cast<int>(dim / 8), static_cast<cudaStream_t>(stream),
                                               overlap(h)));
}

gemm_status_t gemm_run_experts(gemm_handle_t h, int64_t rows, int64_t experts, int64_t N, int64_t K, const void *A,
                               const void *B, const int32_t *offsets, void *C, gemm_dtype_t dtype, float scale_a,
                               float scale_b, void *stream)
{
    if (dtype < GEMM_F16 || dtype > GEMM_E4M3) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_product(h, rows, experts, N, K, offsets);
    if (st != GEMM_OK) return st;
    if ((K * elem_bytes(dtype)) % 16 != 0 || (N * 2) % 16 != 0) return GEMM_ERR_INVALID_ARG;
    float scale = 1.0f;
    if (dtype == GEMM_E4M3) {
        if (!(scale_a > 0.0f) || !(scale_b > 0.0f) || !std::isfinite(scale_a) || !std::isfinite(scale_b))
            return GEMM_ERR_INVALID_ARG;
        scale = static_cast<float>(1.0 / (static_cast<double>(scale_a) * static_cast<double>(scale_b)));
    }
    if (rows == 0 || experts == 0 || N == 0) return GEMM_OK;
    if (C == nullptr || !aligned16(C)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (A == nullptr || B == nullptr || !aligned16(A) || !aligned16(B))) return GEMM_ERR_INVALID_ARG;
    if ((st = on_device(h)) != GEMM_OK) return st;
    return run_product(h, EXPERT_FWD, rows, experts, N, K, B, A, offsets, C, dtype, scale,
                       static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_run_experts_dgrad(gemm_handle_t h, int64_t rows, int64_t experts, int64_t N, int64_t K,
                                     const void *dC, const void *B, const int32_t *offsets, void *dA,
                                     gemm_dtype_t dtype, void *stream)
{
    if (!is16(dtype)) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_product(h, rows, experts, N, K, offsets);
    if (st != GEMM_OK) return st;
    if ((K * 2) % 16 != 0 || (N * 2) % 16 != 0) return GEMM_ERR_INVALID_ARG;
    if (rows == 0 || experts == 0 || K == 0) return GEMM_OK;
    if (dA == nullptr || !aligned16(dA)) return GEMM_ERR_INVALID_ARG;
    if (N > 0 && (dC == nullptr || B == nullptr || !aligned16(dC) || !aligned16(B))) return GEMM_ERR_INVALID_ARG;
    if ((st = on_device(h)) != GEMM_OK) return st;
    return run_product(h, EXPERT_DGRAD, rows, experts, N, K, B, dC, offsets, dA, dtype, 1.0f,
                       static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_run_experts_wgrad(gemm_handle_t h, int64_t rows, int64_t experts, int64_t N, int64_t K,
                                     const void *dC, const void *A, const int32_t *offsets, void *dB,
                                     gemm_dtype_t dtype, void *stream)
{
    if (!is16(dtype)) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_product(h, rows, experts, N, K, offsets);
    if (st != GEMM_OK) return st;
    if ((K * 2) % 16 != 0 || (N * 2) % 16 != 0) return GEMM_ERR_INVALID_ARG;
    if (experts == 0 || N == 0 || K == 0) return GEMM_OK;
    if (dB == nullptr || !aligned16(dB)) return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && (dC == nullptr || A == nullptr || !aligned16(dC) || !aligned16(A))) return GEMM_ERR_INVALID_ARG;
    if ((st = on_device(h)) != GEMM_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0)   // every sum is empty
        return launched(cudaMemsetAsync(dB, 0, static_cast<size_t>(experts) * N * K * 2, s));
    return run_product(h, EXPERT_WGRAD, rows, experts, N, K, A, dC, offsets, dB, dtype, 1.0f, s);
}

gemm_status_t gemm_run_nibble(gemm_handle_t h, int64_t rows, int64_t experts, int64_t N, int64_t K, int64_t group,
                              const void *A, const void *B, const void *scales, const uint8_t *zeros,
                              const int32_t *offsets, void *C, gemm_dtype_t dtype, void *stream)
{
    if (!is16(dtype) || h == nullptr || rows < 0 || experts < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (rows > kMaxSize || experts > kMaxSize || N > kMaxSize || K > kMaxSize) return GEMM_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return GEMM_ERR_INVALID_ARG;
    if (K % 32 != 0 || N % 8 != 0) return GEMM_ERR_INVALID_ARG;
    if (rows == 0 || experts == 0 || N == 0) return GEMM_OK;
    if ((offsets == nullptr && experts != 1) || !aligned4(offsets)) return GEMM_ERR_INVALID_ARG;
    if (experts > kMaxSize / N) return GEMM_ERR_INVALID_ARG;   // rows of the weights
    // the kernel counts its pieces of work in 32 bits
    const NibbleForm form = nibble_form(h, rows, experts, N, K, offsets != nullptr);
    const int64_t used = rows < experts ? rows : experts;
    const int64_t max_blocks = (rows + (form.block_rows - 1) * used) / form.block_rows;
    if (max_blocks * (N / 16 + 1) > 2000000000) return GEMM_ERR_INVALID_ARG;
    if (C == nullptr || !aligned16(C)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (A == nullptr || B == nullptr || scales == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(A) || !aligned16(B) || !aligned16(scales) || !aligned16(zeros)) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = on_device(h);
    if (st != GEMM_OK) return st;
    NibbleParams p{};
    p.rows = static_cast<int32_t>(rows);
    p.experts = static_cast<int32_t>(experts);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.group = static_cast<int32_t>(group);
    p.groups = static_cast<int32_t>((K + group - 1) / group);
    p.a = A;
    p.b = static_cast<const uint8_t *>(B);
    p.scales = scales;
    p.zeros = zeros;
    p.offsets = offsets;
    p.c = C;
    p.block_rows = form.block_rows;
    p.cluster = form.cluster;
    p.max_blocks = static_cast<int32_t>(max_blocks);
    p.ctas = h->sm_count;
    p.fault_load = fault_load(h);
    p.timeout_ns = h->opts.timeout_ns;
    p.status = h->d_status;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    NibPrepared *prepared = &h->nibble[dtype];
    CUtensorMap mb, mx;
    std::memset(&mb, 0, sizeof(mb));
    mx = mb;
    // (by 8 the test hook is a box that is a row short of what every load announces)
    const uint32_t features = form.block_rows == 8 ? kNibFeatures - (p.fault_load >= 0 ? 1 : 0) : kNibWideFeatures;
    if (K > 0 && !encode_map3(h, &mb, B, 1, experts * N, K / 2, GEMM_E4M3, features, kNibStageK / 2)) return GEMM_ERR_INVALID_ARG;
    if (form.block_rows == 8)
        return launched((dtype == GEMM_F16 ? launch_nibble_f16 : launch_nibble_bf16)(mb, p, prepared, s, overlap(h)));
    if (K > 0 && !encode_map3(h, &mx, A, 1, rows, K, dtype, static_cast<uint32_t>(form.block_rows), 64)) return GEMM_ERR_INVALID_ARG;
    return launched((dtype == GEMM_F16 ? launch_nibble_rows_f16 : launch_nibble_rows_bf16)(mb, mx, p, prepared, s, overlap(h)));
}

}  // extern "C"
