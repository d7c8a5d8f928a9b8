// Rows to the experts and back: assignments sorted by expert, the rows copied
// into that order, and the experts' rows summed with weights, with gradients.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_launch.h"
#include "ptx.cuh"

namespace pts {

namespace {

// ---- sort --------------------------------------------------------------------
//
// A stable counting sort in one launch: one cluster of up to 8 CTAs, CTA c and
// in it warp w taking consecutive stretches of the assignments.  A warp counts
// its stretch per expert (a histogram of its own in shared memory, so the order
// of the counts is that of the assignments and no atomics are needed) and notes
// every assignment's place among the stretch's of its expert in row_of; the
// counts are summed over warps (a warp per expert), CTAs (through distributed
// shared memory) and experts; then the places become rows.  Latency bounds it
// (0.8 MB in and out for 65536 assignments): 8 loads are on their way at a time.
// (One load at a time, the places found a second time, and a thread per expert
// for the sums over warps: 19 us for 65536 over 32 experts, this 10.)
constexpr int kSortMaxWarps = 32;
constexpr int kSortMaxCtas = 8;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cluster_addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// BATCH: assignments per lane at a time
template <int BATCH>
__global__ void __launch_bounds__(32 * kSortMaxWarps, 1)
    expert_sort_kernel(const int32_t *__restrict__ ids, int n, int experts, int32_t *__restrict__ offsets,
                       int32_t *__restrict__ row_of, int32_t *__restrict__ src_of)
{
    extern __shared__ uint32_t sm[];
    const int warps = static_cast<int>(blockDim.x >> 5);
    const int pitch = experts | 1;              // (odd: a warp's lanes read one expert's counts without conflicts)
    uint32_t *hist = sm;                        // [warps][pitch]
    uint32_t *total = sm + warps * pitch;       // [experts], this CTA's counts; then its first row of each expert
    uint32_t *scan = total + experts;           // [warps]
    const int warp = static_cast<int>(threadIdx.x >> 5);
    const int lane = static_cast<int>(lane_id());
    const int ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
    uint32_t *mine = hist + warp * pitch;

    for (int i = threadIdx.x; i < warps * pitch; i += blockDim.x) hist[i] = 0u;
    // (unsigned: a stretch may end within 32 of 2^31)
    const uint32_t count = static_cast<uint32_t>(n), all_warps = static_cast<uint32_t>(ctas * warps);
    const uint32_t per_warp = ((count + all_warps - 1) / all_warps + 31) / 32 * 32;
    const unsigned long long first = static_cast<unsigned long long>(cta * warps + warp) * per_warp;
    const uint32_t lo = first < count ? static_cast<uint32_t>(first) : count;
    const uint32_t hi = count - lo < per_warp ? count : lo + per_warp;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();

    // count, and note each assignment's place (in registers if they hold the
    // whole stretch, else in row_of)
    const bool one_batch = per_warp <= 32 * BATCH;
    int id[BATCH];
    int32_t place[BATCH];
    for (uint32_t b = lo; b < hi; b += 32 * BATCH) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const uint32_t i = b + 32 * k + static_cast<uint32_t>(lane);
            id[k] = i < hi ? ld_global(ids + i) : -1;
            if (id[k] >= experts) id[k] = -1;
        }
        // lanes with the same expert: bit by bit of its number (match.any would
        // say so at once, but takes some 100 cycles of the SM per warp)
        uint32_t peers[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) peers[k] = __ballot_sync(0xffffffffu, id[k] >= 0);
        for (int bit = 1; bit < experts; bit <<= 1)
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const uint32_t set = __ballot_sync(0xffffffffu, id[k] & bit);
                peers[k] &= id[k] & bit ? set : ~set;
            }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            place[k] = -1;
            if (b + 32 * k >= hi) continue;
            const bool held = id[k] >= 0;
            const uint32_t rank = __popc(peers[k] & ((1u << lane) - 1u));
            if (held) place[k] = static_cast<int32_t>(mine[id[k]] + rank);
            __syncwarp();
            if (held && rank == 0) mine[id[k]] = static_cast<uint32_t>(place[k]) + __popc(peers[k]);
            __syncwarp();
            const uint32_t i = b + 32 * k + static_cast<uint32_t>(lane);
            if (i < hi && (!one_batch || !held)) row_of[i] = place[k];
        }
    }
    __syncthreads();
    // exclusive over the warps: a warp per expert, a lane per warp
    for (int e = warp; e < experts; e += warps) {
        const uint32_t c = lane < warps ? hist[lane * pitch + e] : 0u;
        uint32_t incl = c;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, incl, s);
            if (lane >= s) incl += o;
        }
        if (lane < warps) hist[lane * pitch + e] = incl - c;
        if (lane == 31) total[e] = incl;
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    // start of each expert's rows: over all CTAs and the experts before it;
    // `carry` runs over blocks of blockDim.x experts
    uint32_t carry = 0;
    for (int e0 = 0; e0 < experts; e0 += static_cast<int>(blockDim.x)) {
        const int e = e0 + static_cast<int>(threadIdx.x);
        uint32_t all = 0, below = 0;
        if (e < experts) {
            if (ctas > 1) {
                uint32_t v[kSortMaxCtas];
#pragma unroll
                for (int c = 0; c < kSortMaxCtas; ++c)
                    v[c] = c < ctas ? ld_cluster_u32(mapa(smem_u32(total + e), static_cast<uint32_t>(c))) : 0u;
#pragma unroll
                for (int c = 0; c < kSortMaxCtas; ++c) {
                    all += v[c];
                    if (c < cta) below += v[c];
                }
            } else {
                all = total[e];
            }
        }
        uint32_t incl = all;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, incl, s);
            if (lane >= s) incl += o;
        }
        if (lane == 31) scan[warp] = incl;
        // (the counts are read by the whole cluster before they are replaced)
        if (ctas > 1) cluster_sync();
        else __syncthreads();
        uint32_t before = carry, block = 0;
        for (int w = 0; w < warps; ++w) {
            const uint32_t v = scan[w];
            if (w < warp) before += v;
            block += v;
        }
        const uint32_t start = before + incl - all;
        if (e < experts) {
            if (cta == 0) offsets[e] = static_cast<int32_t>(start);
            total[e] = start + below;
        }
        carry += block;
        __syncthreads();
    }
    if (cta == 0 && threadIdx.x == 0) offsets[experts] = static_cast<int32_t>(carry);

    // places to rows
    for (uint32_t b = lo; b < hi; b += 32 * BATCH) {
        if (!one_batch) {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const uint32_t i = b + 32 * k + static_cast<uint32_t>(lane);
                id[k] = i < hi ? ld_global(ids + i) : -1;
                place[k] = i < hi ? row_of[i] : -1;   // (as this lane wrote it)
            }
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (place[k] >= 0) {
                const uint32_t i = b + 32 * k + static_cast<uint32_t>(lane);
                const uint32_t row = static_cast<uint32_t>(place[k]) + mine[id[k]] + total[id[k]];
                row_of[i] = static_cast<int32_t>(row);
                src_of[row] = static_cast<int32_t>(i);
            }
    }
    // rows behind the last held assignment have no source
    for (long long r = static_cast<long long>(carry) + cta * static_cast<long long>(blockDim.x) + threadIdx.x; r < n;
         r += static_cast<long long>(ctas) * blockDim.x)
        src_of[r] = -1;
}

// ---- rows ----------------------------------------------------------------------

template <int KIND>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 t;
        if constexpr (KIND == 0)
            t = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        else
            t = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

template <int KIND>
__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (KIND == 0) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The copy below is bound by the rows' bytes, most of them written (16384 tokens
// of 8 KB, half of their 4 assignments held: 403 MB in 50 us).  Every thread takes
// PIECES 16-byte pieces, kRowThreads apart in the tokens' pieces counted
// through: rows of any length fill whole blocks, and the loads of all its
// pieces (and of 4 assignments of each) are on their way together.
constexpr int kRowThreads = 256;
constexpr int kGatherPieces = 2;

// Token and place in it of piece i (0 .. PIECES - 1) of this thread.
struct Piece {
    long long token;
    int at;
};

template <int PIECES>
__device__ __forceinline__ void pieces_of(int tokens, int chunks, Piece (&q)[PIECES], bool (&there)[PIECES])
{
    const long long first = static_cast<long long>(blockIdx.x) * (kRowThreads * PIECES);
    const long long t0 = first / chunks;
    const uint32_t rest = static_cast<uint32_t>(first - t0 * chunks) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const uint32_t local = rest + i * kRowThreads, over = local / static_cast<uint32_t>(chunks);
        q[i].token = t0 + over;
        q[i].at = static_cast<int>(local - over * chunks);
        there[i] = q[i].token < tokens;
    }
}

// Xs[row_of[t, j]] = X[t]: a row is read once and written top_k times.
__global__ void __launch_bounds__(kRowThreads)
    expert_gather_kernel(const uint4 *__restrict__ x, const int32_t *__restrict__ row_of, uint4 *__restrict__ xs,
                         int tokens, int top_k, int chunks)
{
    pdl_launch_dependents();
    const long long n = static_cast<long long>(tokens) * top_k;
    Piece q[kGatherPieces];
    bool there[kGatherPieces];
    pieces_of(tokens, chunks, q, there);
    pdl_wait();
    uint4 v[kGatherPieces];
#pragma unroll
    for (int i = 0; i < kGatherPieces; ++i)
        if (there[i]) v[i] = ld_global_streamed(x + q[i].token * chunks + q[i].at);
    for (int j0 = 0; j0 < top_k; j0 += 4) {
        int32_t r[kGatherPieces][4];
#pragma unroll
        for (int i = 0; i < kGatherPieces; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r[i][j] = there[i] && j0 + j < top_k ? ld_global(row_of + q[i].token * top_k + j0 + j) : -1;
#pragma unroll
        for (int i = 0; i < kGatherPieces; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r[i][j] >= 0 && r[i][j] < n) xs[static_cast<long long>(r[i][j]) * chunks + q[i].at] = v[i];
    }
}

// Y[t] = sum_j w[t, j] Ys[row_of[t, j]], in 32 bits in the order of j.  A block
// per token, S pieces per thread: a token's rows are looked up once, and S
// pieces of two of its rows are on their way together.  (A thread per piece of
// all tokens, as in the copy, looks rows up for every piece: 24 us where this
// takes 18.4; 104 MB.)
template <int KIND, int S>
__global__ void __launch_bounds__(kRowThreads)
    expert_combine_kernel(const uint4 *__restrict__ ys, const int32_t *__restrict__ row_of, const float *__restrict__ w,
                          uint4 *__restrict__ y, int tokens, int top_k, int chunks)
{
    pdl_launch_dependents();
    pdl_wait();
    const long long t = blockIdx.x;
    const long long n = static_cast<long long>(tokens) * top_k;
    for (int c0 = threadIdx.x; c0 < chunks; c0 += S * blockDim.x) {
        float acc[S][8] = {};
        for (int j = 0; j < top_k; j += 2) {
            int32_t r[2];
            float f[2] = {1.0f, 1.0f};
            uint4 v[2][S];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                r[i] = j + i < top_k ? ld_global(row_of + t * top_k + j + i) : -1;
                if (r[i] >= n) r[i] = -1;
                if (w && j + i < top_k) f[i] = ld_global(w + t * top_k + j + i);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const int c = c0 + s * static_cast<int>(blockDim.x);
                    if (r[i] >= 0 && c < chunks) v[i][s] = ld_global_streamed(ys + static_cast<long long>(r[i]) * chunks + c);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (r[i] >= 0) {
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        float x[8];
                        unpack8<KIND>(v[i][s], x);
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[s][e] = fmaf(f[i], x[e], acc[s][e]);
                    }
                }
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int c = c0 + s * static_cast<int>(blockDim.x);
            if (c < chunks) y[t * chunks + c] = pack8<KIND>(acc[s]);
        }
    }
}

// dYs[row] = w[t, j] dY[t], dw[t, j] = <dY[t], Ys[row]> with row = row_of[t, j];
// dw is 0 where there is no row.  A block per token: dY[t] is read from L1 after
// the first assignment, Ys once, dYs written once; 755 MB in 118 us (8192 tokens
// of 10 KB, 4 assignments), 0.94 of the copy bandwidth.
template <int KIND>
__global__ void __launch_bounds__(256)
    expert_combine_grad_kernel(const uint4 *__restrict__ dy, const uint4 *__restrict__ ys,
                               const int32_t *__restrict__ row_of, const float *__restrict__ w, uint4 *__restrict__ dys,
                               float *__restrict__ dw, int tokens, int top_k, int chunks)
{
    __shared__ float part[8];
    pdl_launch_dependents();
    pdl_wait();
    const long long t = blockIdx.x;
    const long long n = static_cast<long long>(tokens) * top_k;
    for (int j = 0; j < top_k; ++j) {
        const int32_t r = ld_global(row_of + t * top_k + j);
        float dot = 0.0f;
        if (r >= 0 && r < n) {
            const float s = ld_global(w + t * top_k + j);
            for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
                float d[8], f[8];
                unpack8<KIND>(ld_global(dy + t * chunks + c), d);
                unpack8<KIND>(ld_global(ys + static_cast<long long>(r) * chunks + c), f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot = fmaf(d[i], f[i], dot);
                    d[i] *= s;
                }
                dys[static_cast<long long>(r) * chunks + c] = pack8<KIND>(d);
            }
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        if (lane_id() == 0) part[threadIdx.x >> 5] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float all = 0.0f;
            for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) all += part[i];
            dw[t * top_k + j] = all;
        }
        __syncthreads();
    }
}

template <class... P, class... A>
cudaError_t go(void (*kernel)(P...), long long grid, int block, size_t smem, int cluster, cudaStream_t stream,
               bool overlap, A... args)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(block), 1, 1);
    cfg.dynamicSmemBytes = smem;
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
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// blocks of the kernels over all pieces
long long piece_blocks(long long tokens, long long chunks, int pieces)
{
    return (tokens * chunks + kRowThreads * pieces - 1) / (kRowThreads * pieces);
}

// counts per warp and expert (an odd pitch), a row per expert, a sum per warp
size_t sort_smem_bytes(int warps, int experts)
{
    return (static_cast<size_t>(warps) * (experts | 1) + experts + warps) * sizeof(uint32_t);
}

// threads of a block per token: one 16-byte chunk each, up to 256 (a warp where rows are empty: dweights is written)
int row_threads(int chunks) { return chunks >= 256 ? 256 : (chunks < 1 ? 32 : (chunks + 31) / 32 * 32); }

}  // namespace

cudaError_t launch_expert_sort(const int32_t *ids, int64_t n, int experts, int32_t *offsets, int32_t *row_of,
                               int32_t *src_of, bool *prepared, cudaStream_t stream, bool overlap)
{
    // Up to 1024: a warp per 32, the shortest chain of steps (32 over 8 experts 2.6
    // us, with 8 per lane 2.9).  Above 2048 8 CTAs, since a warp's scattered stores
    // to src_of keep its SM busy (8192 over 64: 4.7 us, on one SM 10.0).
    const bool few = n <= 32 * kSortMaxWarps;
    const int ctas = n > 2048 ? kSortMaxCtas : 1, each = few ? 32 : 128;
    const int64_t wanted = (n + each * ctas - 1) / (each * ctas);
    const int warps = wanted < 1 ? 1 : (wanted > kSortMaxWarps ? kSortMaxWarps : static_cast<int>(wanted));
    const size_t smem = sort_smem_bytes(warps, experts);
    const auto kernel = few ? expert_sort_kernel<1> : expert_sort_kernel<8>;
    // (the limit is the function's, on this device, whichever handle or thread launches it: always the most that any call needs)
    if (smem > 48 * 1024 && !prepared[few]) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(sort_smem_bytes(kSortMaxWarps, kMaxExpertsSorted)));
        if (e != cudaSuccess) return e;
        prepared[few] = true;
    }
    return go(kernel, ctas, warps * 32, smem, ctas, stream, overlap, ids, static_cast<int>(n), experts, offsets, row_of,
              src_of);
}

cudaError_t launch_expert_gather(const void *x, const int32_t *row_of, void *xs, int tokens, int top_k, int chunks,
                                 cudaStream_t stream, bool overlap)
{
    return go(expert_gather_kernel, piece_blocks(tokens, chunks, kGatherPieces), kRowThreads, 0, 1, stream, overlap, static_cast<const uint4 *>(x),
              row_of, static_cast<uint4 *>(xs), tokens, top_k, chunks);
}

cudaError_t launch_expert_combine(int kind, const void *ys, const int32_t *row_of, const float *w, void *y, int tokens,
                                  int top_k, int chunks, cudaStream_t stream, bool overlap)
{
    // Pieces per thread: as leave the fewest idle, the most of those (528 pieces
    // of 16 bytes: 3 x 192 threads take 18.4 us, 4 x 160 take 20.3, 2 rounds of
    // 2 x 256 take 21.8).  At most 2 where tokens are few, so that more warps
    // share a token (64 tokens of 8 rows of 8 KB: 3.3 us, with 4 pieces 4.1).
    int best = 1, best_threads = 32;
    long long least = -1;
    for (int s = 1; s <= (tokens <= 512 ? 2 : 4); ++s) {
        int threads = ((chunks + s - 1) / s + 31) / 32 * 32;
        threads = threads > kRowThreads ? kRowThreads : threads;
        const long long slots = (chunks + s * threads - 1) / (s * threads) * static_cast<long long>(s) * threads;
        if (least < 0 || slots <= least) least = slots, best = s, best_threads = threads;
    }
    const auto run = [&](auto kernel) {
        return go(kernel, tokens, best_threads, 0, 1, stream, overlap, static_cast<const uint4 *>(ys), row_of, w,
                  static_cast<uint4 *>(y), tokens, top_k, chunks);
    };
    switch (best) {
    case 1: return run(kind == 0 ? expert_combine_kernel<0, 1> : expert_combine_kernel<1, 1>);
    case 2: return run(kind == 0 ? expert_combine_kernel<0, 2> : expert_combine_kernel<1, 2>);
    case 3: return run(kind == 0 ? expert_combine_kernel<0, 3> : expert_combine_kernel<1, 3>);
    default: return run(kind == 0 ? expert_combine_kernel<0, 4> : expert_combine_kernel<1, 4>);
    }
}

cudaError_t launch_expert_combine_grad(int kind, const void *dy, const void *ys, const int32_t *row_of, const float *w,
                                       void *dys, float *dw, int tokens, int top_k, int chunks, cudaStream_t stream,
                                       bool overlap)
{
    return go(kind == 0 ? expert_combine_grad_kernel<0> : expert_combine_grad_kernel<1>, tokens, row_threads(chunks), 0,
              1, stream, overlap, static_cast<const uint4 *>(dy), static_cast<const uint4 *>(ys), row_of, w,
              static_cast<uint4 *>(dys), dw, tokens, top_k, chunks);
}

}  // namespace pts
