"""The expert layer's operators against plain implementations in 64 bits.

Bounds.  An output of a product is rounded once to a format of unit roundoff u
(2^-11 fp16, 2^-8 bf16), after an fp32 sum of n exact products whose every
addition may be off by 2^-23 of the partial sums' size (the tensor cores may
truncate): |got - ref| <= u |ref| + n 2^-23 sum|a||b| + 2^-25 (half the
smallest fp16 subnormal).  combine sums n = top_k rounded products, so n + 1
takes the place of n; its gradient's rows are one fp32 product rounded twice,
its weights an fp32 sum of dim products.  Where every value is a small integer
all of it is exact and the results must be equal.
"""
import numpy as np
import pytest
import torch

import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu

F16, BF16, E4M3 = pts.GEMM_F16, pts.GEMM_BF16, pts.GEMM_E4M3
TORCH = {F16: torch.float16, BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn}
OUT = {F16: torch.float16, BF16: torch.bfloat16, E4M3: torch.bfloat16}
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
ids16 = {F16: "f16", BF16: "bf16", E4M3: "e4m3"}.get


@pytest.fixture(scope="module")
def h():
    h = pts.gemm_create(0)
    yield h
    st, dev = pts.gemm_check(h)
    pts.gemm_destroy(h)
    assert st == 0, f"device status {dev:#x}"


@pytest.fixture(scope="module", params=[dict(), dict(cta_group=1), dict(cta_group=2), dict(cta_group=1, max_clusters=3),
                                        dict(cta_group=2, max_clusters=2, group_size_m=2)],
                ids=["auto", "single", "pair", "single3", "pair2"])
def hv(request):
    """Handles that take every variant of the products, and several tiles per cluster."""
    h = pts.gemm_create(0, pts.make_opts(**request.param))
    yield h
    st, dev = pts.gemm_check(h)
    pts.gemm_destroy(h)
    assert st == 0, f"device status {dev:#x}"


def rand(shape, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=gen) * scale
    return x.clamp(-448, 448).to(TORCH[dtype]).cuda() if dtype == E4M3 else x.to(TORCH[dtype]).cuda()


def ints(shape, dtype, seed, most=3):
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=gen).float().to(TORCH[dtype]).cuda()


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def close(got, ref, ref_abs, n, what=""):
    u = U[got.dtype]
    bound = u * ref.abs() + n * 2.0 ** -23 * ref_abs + 2.0 ** -25
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(((got.double() - ref).abs() / bound).nan_to_num(9e9).max()))


# ---- sort --------------------------------------------------------------------


def plain_sort(ids, experts):
    flat = ids.reshape(-1).numpy()
    src = np.array([i for e in range(experts) for i in np.nonzero(flat == e)[0]], dtype=np.int64)
    row_of = np.full(flat.size, -1)
    row_of[src] = np.arange(src.size)
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(experts)])])
    return offsets, row_of, np.concatenate([src, np.full(flat.size - src.size, -1)])


@pytest.mark.parametrize("tokens,top_k,experts,lo,hi", [
    (0, 2, 8, 0, 8), (1, 1, 1, 0, 1), (1, 8, 64, 0, 64), (16, 2, 8, 0, 8), (33, 3, 5, -2, 7), (129, 1, 1024, 0, 1024),
    (1000, 4, 100, 0, 100), (777, 6, 33, 0, 1), (500, 2, 8, -5, 0), (500, 2, 8, 8, 100), (4099, 2, 8, 0, 16),
    (20001, 3, 256, -20, 300), (70001, 8, 128, 0, 128), (40000, 2, 1024, 0, 1024)])
def test_sort(h, tokens, top_k, experts, lo, hi):
    gen = torch.Generator().manual_seed(tokens + experts)
    ids = torch.randint(lo, hi, (tokens, top_k), generator=gen, dtype=torch.int32)
    want = plain_sort(ids, experts)
    n = tokens * top_k
    guard = 7
    offsets = torch.full((experts + 1 + guard,), -9, dtype=torch.int32, device="cuda")
    row_of, src_of = (torch.full((n + guard,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    pts.gemm_expert_sort(h, tokens, top_k, experts, ids.cuda(), offsets, row_of, src_of)
    for got, ref, size in ((offsets, want[0], experts + 1), (row_of, want[1], n), (src_of, want[2], n)):
        got = got.cpu().numpy()
        assert (got[:size] == ref).all()
        assert (got[size:] == -9).all()


# ---- rows --------------------------------------------------------------------


def routing(tokens, top_k, seed, held=0.8):
    """row_of with a share of assignments that have no row; the last token has none at all."""
    rng = np.random.default_rng(seed)
    n = tokens * top_k
    keep = rng.random(n) < held
    keep[n - top_k:] = False
    row_of = np.full(n, -1)
    row_of[keep] = rng.permutation(int(keep.sum()))
    return torch.tensor(row_of, dtype=torch.int32, device="cuda").view(tokens, top_k), int(keep.sum())


ROWS = [(1, 1, 8), (2, 3, 264), (37, 2, 4096), (5, 8, 1032), (301, 4, 512), (3, 11, 8200)]


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids=ids16)
@pytest.mark.parametrize("tokens,top_k,dim", [(t, k, -(-d // 16) * 16) for t, k, d in ROWS])
def test_gather(h, tokens, top_k, dim, dtype):
    row_of, held = routing(tokens, top_k, dim)
    X = rand((tokens, dim), dtype, 1)
    Xs = rand((tokens * top_k, dim), dtype, 2)
    want = Xs.clone().view(torch.uint8)
    t, j = (row_of >= 0).nonzero(as_tuple=True)
    want[row_of[t, j].long()] = X.view(torch.uint8)[t]
    pts.gemm_expert_gather(h, tokens, top_k, dim, X, row_of, Xs, dtype)
    assert torch.equal(Xs.view(torch.uint8), want)   # rows without an assignment keep what they held


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids16)
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("tokens,top_k,dim", ROWS)
def test_combine(h, tokens, top_k, dim, weighted, dtype):
    row_of, held = routing(tokens, top_k, dim + 1)
    Ys = rand((tokens * top_k, dim), dtype, 3)
    Ys[held:] = float("nan")   # rows nobody refers to
    w = torch.randn(tokens, top_k, generator=torch.Generator().manual_seed(4)).cuda() if weighted else None
    Y = torch.full((tokens, dim), float("nan"), dtype=TORCH[dtype], device="cuda")
    pts.gemm_expert_combine(h, tokens, top_k, dim, Ys, row_of, w, Y, dtype)
    there = (row_of >= 0)[..., None]
    terms = torch.where(there, Ys.double()[row_of.clamp(min=0).long()], 0.0) * (1.0 if w is None else w.double()[..., None])
    close(Y, terms.sum(1), terms.abs().sum(1), top_k + 1)
    assert (Y[-1] == 0).all()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids16)
@pytest.mark.parametrize("tokens,top_k,dim", ROWS)
def test_combine_grad(h, tokens, top_k, dim, dtype):
    row_of, held = routing(tokens, top_k, dim + 2)
    dY, Ys = rand((tokens, dim), dtype, 5), rand((tokens * top_k, dim), dtype, 6)
    Ys[held:] = float("inf")
    w = torch.randn(tokens, top_k, generator=torch.Generator().manual_seed(7)).cuda()
    dYs = torch.full((tokens * top_k, dim), 5.0, dtype=TORCH[dtype], device="cuda")
    dw = torch.full((tokens, top_k), float("nan"), device="cuda")
    pts.gemm_expert_combine_grad(h, tokens, top_k, dim, dY, Ys, row_of, w, dYs, dw, dtype)
    t, j = (row_of >= 0).nonzero(as_tuple=True)
    r = row_of[t, j].long()
    ref = w.double()[t, j, None] * dY.double()[t]
    close(dYs[r], ref, ref.abs(), 1, "rows")
    assert (dYs[held:] == 5.0).all()
    terms = torch.zeros(tokens, top_k, dim, dtype=torch.float64, device="cuda")
    terms[t, j] = dY.double()[t] * Ys.double()[r]
    close(dw, terms.sum(2), terms.abs().sum(2), dim, "weights")
    assert (dw[row_of < 0] == 0).all()


def test_combine_grad_of_empty_rows(h):
    row_of = torch.tensor([[0, -1], [1, 2]], dtype=torch.int32, device="cuda")
    w, dw = torch.ones(2, 2, device="cuda"), torch.full((2, 2), float("nan"), device="cuda")
    pts.gemm_expert_combine_grad(h, 2, 2, 0, None, None, row_of, w, None, dw, F16)
    assert (dw == 0).all()


def test_row_of_outside_the_rows_counts_as_none(h):
    tokens, top_k, dim = 4, 2, 64
    row_of = torch.tensor([[0, 8], [1 << 30, -7], [2, 3], [-1 << 31, 7]], dtype=torch.int32, device="cuda")
    fixed = torch.where((row_of >= 0) & (row_of < 8), row_of, -1)
    Ys, w = rand((8, dim), F16, 8), torch.ones(tokens, top_k, device="cuda")
    got = []
    for ro in (row_of, fixed):
        Y, dYs = torch.zeros(tokens, dim, dtype=torch.float16, device="cuda"), torch.zeros_like(Ys)
        dw, Xs = torch.zeros(tokens, top_k, device="cuda"), torch.zeros_like(Ys)
        pts.gemm_expert_combine(h, tokens, top_k, dim, Ys, ro, w, Y, F16)
        pts.gemm_expert_combine_grad(h, tokens, top_k, dim, Ys[:tokens], Ys, ro, w, dYs, dw, F16)
        pts.gemm_expert_gather(h, tokens, top_k, dim, Ys[:tokens], ro, Xs, F16)
        got.append((Y, dYs, dw, Xs))
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ---- products ----------------------------------------------------------------

# rows per expert, rows behind the last, N, K
SHAPES = [
    ([1], 0, 8, 16), ([5, 0, 3], 2, 264, 208), ([0, 0, 40, 1, 0], 0, 128, 64), ([16, 17, 15, 64, 65], 5, 392, 1008),
    ([300, 0, 1, 257, 128], 31, 520, 144), ([1025, 63], 0, 256, 336), ([3] * 45, 0, 144, 80), ([700], 0, 1000, 272),
]


def run_fwd(h, counts, spare, N, K, dtype, make=rand, poison=True):
    rows, E = sum(counts) + spare, len(counts)
    A, B = make((rows, K), dtype, 11), make((E, N, K), dtype, 12)
    if poison and dtype != E4M3:
        A[sum(counts):] = float("nan")
    C = torch.full((rows, N), 7.0, dtype=OUT[dtype], device="cuda")
    sa, sb = (2.0, 0.25) if dtype == E4M3 else (1.0, 1.0)
    pts.gemm_run_experts(h, rows, E, N, K, A, B, offsets_of(counts), C, dtype, sa, sb)
    return A, B, C, sa * sb


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids=ids16)
@pytest.mark.parametrize("counts,spare,N,K", SHAPES)
def test_forward(hv, counts, spare, N, K, dtype):
    A, B, C, scale = run_fwd(hv, counts, spare, N, K, dtype)
    off = 0
    for e, c in enumerate(counts):
        a, b = A[off:off + c].double(), B[e].double()
        close(C[off:off + c], a @ b.T / scale, a.abs() @ b.abs().T / scale, K, (e, c))
        off += c
    assert (C[off:] == 7.0).all()   # rows of no expert are not written


# few tiles and a long contraction: CTAs that share it
FEW = [([1], 0, 128, 1024), ([1], 0, 8, 4112), ([0, 0, 1, 0], 0, 2056, 2064), ([3, 0, 0, 2], 4, 136, 8208), ([0, 1], 1, 8192, 1536),
       ([32], 0, 264, 1040), ([20, 9, 0], 3, 1000, 2000), ([0, 0, 64], 0, 512, 1104), ([0, 0, 65], 31, 72, 1504),
       ([0] * 40 + [1, 0, 2], 0, 520, 1072), ([7, 1, 1, 7], 0, 1024, 4096), ([0, 0], 4, 256, 2048)]


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids=ids16)
@pytest.mark.parametrize("counts,spare,N,K", FEW)
def test_forward_of_few_tiles(hv, counts, spare, N, K, dtype):
    test_forward(hv, counts, spare, N, K, dtype)


def test_few_tiles_exact_and_their_values_stay(h):
    """Small integers are exact however the contraction is shared; an infinity stays with its row and feature."""
    A, B = ints((6, 4096), F16, 4, 1), ints((5, 264, 4096), F16, 5, 1)
    off = offsets_of([2, 0, 3, 0, 1])
    C = torch.full((6, 264), 7.0, dtype=torch.float16, device="cuda")
    pts.gemm_run_experts(h, 6, 5, 264, 4096, A, B, off, C, F16)
    want = torch.cat([A[:2].double() @ B[0].double().T, A[2:5].double() @ B[2].double().T, A[5:].double() @ B[4].double().T])
    assert torch.equal(C.double(), want)
    A[3, 4000], B[1] = float("inf"), float("nan")
    B[4, 17, 3] = float("nan")
    pts.gemm_run_experts(h, 6, 5, 264, 4096, A, B, off, C, F16)
    bad = ~torch.isfinite(C)
    bad[3] &= B[2, :, 4000] == 0   # inf * 0 is NaN there, infinite elsewhere: all of row 3 may be
    keep = torch.ones_like(bad)
    keep[3], keep[5, 17] = False, False
    assert not bad[keep].any() and torch.equal(C.double()[keep], want[keep]) and torch.isnan(C[5, 17])


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids16)
@pytest.mark.parametrize("counts,spare,N,K", SHAPES)
def test_dgrad(hv, counts, spare, N, K, dtype):
    rows, E = sum(counts) + spare, len(counts)
    dC, B = rand((rows, N), dtype, 13), rand((E, N, K), dtype, 14)
    dC[sum(counts):] = float("nan")
    dA = torch.full((rows, K), 7.0, dtype=TORCH[dtype], device="cuda")
    pts.gemm_run_experts_dgrad(hv, rows, E, N, K, dC, B, offsets_of(counts), dA, dtype)
    off = 0
    for e, c in enumerate(counts):
        d, b = dC[off:off + c].double(), B[e].double()
        close(dA[off:off + c], d @ b, d.abs() @ b.abs(), N, (e, c))
        off += c
    assert (dA[off:] == 7.0).all()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids16)
@pytest.mark.parametrize("counts,spare,N,K", SHAPES)
def test_wgrad(hv, counts, spare, N, K, dtype):
    rows, E = sum(counts) + spare, len(counts)
    dC, A = rand((rows, N), dtype, 15), rand((rows, K), dtype, 16)
    dC[sum(counts):] = float("nan")
    A[sum(counts):] = float("nan")
    dB = torch.full((E, N, K), float("nan"), dtype=TORCH[dtype], device="cuda")
    pts.gemm_run_experts_wgrad(hv, rows, E, N, K, dC, A, offsets_of(counts), dB, dtype)
    off = 0
    for e, c in enumerate(counts):
        d, a = dC[off:off + c].double(), A[off:off + c].double()
        close(dB[e], d.T @ a, d.abs().T @ a.abs(), c, (e, c))
        off += c


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_values_of_one_expert_stay_with_it(hv, poison):
    counts, N, K = [20, 7, 64, 33], 136, 200
    rows, E = sum(counts), len(counts)
    A, B, dC = ints((rows, K), F16, 1), ints((E, N, K), F16, 2), ints((rows, N), F16, 3)
    off = offsets_of(counts)
    C, dA = torch.empty(rows, N, dtype=torch.float16, device="cuda"), torch.empty_like(A)
    dB = torch.empty_like(B)
    A[20:27] = poison      # expert 1's rows, and its weights
    dC[20:27] = poison
    B[1] = poison
    pts.gemm_run_experts(hv, rows, E, N, K, A, B, off, C, F16)
    pts.gemm_run_experts_dgrad(hv, rows, E, N, K, dC, B, off, dA, F16)
    pts.gemm_run_experts_wgrad(hv, rows, E, N, K, dC, A, off, dB, F16)
    o = [0] + list(np.cumsum(counts))
    for e in (0, 2, 3):
        a, d, b = A[o[e]:o[e + 1]].double(), dC[o[e]:o[e + 1]].double(), B[e].double()
        assert torch.equal(C[o[e]:o[e + 1]].double(), a @ b.T)
        assert torch.equal(dA[o[e]:o[e + 1]].double(), d @ b)
        assert torch.equal(dB[e].double(), d.T @ a)


def test_no_contraction_writes_zeros(h):
    counts, rows = [3, 0, 70], 75
    C = torch.full((rows, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    pts.gemm_run_experts(h, rows, 3, 40, 0, None, None, offsets_of(counts), C, BF16)
    assert (C[:73] == 0).all() and (C[73:] == 7).all()
    dB = torch.full((2, 16, 24), 7.0, dtype=torch.bfloat16, device="cuda")
    pts.gemm_run_experts_wgrad(h, 0, 2, 16, 24, None, None, offsets_of([0, 0]), dB, BF16)
    assert (dB == 0).all()


def test_offsets_outside_the_rows_stay_inside(h):
    rows, E, N, K = 100, 4, 64, 64
    A, B = ints((rows, K), F16, 4), ints((E, N, K), F16, 5)
    off = torch.tensor([-50, 30, 20, 1 << 30, 1 << 30], dtype=torch.int32, device="cuda")   # 30, none, 80, none
    C = torch.full((rows + 4, N), 7.0, dtype=torch.float16, device="cuda")
    pts.gemm_run_experts(h, rows, E, N, K, A, B, off, C, F16)
    a, b = A.double(), B.double()
    assert torch.equal(C[30:rows].double(), a[30:] @ b[2].T)
    assert torch.equal(C[:20].double(), a[:20] @ b[0].T)
    # rows 20..29 are in two experts' ranges: each element is one of the two's
    both = C[20:30].double()
    assert ((both == a[20:30] @ b[0].T) | (both == a[20:30] @ b[2].T)).all()
    assert (C[rows:] == 7).all()


@pytest.mark.parametrize("counts,N,K", [([5, 0, 18, 33], 24, 40), ([130, 1], 72, 136)])
def test_gradients_against_differences(hv, counts, N, K):
    """Small integers: L = sum(G * C) is bilinear and everything is exact, so differences of L equal the gradient."""
    rows, E = sum(counts), len(counts)
    A, B, G = ints((rows, K), F16, 21, 1), ints((E, N, K), F16, 22, 1), ints((rows, N), F16, 23, 1)
    V, W = ints((rows, K), F16, 24, 1), ints((E, N, K), F16, 25, 1)
    off = offsets_of(counts)

    def loss(a, b):
        C = torch.zeros(rows, N, dtype=torch.float16, device="cuda")
        pts.gemm_run_experts(hv, rows, E, N, K, a, b, off, C, F16)
        return float((C.double() * G.double()).sum())

    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    pts.gemm_run_experts_dgrad(hv, rows, E, N, K, G, B, off, dA, F16)
    pts.gemm_run_experts_wgrad(hv, rows, E, N, K, G, A, off, dB, F16)
    assert (loss(A + V, B) - loss(A - V, B)) / 2 == float((dA.double() * V.double()).sum())
    assert (loss(A, B + W) - loss(A, B - W)) / 2 == float((dB.double() * W.double()).sum())


def test_combine_gradient_against_differences(h):
    tokens, top_k, dim = 19, 3, 72
    row_of, held = routing(tokens, top_k, 5)
    Ys, V, G = (ints((tokens * top_k, dim), F16, s) for s in (31, 32, 33))
    G = G[:tokens].contiguous()
    w = torch.randint(-3, 4, (tokens, top_k), generator=torch.Generator().manual_seed(34)).float().cuda()
    dw_ = torch.randint(-3, 4, (tokens, top_k), generator=torch.Generator().manual_seed(35)).float().cuda()
    V[held:] = 0

    def loss(y, ww):
        Y = torch.zeros(tokens, dim, dtype=torch.float16, device="cuda")
        pts.gemm_expert_combine(h, tokens, top_k, dim, y, row_of, ww, Y, F16)
        return float((Y.double() * G.double()).sum())

    dYs, dw = torch.zeros_like(Ys), torch.zeros_like(w)
    pts.gemm_expert_combine_grad(h, tokens, top_k, dim, G, Ys, row_of, w, dYs, dw, F16)
    assert (loss(Ys + V, w) - loss(Ys - V, w)) / 2 == float((dYs.double() * V.double()).sum())
    assert (loss(Ys, w + dw_) - loss(Ys, w - dw_)) / 2 == float((dw.double() * dw_.double()).sum())


# ---- 4-bit weights -------------------------------------------------------------

NIBBLE = [  # rows per expert, N, K, group
    ([1], 8, 32, 32), ([1], 264, 4096, 128), ([7], 24, 96, 64), ([8], 1000, 544, 32), ([9], 40, 1056, 128),
    ([33], 72, 224, 64), ([100], 16, 160, 128), ([1, 0, 2, 17, 0], 136, 352, 32), ([2] * 70, 48, 288, 64),
    ([1], 4096, 8224, 64),
]


def packed(E, N, K, group, dtype, zeros, seed, scale=None):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 16, (E, N, K), generator=gen, dtype=torch.uint8)
    groups = -(-K // group)
    s = torch.rand(E, N, groups, generator=gen) * 0.02 + 0.005 if scale is None else torch.full((E, N, groups), scale)
    s = s.to(TORCH[dtype])
    z = torch.randint(0, 16, (E, N, groups), generator=gen, dtype=torch.uint8) if zeros else None
    at = torch.arange(K) // group
    w = (q.double() - (8.0 if z is None else z.double()[..., at])) * s.double()[..., at]
    b = q.view(E, N, K // 2, 2)
    return (b[..., 0] | (b[..., 1] << 4)).contiguous().cuda(), s.cuda(), None if z is None else z.cuda(), w.cuda()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids16)
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("counts,N,K,group", NIBBLE)
def test_nibble(h, counts, N, K, group, zeros, dtype):
    E, spare = len(counts), 0 if len(counts) == 1 else 3
    rows = sum(counts) + spare
    B, s, z, w = packed(E, N, K, group, dtype, zeros, 41)
    A = rand((rows, K), dtype, 42)
    A[sum(counts):] = float("nan")
    C = torch.full((rows, N), 7.0, dtype=TORCH[dtype], device="cuda")
    pts.gemm_run_nibble(h, rows, E, N, K, group, A, B, s, z, None if E == 1 else offsets_of(counts), C, dtype)
    off = 0
    for e, c in enumerate(counts):
        a = A[off:off + c].double()
        # a scaled weight may itself be rounded in fp32: one more rounding per product
        close(C[off:off + c], a @ w[e].T, a.abs() @ w[e].abs().T, K + 1, (e, c))
        off += c
    assert (C[off:] == 7.0).all()


NIBBLE_MORE = [  # above 8 rows per expert
    ([9], 8, 32, 32), ([16], 264, 4096, 128), ([17], 24, 96, 64), ([12], 1000, 544, 32), ([31], 40, 1056, 128),
    ([20, 0, 9, 40], 72, 224, 64), ([33, 1, 16, 17, 0], 136, 352, 32), ([18] * 33, 48, 160, 128), ([24], 4096, 8224, 64),
    ([11], 2432, 16384, 32), ([25, 8], 520, 12320, 128), ([15], 8, 128, 128), ([10, 10, 10], 16, 8192, 32),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids16)
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("counts,N,K,group", NIBBLE_MORE)
def test_nibble_of_more_rows(h, counts, N, K, group, zeros, dtype):
    test_nibble(h, counts, N, K, group, zeros, dtype)


NIBBLE_MANY = [  # enough rows that the weights are expanded for 32 or 64 of them at a time; odd sizes on both sides
    ([33], 4104, 4128, 32), ([64], 4096, 8192, 64), ([24], 8200, 8224, 128), ([129], 1000, 4064, 64), ([250], 136, 8160, 32),
    ([500], 520, 2080, 128), ([140, 0, 77, 164, 33], 1032, 2080, 32), ([65, 66, 1, 0, 200], 2056, 1056, 64),
    ([40] * 33, 264, 1184, 128), ([70, 3] * 20, 1096, 544, 32), ([400, 30], 2048, 96, 64), ([31, 33] * 16, 1032, 1536, 64),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids16)
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("counts,N,K,group", NIBBLE_MANY)
def test_nibble_of_many_rows(h, counts, N, K, group, zeros, dtype):
    test_nibble(h, counts, N, K, group, zeros, dtype)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_nibble_of_many_rows_exact(h, group):
    """Every code: row r takes weight r of its 512, times a power of two, so each result is one weight, exactly."""
    rows, N, K = 512, 2056, 512
    B, s, z, w = packed(1, N, K, group, BF16, True, 43, scale=0.5)
    A = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    A[torch.arange(rows), torch.arange(rows)] = 2.0
    C = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    pts.gemm_run_nibble(h, rows, 1, N, K, group, A, B, s, z, None, C, BF16)
    assert torch.equal(C.double(), 2.0 * w[0].T)


def test_nibble_of_many_rows_keeps_infinities(h):
    """An infinity in one row reaches that row alone, an infinite scale its feature alone."""
    rows, N, K = 300, 1032, 1056
    B, s, z, w = packed(1, N, K, 64, F16, False, 44)
    A = rand((rows, K), F16, 45)
    A[10, 7] = float("inf")
    C = torch.empty(rows, N, dtype=torch.float16, device="cuda")
    pts.gemm_run_nibble(h, rows, 1, N, K, 64, A, B, s, z, None, C, F16)
    others = [i for i in range(rows) if i != 10]
    assert torch.isfinite(C[others]).all() and not torch.isfinite(C[10][w[0, :, 7] != 0]).any()
    A, B, s = torch.ones(rows, K).half().cuda(), torch.full_like(B, 0x99), torch.ones_like(s)
    s[0, 5, -1] = float("inf")
    pts.gemm_run_nibble(h, rows, 1, N, K, 64, A, B, s, z, None, C, F16)
    want = torch.full_like(C, float(K))
    want[:, 5] = float("inf")
    assert torch.equal(C, want)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids16)
def test_nibble_of_more_rows_exact(h, dtype):
    """Every code, every position, rows on both sides of the eighth."""
    rows, N, K, group = 11, 16, 128, 32
    B, s, z, w = packed(1, N, K, group, dtype, True, 43, scale=0.5)
    A = torch.zeros(rows, K, dtype=TORCH[dtype], device="cuda")
    C = torch.empty(rows, N, dtype=TORCH[dtype], device="cuda")
    for k in range(K):
        A.zero_()
        A[2, k], A[9, k] = 2.0, -1.0
        pts.gemm_run_nibble(h, rows, 1, N, K, group, A, B, s, z, None, C, dtype)
        want = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
        want[2], want[9] = 2.0 * w[0, :, k], -w[0, :, k]
        assert torch.equal(C.double(), want), k


def test_nibble_rows_keep_their_infinities_above_eight(h):
    B, s, z, w = packed(1, 24, 64, 32, F16, False, 44)
    A = rand((21, 64), F16, 45)
    A[10, 7] = float("inf")
    C = torch.empty(21, 24, dtype=torch.float16, device="cuda")
    pts.gemm_run_nibble(h, 21, 1, 24, 64, 32, A, B, s, z, None, C, F16)
    others = [i for i in range(21) if i != 10]
    assert torch.isfinite(C[others]).all() and not torch.isfinite(C[10][w[0, :, 7] != 0]).any()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids16)
def test_nibble_exact(h, dtype):
    """Every code, every position: small integers and a power of two are exact."""
    rows, N, K, group = 3, 16, 128, 32
    B, s, z, w = packed(1, N, K, group, dtype, True, 43, scale=0.5)
    A = torch.zeros(rows, K, dtype=TORCH[dtype], device="cuda")
    C = torch.empty(rows, N, dtype=TORCH[dtype], device="cuda")
    for k in range(K):
        A.zero_()
        A[1, k] = 2.0
        pts.gemm_run_nibble(h, rows, 1, N, K, group, A, B, s, z, None, C, dtype)
        want = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
        want[1] = 2.0 * w[0, :, k]
        assert torch.equal(C.double(), want), k


def test_nibble_rows_keep_their_infinities(h):
    """An infinity in one row reaches that row alone."""
    B, s, z, w = packed(1, 24, 64, 32, F16, False, 44)
    A = rand((5, 64), F16, 45)
    A[2, 7] = float("inf")
    C = torch.empty(5, 24, dtype=torch.float16, device="cuda")
    pts.gemm_run_nibble(h, 5, 1, 24, 64, 32, A, B, s, z, None, C, F16)
    assert torch.isfinite(C[[0, 1, 3, 4]]).all() and not torch.isfinite(C[2][w[0, :, 7] != 0]).any()


@pytest.mark.parametrize("K,group", [(32, 32), (96, 64), (256, 128), (320, 32)])
def test_nibble_scales_keep_their_infinities(h, K, group):
    """An infinite scale of the last group, which a unit of the contraction may not be full of, gives infinities (all
    its products are positive) and reaches its feature alone."""
    A, B = torch.ones(2, K).half().cuda(), torch.full((1, 16, K // 2), 0x99, dtype=torch.uint8, device="cuda")
    s = torch.ones(1, 16, -(-K // group)).half()
    s[0, 5, -1] = float("inf")
    C = torch.empty(2, 16, dtype=torch.float16, device="cuda")
    pts.gemm_run_nibble(h, 2, 1, 16, K, group, A, B, s.cuda(), None, None, C, F16)
    want = torch.full((2, 16), float(K)).half().cuda()
    want[:, 5] = float("inf")
    assert torch.equal(C, want)


@pytest.mark.parametrize("rows,E,N", [(64, 64, 40), (1 << 15, 1024, 16400)])
def test_nibble_offsets_that_go_back_and_forth_stay_inside(h, rows, E, N):
    """Every other expert claims all rows (in the larger case more pieces of work than 32 bits count); every expert's
    weights are ones, so that each row is its sum whoever multiplies it."""
    K = 32
    A = ints((rows, K), F16, 47)
    B, s = torch.full((E, N, K // 2), 0x99, dtype=torch.uint8, device="cuda"), torch.ones(E, N, 1).half().cuda()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1::2] = rows
    C = torch.full((rows + 8, N), 7.0, dtype=torch.float16, device="cuda")
    pts.gemm_run_nibble(h, rows, E, N, K, 32, A, B, s, None, off, C, F16)
    assert (C[:rows] == A.sum(1, dtype=torch.float32).half()[:, None]).all() and (C[rows:] == 7).all()


# ---- streams, graphs, refusals -------------------------------------------------


def test_a_layer_in_a_graph_follows_new_routing(h):
    """Sort, gather, product and combine captured once; replayed with other ids the layer goes where they say."""
    T, k, E, D, N = 50, 2, 6, 64, 72
    s = torch.cuda.Stream()
    X, B = ints((T, D), F16, 51, 2), ints((E, N, D), F16, 52, 1)
    w = torch.ones(T, k, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    off, row_of = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
    src = torch.zeros(T * k, dtype=torch.int32, device="cuda")
    Xs = torch.zeros(T * k, D, dtype=torch.float16, device="cuda")
    Cs, Y = torch.zeros(T * k, N, dtype=torch.float16, device="cuda"), torch.zeros(T, N, dtype=torch.float16, device="cuda")

    def layer():
        pts.gemm_expert_sort(h, T, k, E, ids, off, row_of, src, stream=s)
        pts.gemm_expert_gather(h, T, k, D, X, row_of, Xs, F16, stream=s)
        pts.gemm_run_experts(h, T * k, E, N, D, Xs, B, off, Cs, F16, stream=s)
        pts.gemm_expert_combine(h, T, k, N, Cs, row_of, w, Y, F16, stream=s)

    torch.cuda.synchronize()
    layer()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer()
    for seed in (1, 2):
        new = torch.randint(-1, E + 1, (T, k), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()
        ids.copy_(new)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        for t in range(T):
            for j in range(k):
                e = int(new[t, j])
                if 0 <= e < E:
                    want[t] += B[e].double() @ X[t].double()
        assert torch.equal(Y.double(), want)


def test_refusals(h):
    i32 = torch.zeros(64, dtype=torch.int32, device="cuda")
    f32 = torch.zeros(64, device="cuda")
    x = torch.zeros(4096, dtype=torch.float16, device="cuda")
    u8 = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    bad = [
        lambda: pts.gemm_expert_sort(h, 4, 0, 8, i32, i32, i32, i32),            # top_k
        lambda: pts.gemm_expert_sort(h, -1, 2, 8, i32, i32, i32, i32),
        lambda: pts.gemm_expert_sort(h, 4, 2, 0, i32, i32, i32, i32),            # experts
        lambda: pts.gemm_expert_sort(h, 4, 2, 1025, i32.data_ptr(), i32.data_ptr(), i32, i32),
        lambda: pts.gemm_expert_sort(h, 4, 2, 8, None, i32, i32, i32),           # no ids
        lambda: pts.gemm_expert_sort(h, 4, 2, 8, i32.long(), i32, i32, i32),     # type
        lambda: pts.gemm_expert_sort(h, 64, 2, 8, i32, i32, i32, i32),           # too small
        lambda: pts.gemm_expert_sort(h, 1 << 20, 1 << 12, 8, 16, 16, 16, 16),    # tokens * top_k
        lambda: pts.gemm_expert_sort(None, 4, 2, 8, i32, i32, i32, i32),         # no handle
        lambda: pts.gemm_expert_gather(h, 4, 2, 12, x, i32, x, F16),             # 24-byte rows
        lambda: pts.gemm_expert_gather(h, 4, 2, 16, x, None, x, F16),
        lambda: pts.gemm_expert_gather(h, 4, 2, 16, x.data_ptr() + 2, i32, x, F16),   # alignment
        lambda: pts.gemm_expert_gather(h, 4, 2, 16, x[::2], i32, x, F16),        # strided
        lambda: pts.gemm_expert_gather(h, 4, 2, 16, x.cpu(), i32, x, F16),       # host memory
        lambda: pts.gemm_expert_gather(h, 4, 2, 16, x, i32, x, 3),
        lambda: pts.gemm_expert_combine(h, 4, 2, 16, x, i32, f32, x, E4M3),
        lambda: pts.gemm_expert_combine(h, 4, 2, 16, x, i32, f32.half(), x, F16),
        lambda: pts.gemm_expert_combine_grad(h, 4, 2, 16, x, x, i32, None, x, f32, F16),
        lambda: pts.gemm_run_experts(h, 4, 2, 8, 12, x, x, i32, x, F16),
        lambda: pts.gemm_run_experts(h, 4, 2, 12, 8, x, x, i32, x, F16),
        lambda: pts.gemm_run_experts(h, 4, 2, 8, 8, x, x, None, x, F16),
        lambda: pts.gemm_run_experts(h, 4, 2, 8, 16, 1024, 1024, i32, 1024, E4M3, 0.0, 1.0),
        lambda: pts.gemm_run_experts(h, 4, 2, 8, 16, 1024, 1024, i32, 1024, E4M3, 1.0, float("inf")),
        lambda: pts.gemm_run_experts(h, 4, -2, 8, 8, x, x, i32, x, F16),
        lambda: pts.gemm_run_experts_dgrad(h, 4, 2, 8, 8, x, None, i32, x, F16),
        lambda: pts.gemm_run_experts_wgrad(h, 4, 2, 8, 8, x, x, i32, None, F16),
        lambda: pts.gemm_run_experts_wgrad(h, 4, 2, 8, 8, x.data_ptr(), x.data_ptr(), i32, x.data_ptr(), E4M3),
        lambda: pts.gemm_run_nibble(h, 1, 1, 8, 32, 16, x, u8, x, None, None, x, F16),      # group
        lambda: pts.gemm_run_nibble(h, 1, 1, 8, 48, 32, x, u8, x, None, None, x, F16),      # K
        lambda: pts.gemm_run_nibble(h, 1, 1, 12, 32, 32, x, u8, x, None, None, x, F16),     # N
        lambda: pts.gemm_run_nibble(h, 1, 2, 8, 32, 32, x, u8, x, None, None, x, F16),      # offsets
        lambda: pts.gemm_run_nibble(h, 1, 1, 8, 32, 32, x, u8, x.float(), None, None, x, F16),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(pts.GemmError) as err:
            call()
        assert err.value.status == 1, i
    st, dev = pts.gemm_check(h)
    assert st == 0 and dev == 0


@pytest.mark.parametrize("which", range(4), ids=["rows", "experts", "N", "K"])
def test_sizes_whose_counts_would_pass_32_bits_are_refused(h, which):
    size = [16, 2, 16, 32]
    size[which] = (1 << 31) - 32   # (a multiple of 32, above the limit)
    for call in (lambda: pts.gemm_run_experts(h, *size, 1024, 1024, 1024, 1024, BF16),
                 lambda: pts.gemm_run_experts_dgrad(h, *size, 1024, 1024, 1024, 1024, BF16),
                 lambda: pts.gemm_run_experts_wgrad(h, *size, 1024, 1024, 1024, 1024, BF16),
                 lambda: pts.gemm_run_nibble(h, *size, 32, 1024, 1024, 1024, None, 1024, 1024, BF16)):
        with pytest.raises(pts.GemmError) as err:
            call()
        assert err.value.status == 1


# ---- the layer of the example, forwards, backwards and in 4 bits ------------------


def test_example_layer():
    """Forward and gradients of examples/expert_layer.py against the same layer written out in 64 bits.

    Each 16-bit tensor between two operators is rounded to 2^-8 of itself and
    a product of n terms keeps that relative to the root of its sum of squares;
    4 roundings (6 backwards) in a row are below 2^-5 of the result's norm."""
    import os
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    import expert_layer as ex

    T, D, H, E, k = 100, 72, 136, 5, 2
    layer = _layer_without_4_bits(ex, D, H, E, k)
    gen = torch.Generator().manual_seed(9)
    x = torch.randn(T, D, generator=gen).to(torch.bfloat16).cuda()
    ids = torch.randint(-1, E, (T, k), generator=gen, dtype=torch.int32).cuda()
    w = torch.rand(T, k, generator=gen).cuda()
    dy = torch.randn(T, D, generator=gen).to(torch.bfloat16).cuda()
    y, saved = layer.forward(x, ids, w)
    got = layer.backward(dy, saved)

    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    up, down = layer.up.double().requires_grad_(), layer.down.double().requires_grad_()
    y64 = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e >= 0:
                y64[t] = y64[t] + w64[t, j] * (down[e] @ (up[e] @ x64[t]).relu().square())
    want = torch.autograd.grad((y64 * dy.double()).sum(), (x64, w64, up, down))
    for a, b in zip((y, *got), (y64.detach(), *want)):
        assert float((a.double() - b).norm()) <= 2.0 ** -5 * float(b.norm())
    st, dev = pts.gemm_check(layer.h)
    layer.close()
    assert st == 0, f"device status {dev:#x}"


def _layer_without_4_bits(ex, D, H, E, k):
    quantise, ex.quantise = ex.quantise, lambda w, group: None   # (sizes that are no multiple of a group)
    try:
        return ex.ExpertLayer(D, H, E, k)
    finally:
        ex.quantise = quantise


def test_example_decode():
    """The 4-bit forward equals the 16-bit one with the matrices that the codes stand for."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import expert_layer as ex
    T, D, H, E, k = 5, 128, 256, 6, 3
    layer = ex.ExpertLayer(D, H, E, k, seed=2)
    for name in ("up", "down"):
        q, s = getattr(layer, name + "4")
        code = torch.stack([q & 15, q >> 4], -1).flatten(-2).double() - 8.0
        setattr(layer, name, (code * s.double().repeat_interleave(128, -1)))
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(T, D, generator=gen).to(torch.bfloat16).cuda()
    ids = torch.randint(0, E + 1, (T, k), generator=gen, dtype=torch.int32).cuda()
    w = torch.rand(T, k, generator=gen).cuda()
    y = layer.decode(x, ids, w)
    want = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e < E:
                want[t] += w[t, j].double() * (layer.down[e] @ (layer.up[e] @ x[t].double()).relu().square())
    layer.close()
    assert float((y.double() - want).norm()) <= 2.0 ** -5 * float(want.norm())


@pytest.mark.parametrize("tokens,dim", [(8, 64), (64, 128), (700, 256)])
def test_back_to_back_layers_see_their_own_routing(h, tokens, dim):
    """Layers queued one after another on the same buffers, each with other ids, its kernels started while the ones
    before still run: every one must follow its own offsets and rows.  Expert e multiplies by e + 1, exactly."""
    E, k, n = 6, 2, 60
    gen = torch.Generator().manual_seed(tokens)
    x = ints((tokens, dim), F16, 61, 3)
    B = torch.stack([torch.eye(dim) * (e + 1) for e in range(E)]).half().cuda()
    q = torch.zeros(E, dim, dim, dtype=torch.uint8)
    for e in range(E):
        q[e] = 8 + torch.eye(dim, dtype=torch.uint8) * (e + 1)
    q = q.view(E, dim, dim // 2, 2)
    B4, s4 = (q[..., 0] | (q[..., 1] << 4)).contiguous().cuda(), torch.ones(E, dim, dim // 32).half().cuda()
    ids = torch.randint(-1, E, (n, tokens, k), generator=gen, dtype=torch.int32).cuda()
    w = torch.ones(tokens, k, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    off, row_of, src = i32(E + 1), i32(tokens, k), i32(tokens * k)
    xs, c = (torch.zeros(tokens * k, dim, dtype=torch.float16, device="cuda") for _ in range(2))
    y = torch.zeros(n, 2, tokens, dim, dtype=torch.float16, device="cuda")
    dw = torch.zeros(n, tokens, k, device="cuda")
    torch.cuda.synchronize()
    for i in range(n):
        pts.gemm_expert_sort(h, tokens, k, E, ids[i], off, row_of, src)
        pts.gemm_expert_gather(h, tokens, k, dim, x, row_of, xs, F16)
        pts.gemm_run_experts(h, tokens * k, E, dim, dim, xs, B, off, c, F16)
        pts.gemm_expert_combine(h, tokens, k, dim, c, row_of, w, y[i, 0], F16)
        pts.gemm_run_nibble(h, tokens * k, E, dim, dim, 32, xs, B4, s4, None, off, c, F16)
        pts.gemm_expert_combine(h, tokens, k, dim, c, row_of, w, y[i, 1], F16)
        pts.gemm_expert_combine_grad(h, tokens, k, dim, x, c, row_of, w, xs, dw[i], F16)
    torch.cuda.synchronize()
    factor = torch.where(ids >= 0, ids + 1, 0)
    assert torch.equal(y.double(), (factor.sum(2).double()[..., None] * x.double())[:, None].expand_as(y))
    assert torch.equal(dw.double(), factor.double() * (x.double() ** 2).sum(1)[None, :, None])


@pytest.mark.parametrize("tokens,dim", [(8, 64), (64, 256), (1000, 128)])
def test_a_reader_sees_what_the_call_before_it_wrote(h, tokens, dim):
    """Pairs of calls queued over and over, the first writing what the second reads, on the same addresses and with
    other values each time: a call may start while the one before the previous still reads the old values."""
    E, k, n = 5, 2, 40
    rows = tokens * k
    gen = torch.Generator().manual_seed(dim)
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    ids = torch.randint(0, E, (n, tokens, k), generator=gen, dtype=torch.int32).cuda()
    x = torch.randint(-3, 4, (n, tokens, dim), generator=gen).half().cuda()
    w = torch.ones(tokens, k, device="cuda")
    eye = torch.eye(dim, dtype=torch.uint8)
    B = torch.stack([eye * (e + 1) for e in range(E)]).half().cuda()                     # expert e: times e + 1
    q = torch.stack([8 + eye * 2 * (i + 1) for i in range(3)]).view(3, dim, dim // 2, 2)   # i: times 2 (i + 1)
    B4, s4 = (q[..., 0] | (q[..., 1] << 4)).contiguous().cuda(), torch.ones(1, dim, dim // 32).half().cuda()
    off, row_of, src = i32(E + 1), i32(tokens, k), i32(rows)
    xs, c, out = zeros(rows, dim), zeros(rows, dim), zeros(n, tokens, dim)
    torch.cuda.synchronize()
    # routing: sort writes row_of, gather and combine read it
    for i in range(n):
        pts.gemm_expert_sort(h, tokens, k, E, ids[i], off, row_of, src)
        pts.gemm_expert_gather(h, tokens, k, dim, x[i], row_of, xs, F16)
        pts.gemm_expert_combine(h, tokens, k, dim, xs, row_of, w, out[i], F16)
    torch.cuda.synchronize()
    assert torch.equal(out, 2 * x)
    # rows: gather writes them, the 4-bit product reads them
    got = zeros(n, rows, dim)
    for i in range(n):
        pts.gemm_expert_gather(h, tokens, k, dim, x[i], row_of, xs, F16)
        pts.gemm_run_nibble(h, rows, 1, dim, dim, 32, xs, B4[0], s4, None, None, got[i], F16)
    torch.cuda.synchronize()
    assert torch.equal(got[:, row_of.long()], 2 * x[:, :, None].expand(-1, -1, k, -1))
    # sums: the 4-bit product, with other weights each time, writes the rows, combine reads them
    for i in range(n):
        pts.gemm_run_nibble(h, rows, 1, dim, dim, 32, xs, B4[i % 3], s4, None, None, c, F16)
        pts.gemm_expert_combine(h, tokens, k, dim, c, row_of, w, out[i], F16)
    torch.cuda.synchronize()
    factor = 4.0 * (1 + torch.arange(n, device="cuda") % 3)
    assert torch.equal(out.float(), factor[:, None, None] * x[-1].float())
    # offsets: sort writes them, the products read them (the row's factor tells whose it was)
    for i in range(n):
        pts.gemm_expert_sort(h, tokens, k, E, ids[i], off, row_of, src)
        pts.gemm_run_experts(h, rows, E, dim, dim, xs, B, off, got[i], F16)
    torch.cuda.synchronize()
    for i in range(n):
        e = ids[i].flatten().sort()[0]
        assert torch.equal(got[i].float(), (e + 1).float()[:, None] * xs.float()), i
