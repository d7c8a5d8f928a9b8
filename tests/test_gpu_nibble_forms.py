"""Every form of the product with 4-bit weights (blocks of 8, 32 and 64 rows, the latter two with 1, 2 and 4 CTAs to a
tile's contraction), taken whatever the sizes.

Rows of -1, 0 and 1 and scales that are powers of two: every partial sum is a multiple of 1/4 below 2^24 of them, so
the sums are exact in fp32 in any order, and the result has to be the exact sum rounded once, bit for bit."""
import numpy as np
import pytest
import torch

import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu

F16, BF16 = pts.GEMM_F16, pts.GEMM_BF16
TORCH = {F16: torch.float16, BF16: torch.bfloat16}
FORMS = [(8, 1), (32, 1), (32, 2), (32, 4), (64, 1), (64, 2), (64, 4)]


@pytest.fixture(scope="module", params=FORMS, ids=lambda f: f"{f[0]}x{f[1]}")
def hf(request):
    h = pts.gemm_create(0, pts.make_opts(debug_flags=pts.GEMM_DEBUG_NIBBLE_FORM(*request.param)))
    yield h
    st, dev = pts.gemm_check(h)
    pts.gemm_destroy(h)
    assert st == 0, f"device status {dev:#x}"


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def weights(E, N, K, group, dtype, zeros, seed):
    """-> codes, scales (1/4 .. 2, another one for each group), zeros or None, and the matrices they stand for."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 16, (E, N, K), generator=gen, dtype=torch.uint8, device="cuda")
    groups = -(-K // group)
    s = 2.0 ** torch.randint(-2, 2, (E, N, groups), generator=gen, device="cuda").double()
    z = torch.randint(0, 16, (E, N, groups), generator=gen, dtype=torch.uint8, device="cuda") if zeros else None
    at = torch.arange(K, device="cuda") // group
    w = (q.double() - (8.0 if z is None else z.double()[..., at])) * s[..., at]
    b = q.view(E, N, K // 2, 2)
    return (b[..., 0] | (b[..., 1] << 4)).contiguous(), s.to(TORCH[dtype]), z, w


def signs(rows, K, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, (rows, K), generator=gen, device="cuda").to(TORCH[dtype])


def product(A, w, counts):
    at = np.concatenate([[0], np.cumsum(counts)])
    return torch.cat([A[int(at[e]):int(at[e + 1])].double() @ w[e].T for e in range(len(counts))])


# rows per expert, rows behind the last, N, the contraction in whole units of 256 and not; one expert has no offsets
SIZES = [([1], 0, 8, (256, 32)), ([64], 0, 264, (1024, 1056)), ([70, 0, 3, 33], 5, 136, (2048, 2080)),
         ([31] * 20, 1, 72, (256, 352)), ([500], 0, 2056, (512, 800)), ([200], 0, 520, (16384, 16224)),
         ([33, 40], 0, 1000, (8192, 8224))]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("counts,spare,N,Ks", SIZES)
def test_exact(hf, counts, spare, N, Ks, dtype):
    rows, E = sum(counts) + spare, len(counts)
    off = None if E == 1 else offsets_of(counts)
    for K in Ks:
        A = signs(rows, K, dtype, 1)
        A[sum(counts):] = float("nan")
        for group in (32, 64, 128):
            for zeros in (False, True):
                B, s, z, w = weights(E, N, K, group, dtype, zeros, group + zeros)
                C = torch.full((rows, N), 7.0, dtype=TORCH[dtype], device="cuda")
                pts.gemm_run_nibble(hf, rows, E, N, K, group, A, B, s, z, off, C, dtype)
                want = product(A, w, counts).to(TORCH[dtype])
                assert torch.equal(C[:sum(counts)], want), (K, group, zeros, int((C[:sum(counts)] != want).sum()))
                assert (C[sum(counts):] == 7.0).all()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("K", [1056, 4096])
def test_values_stay_with_their_row_and_feature(hf, K, dtype):
    """Infinities and NaN in a row, in a neighbour expert's rows and in a scale of the last, perhaps short, group."""
    counts, N = [40, 0, 37], 264
    rows, E, off, T = sum(counts), len(counts), offsets_of(counts), TORCH[dtype]
    for group in (32, 64, 128):
        A = signs(rows, K, dtype, 2)
        B, s, z, w = weights(E, N, K, group, dtype, True, group)
        want = product(A, w, counts).to(T)
        A[10, 7], A[76, K - 1] = float("inf"), float("nan")
        s[2, 5, -1], s[2, 6, 0] = float("inf"), float("nan")
        C = torch.empty(rows, N, dtype=T, device="cuda")
        pts.gemm_run_nibble(hf, rows, E, N, K, group, A, B, s, z, off, C, dtype)
        keep = torch.ones(rows, N, dtype=torch.bool, device="cuda")
        keep[10], keep[76], keep[40:, 5:7] = False, False, False
        assert torch.equal(C[keep], want[keep])
        assert not torch.isfinite(C[10]).any()     # (inf times a weight, or NaN where that is 0)
        assert torch.isnan(C[76]).all() and torch.isnan(C[40:, 6]).all()
        assert not torch.isfinite(C[40:, 5]).any()
        # all products positive: an infinite scale gives infinities, not NaN
        ones, nines, one = torch.ones_like(A), torch.full_like(B, 0x99), torch.ones_like(s)
        one[2, 5, -1] = float("inf")
        pts.gemm_run_nibble(hf, rows, E, N, K, group, ones, nines, one, None, off, C, dtype)
        want = torch.full((rows, N), float(K), device="cuda").to(T)
        want[40:, 5] = float("inf")
        assert torch.equal(C, want)


@pytest.mark.parametrize("rows,E,N", [(64, 64, 40), (3000, 200, 1032)])
def test_offsets_that_go_back_and_forth_stay_inside(hf, rows, E, N):
    """Every other expert claims all rows; every expert's weights are ones, so a row is its sum whoever multiplies it."""
    K = 320
    A = signs(rows, K, F16, 3)
    B, s = torch.full((E, N, K // 2), 0x99, dtype=torch.uint8, device="cuda"), torch.ones(E, N, K // 32).half().cuda()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1::2] = rows
    off[E // 2] = 1 << 30
    off[0] = -5
    C = torch.full((rows + 8, N), 7.0, dtype=torch.float16, device="cuda")
    pts.gemm_run_nibble(hf, rows, E, N, K, 32, A, B, s, None, off, C, F16)
    assert (C[:rows] == A.double().sum(1)[:, None]).all() and (C[rows:] == 7).all()


def test_no_contraction_writes_zeros(hf):
    C = torch.full((75, 40), 7.0, dtype=torch.float16, device="cuda")
    pts.gemm_run_nibble(hf, 75, 3, 40, 0, 32, None, None, None, None, offsets_of([3, 0, 70]), C, F16)
    assert (C[:73] == 0).all() and (C[73:] == 7).all()


@pytest.mark.parametrize("tokens,K,N", [(40, 256, 136), (300, 1024, 264), (130, 4128, 72)])
def test_calls_back_to_back_see_what_the_one_before_wrote(hf, tokens, K, N):
    """Queued over and over on the same buffers, with other rows, routing and weights each time: gather writes the rows
    that the product reads, sort its offsets, and combine reads what it wrote, each started while the others run."""
    E, k, n = 5, 2, 40
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    ids = torch.randint(-1, E, (n, tokens, k), generator=gen, dtype=torch.int32, device="cuda")
    x = torch.randint(-1, 2, (n, tokens, K), generator=gen, device="cuda").half()
    B, s, _, w = zip(*(weights(E, N, K, 64, F16, False, i) for i in range(2)))
    i32 = lambda *d: torch.zeros(*d, dtype=torch.int32, device="cuda")  # noqa: E731
    off, row_of, src, ones = i32(E + 1), i32(tokens, k), i32(tokens * k), torch.ones(tokens, k, device="cuda")
    xs, c = (torch.zeros(tokens * k, d, dtype=torch.float16, device="cuda") for d in (K, N))
    y = torch.zeros(n, tokens, N, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    for i in range(n):
        pts.gemm_expert_sort(hf, tokens, k, E, ids[i], off, row_of, src)
        pts.gemm_expert_gather(hf, tokens, k, K, x[i], row_of, xs, F16)
        pts.gemm_run_nibble(hf, tokens * k, E, N, K, 64, xs, B[i % 2], s[i % 2], None, off, c, F16)
        pts.gemm_expert_combine(hf, tokens, k, N, c, row_of, ones, y[i], F16)
    torch.cuda.synchronize()
    for i in range(n):
        all_e = torch.einsum("tk,enk->ten", x[i].double(), w[i % 2]).half().double()   # (as the product rounds it)
        held = (ids[i] >= 0)[..., None]
        terms = torch.where(held, all_e[torch.arange(tokens, device="cuda")[:, None], ids[i].clamp(min=0).long()], 0.0)
        assert torch.equal(y[i], terms.sum(1).half()), i


def test_more_tiles_than_sms_with_shared_contractions():
    """The form that the library takes by itself for this size: 4 CTAs to each of 160 tiles, several rounds of them."""
    rows, N, K = 64, 20480, 16384
    h = pts.gemm_create(0)
    A = signs(rows, K, BF16, 4)
    B, s, _, w = weights(1, N, K, 128, BF16, False, 5)
    C = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    pts.gemm_run_nibble(h, rows, 1, N, K, 128, A, B, s, None, None, C, BF16)
    want = (A.double() @ w[0].T).to(torch.bfloat16)
    st, dev = pts.gemm_check(h)
    pts.gemm_destroy(h)
    assert st == 0 and torch.equal(C, want)


@pytest.mark.parametrize("rows,ctas", [(8, 0), (8, 2), (16, 1), (32, 0), (32, 3), (64, 8), (0, 1), (128, 1)])
def test_other_forms_are_refused(rows, ctas):
    with pytest.raises(pts.GemmError) as err:
        pts.gemm_create(0, pts.make_opts(debug_flags=pts.GEMM_DEBUG_NIBBLE_FORM(rows, ctas)))
    assert err.value.status == pts.gemm.GEMM_ERR_INVALID_ARG
