"""The experts' products over long contractions, bit for bit.

Operands of -1, 0 and 1: every partial sum is an integer below 2^24, exact in fp32 in any order and however CTAs share
a contraction, so the result has to be the exact sum rounded once."""
import numpy as np
import pytest
import torch

import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu

F16, BF16, E4M3 = pts.GEMM_F16, pts.GEMM_BF16, pts.GEMM_E4M3
TORCH = {F16: torch.float16, BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn}
OUT = {F16: torch.float16, BF16: torch.bfloat16, E4M3: torch.bfloat16}
HANDLES = {"auto": {}, "single": dict(cta_group=1), "pair": dict(cta_group=2), "pair2": dict(cta_group=2, max_clusters=2)}


@pytest.fixture(scope="module", params=HANDLES)
def hv(request):
    h = pts.gemm_create(0, pts.make_opts(**HANDLES[request.param]))
    yield h
    st, dev = pts.gemm_check(h)
    pts.gemm_destroy(h)
    assert st == 0, f"device status {dev:#x}"


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def signs(shape, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=gen, device="cuda").float().to(TORCH[dtype])


def spans(counts):
    at = np.concatenate([[0], np.cumsum(counts)])
    return [(e, slice(int(at[e]), int(at[e + 1]))) for e in range(len(counts))]


# rows per expert, rows behind the last, features, contraction: shared contractions (few tiles), tiles of 64 and of 256 rows
LONG = [([1], 0, 520, 16400), ([3, 0, 0, 2], 4, 136, 8208), ([20, 9, 0], 3, 264, 16384), ([100], 0, 264, 12304),
        ([257, 0, 130], 1, 392, 8176), ([33] * 9, 0, 72, 4112)]


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids=["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("counts,spare,N,K", LONG)
def test_forward(hv, counts, spare, N, K, dtype):
    rows, E = sum(counts) + spare, len(counts)
    A, B = signs((rows, K), dtype, 1), signs((E, N, K), dtype, 2)
    C = torch.full((rows, N), 7.0, dtype=OUT[dtype], device="cuda")
    pts.gemm_run_experts(hv, rows, E, N, K, A, B, offsets_of(counts), C, dtype)
    for e, r in spans(counts):
        assert torch.equal(C[r], (A[r].double() @ B[e].double().T).to(OUT[dtype])), e
    assert (C[sum(counts):] == 7.0).all()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("counts,spare,K,N", LONG)
def test_dgrad(hv, counts, spare, K, N, dtype):
    rows, E = sum(counts) + spare, len(counts)
    dC, B = signs((rows, N), dtype, 3), signs((E, N, K), dtype, 4)
    dA = torch.full((rows, K), 7.0, dtype=TORCH[dtype], device="cuda")
    pts.gemm_run_experts_dgrad(hv, rows, E, N, K, dC, B, offsets_of(counts), dA, dtype)
    for e, r in spans(counts):
        assert torch.equal(dA[r], (dC[r].double() @ B[e].double()).to(TORCH[dtype])), e
    assert (dA[sum(counts):] == 7.0).all()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("counts,N,K", [([9001], 136, 264), ([4096, 0, 3, 5005], 264, 72), ([2047, 2049, 1], 72, 520)])
def test_wgrad(hv, counts, N, K, dtype):
    rows, E = sum(counts), len(counts)
    dC, A = signs((rows, N), dtype, 5), signs((rows, K), dtype, 6)
    dB = torch.full((E, N, K), float("nan"), dtype=TORCH[dtype], device="cuda")
    pts.gemm_run_experts_wgrad(hv, rows, E, N, K, dC, A, offsets_of(counts), dB, dtype)
    for e, r in spans(counts):
        assert torch.equal(dB[e], (dC[r].double().T @ A[r].double()).to(TORCH[dtype])), e


@pytest.mark.parametrize("counts,K", [([2, 0, 3, 0, 1], 4096), ([20, 9, 1], 16384), ([200, 0, 90], 4096)])
def test_an_infinity_reaches_its_row_and_all_of_it(hv, counts, K):
    """One infinity in the rows: infinite or NaN wherever its weight is not 0 (NaN where it is: inf * 0), the other rows
    as without it."""
    N, rows, E = 264, sum(counts), len(counts)
    A, B, off = signs((rows, K), F16, 7), signs((E, N, K), F16, 8), offsets_of(counts)
    for row, k in ((0, 0), (rows - 2, K - 1), (rows - 1, K - 96)):
        a = A.clone()
        a[row, k] = float("inf")
        C = torch.full((rows, N), 7.0, dtype=torch.float16, device="cuda")
        pts.gemm_run_experts(hv, rows, E, N, K, a, B, off, C, F16)
        for e, r in spans(counts):
            want = (A[r].double() @ B[e].double().T).half()
            here = row - r.start
            if 0 <= here < r.stop - r.start:
                w = B[e, :, k].double()
                assert (C[row][w > 0] == float("inf")).all() and (C[row][w < 0] == -float("inf")).all()
                assert torch.isnan(C[row][w == 0]).all()
                want[here] = C[row]
            assert torch.equal(C[r].view(torch.int16), want.view(torch.int16)), e
