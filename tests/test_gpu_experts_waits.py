"""Bounded waits of the expert layer's products: a stage load that does not come in full makes a wait run out, the
call reports GEMM_ERR_TIMEOUT (nothing traps, nothing hangs), and the next call on the same context is exact."""
import numpy as np
import pytest
import torch

import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu

F16 = pts.GEMM_F16
TIMEOUT_NS = 20_000_000


def ints(shape, seed, most=1):
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=gen).half().cuda()


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def run_out_then_exact(opts, fault_arg, call):
    """call(h) makes one call and returns its output and what it has to be."""
    h = pts.gemm_create(0, pts.make_opts(debug_flags=pts.GEMM_DEBUG_FAULT_SKIP_TMA, fault_arg=fault_arg,
                                         timeout_ns=TIMEOUT_NS, **opts))
    try:
        call(h)
        st, dev = pts.gemm_check(h)
        assert st == pts.gemm.GEMM_ERR_TIMEOUT and dev >> 24 == 1
        assert pts.gemm_check(h)[0] == 0   # the status block was cleared
    finally:
        pts.gemm_destroy(h)
    h = pts.gemm_create(0, pts.make_opts(**opts))
    try:
        got, want = call(h)
        assert pts.gemm_check(h)[0] == 0
        assert torch.equal(got.double(), want)
    finally:
        pts.gemm_destroy(h)


def per_expert(counts, f):
    at = np.concatenate([[0], np.cumsum(counts)])
    return [f(e, slice(int(at[e]), int(at[e + 1]))) for e in range(len(counts))]


HANDLES = {"auto": {}, "single": dict(cta_group=1), "pair": dict(cta_group=2), "pair2": dict(cta_group=2, max_clusters=2)}

# rows per expert, N, K, the load that is withheld: one of few, which the producer has all issued when the wait runs
# out (the first and the last of them), and one in the middle of many
PRODUCTS = [([5, 0, 70], 264, 128, 0), ([40], 136, 200, 0), ([300, 33], 520, 208, 1), ([700, 90], 1000, 1040, 5)]


@pytest.mark.parametrize("opts", HANDLES)
@pytest.mark.parametrize("counts,N,K,load", PRODUCTS)
def test_forward(opts, counts, N, K, load):
    rows, off = sum(counts), offsets_of(counts)
    A, B = ints((rows, K), 1), ints((len(counts), N, K), 2)

    def call(h):
        C = torch.zeros(rows, N, dtype=torch.float16, device="cuda")
        pts.gemm_run_experts(h, rows, len(counts), N, K, A, B, off, C, F16)
        return C, torch.cat(per_expert(counts, lambda e, r: A[r].double() @ B[e].double().T))

    run_out_then_exact(HANDLES[opts], load, call)


@pytest.mark.parametrize("counts,N,K", [([1], 1024, 4096), ([1], 256, 8192), ([3, 0, 2], 136, 2048)])
@pytest.mark.parametrize("load", [0, 3])
def test_forward_of_few_tiles(counts, N, K, load):
    """CTAs that share a tile's contraction: all of them give up, and meet all the same."""
    test_forward("auto", counts, N, K, load)


@pytest.mark.parametrize("opts", HANDLES)
@pytest.mark.parametrize("counts,K,N,load", PRODUCTS)
def test_dgrad(opts, counts, K, N, load):
    rows, off = sum(counts), offsets_of(counts)
    dC, B = ints((rows, N), 3), ints((len(counts), N, K), 4)

    def call(h):
        dA = torch.zeros(rows, K, dtype=torch.float16, device="cuda")
        pts.gemm_run_experts_dgrad(h, rows, len(counts), N, K, dC, B, off, dA, F16)
        return dA, torch.cat(per_expert(counts, lambda e, r: dC[r].double() @ B[e].double()))

    run_out_then_exact(HANDLES[opts], load, call)


# rows that end inside a 16-row step (the stage that is cleared first: the last of them) and rows that do not
@pytest.mark.parametrize("opts", HANDLES)
@pytest.mark.parametrize("counts,load", [([40], 0), ([48], 0), ([100, 64], 0), ([1000], 7), ([700, 90], 3), ([333] * 5, 2)])
def test_wgrad(opts, counts, load):
    rows, off, N, K = sum(counts), offsets_of(counts), 264, 520
    dC, A = ints((rows, N), 5), ints((rows, K), 6)

    def call(h):
        dB = torch.zeros(len(counts), N, K, dtype=torch.float16, device="cuda")
        pts.gemm_run_experts_wgrad(h, rows, len(counts), N, K, dC, A, off, dB, F16)
        return dB, torch.stack(per_expert(counts, lambda e, r: dC[r].double().T @ A[r].double()))

    run_out_then_exact(HANDLES[opts], load, call)


# one matrix and experts; 8 rows at a time with 1, 2 and 4 CTAs to a contraction, and more rows at a time
NIBBLE = [([3], 264, 256, 0), ([8], 1000, 8192, 0), ([1], 4096, 16384, 0), ([4, 0, 9], 136, 1024, 0),
          ([64], 4096, 4096, 0), ([64], 4096, 16384, 7), ([512], 1032, 1536, 2), ([512], 4104, 512, 3), ([64, 33] * 4, 1032, 1536, 2)]


@pytest.mark.parametrize("counts,N,K,load", NIBBLE)
def test_nibble(counts, N, K, load):
    rows, E, off = sum(counts), len(counts), offsets_of(counts)
    A = torch.zeros(rows, K, dtype=torch.float16, device="cuda")
    A[torch.arange(rows), (torch.arange(rows) * 37) % K] = 1.0
    gen = torch.Generator().manual_seed(7)
    q = torch.randint(0, 16, (E, N, K), generator=gen, dtype=torch.uint8)
    b = q.view(E, N, K // 2, 2)
    B, s = (b[..., 0] | (b[..., 1] << 4)).contiguous().cuda(), torch.ones(E, N, K // 64).half().cuda()
    w = q.double().cuda() - 8.0

    def call(h):
        C = torch.zeros(rows, N, dtype=torch.float16, device="cuda")
        pts.gemm_run_nibble(h, rows, E, N, K, 64, A, B, s, None, None if E == 1 else off, C, F16)
        return C, torch.cat(per_expert(counts, lambda e, r: A[r].double() @ w[e].T))

    run_out_then_exact({}, load, call)


@pytest.mark.parametrize("rows,ctas", [(8, 1), (32, 1), (32, 2), (32, 4), (64, 1), (64, 2), (64, 4)])
@pytest.mark.parametrize("counts,N,K,load", [([70], 264, 1024, 0), ([40, 0, 33], 136, 4096, 3), ([300], 1032, 8192, 7)])
def test_every_form_of_nibble(rows, ctas, counts, N, K, load):
    """The withheld load: the first, the last but some, one in the middle; every CTA has K / 256 / ctas of them at least."""
    E, off, R = len(counts), offsets_of(counts), sum(counts)
    A, form = ints((R, K), 8), pts.GEMM_DEBUG_NIBBLE_FORM(rows, ctas)
    B, s = torch.full((E, N, K // 2), 0x99, dtype=torch.uint8, device="cuda"), torch.ones(E, N, K // 64).half().cuda()
    want = A.double().sum(1)[:, None].expand(R, N)

    def call(flags):
        h = pts.gemm_create(0, pts.make_opts(debug_flags=form | flags, fault_arg=load, timeout_ns=TIMEOUT_NS))
        C = torch.zeros(R, N, dtype=torch.float16, device="cuda")
        pts.gemm_run_nibble(h, R, E, N, K, 64, A, B, s, None, None if E == 1 else off, C, F16)
        st, dev = pts.gemm_check(h)
        pts.gemm_destroy(h)
        return C, st, dev

    C, st, dev = call(pts.GEMM_DEBUG_FAULT_SKIP_TMA)
    assert st == pts.gemm.GEMM_ERR_TIMEOUT and dev >> 24 == 1
    C, st, dev = call(0)
    assert st == 0 and torch.equal(C.double(), want)
