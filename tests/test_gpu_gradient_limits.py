"""The epilogue's gradient where sums are very large, infinite or NaN."""
import pytest
import torch

import layer_reference as ref
import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu

F16, BF16 = pts.GEMM_F16, pts.GEMM_BF16
TORCH = {F16: torch.float16, BF16: torch.bfloat16}
NAMES = {F16: "f16", BF16: "bf16"}.get
GATED, INF, NAN = pts.GEMM_ACT_GATED, float("inf"), float("nan")
# (relu^2's slope is twice its sum, finite in 32 bits up to 1.7e38)
HIGH = [5.0, 20.0, 63.0, 64.0, 65.0, 90.0, 300.0, 5000.0, 65504.0, 1e10, 1e18, 1e19, 1e30, 3e35, 3.8e35, 4e35, 1e36, 1e38, INF]


@pytest.fixture(scope="module")
def h():
    h = pts.gemm_create(0)
    yield h
    pts.gemm_destroy(h)


def high(dtype):
    """8 * 7 values: each of HIGH that the type has beside other ones in a pair, in either place."""
    x = torch.tensor([v for v in HIGH if v <= torch.finfo(dtype).max or v == INF])
    return torch.stack([x[(torch.arange(56) * step) % len(x)] for step in (1, 2, 5)]).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES)
@pytest.mark.parametrize("gated", [0, GATED], ids=["plain", "gated"])
@pytest.mark.parametrize("code", range(1, 6), ids=ref.ACTS[1:])
def test_slopes_of_large_sums(h, code, gated, dtype):
    """Up to the type's largest values and infinity the slope of all but relu^2 is 1 to within its rounding (from 20 on: 20 phi(20) is
    2^-287, and 20 exp(-20) 2^-24; at 5 it is not), and the activation its argument."""
    t, N = TORCH[dtype], 56
    z = high(t)
    Z = torch.cat([z, torch.full_like(z, -0.75)], 1)[:, :N * (2 if gated else 1)].contiguous()
    dC, dZ = torch.full_like(z, 0.5), torch.full_like(Z, 7.0)
    pts.gemm_linear_grad(h, 3, 1, N, dC, Z, None, dZ, None, code | gated, dtype)
    a, s, sa = ref.act(code, z.double().clamp(max=1e100))   # (the formulas' products of an infinity and 0 do not arise)
    factor = -0.75 if gated else 1.0
    want, err = s * 0.5 * factor, sa * 0.5 * abs(factor) * 2 * ref.EPS_ACT
    if gated:
        want, err = torch.cat([want, a * 0.5], 1), torch.cat([err, a.abs() * 0.5 * 2 * ref.EPS_ACT], 1)
    want = want.to(t).double()   # (rounded: what overflows is infinite on both sides)
    same = dZ.double() == want
    assert (same | ((dZ.double() - want).abs() <= 2 * ref.U[t] * want.abs() + err + ref.TINY)).all()
    if code != 2:
        assert torch.equal(dZ[:, :N][z >= 20.0], torch.full_like(dZ[:, :N], 0.5 * factor)[z >= 20.0])


@pytest.mark.parametrize("gated", [0, GATED], ids=["plain", "gated"])
@pytest.mark.parametrize("code", range(1, 6), ids=ref.ACTS[1:])
def test_a_sum_that_overflows_its_type(h, code, gated):
    """A product's fp16 sums of 80000 are kept as infinity: the gradient is finite wherever the slope is."""
    rows, N, K = 20, 64, 80
    A, B = torch.full((rows, K), 1000.0, dtype=torch.float16, device="cuda"), torch.ones(N * (2 if gated else 1), K, dtype=torch.float16, device="cuda")
    A[1::2] *= -1.0
    if gated:
        B[N:] = 0.0
        B[N:, 0] = 2.0 ** -10
    C, Z = torch.zeros(rows, N, dtype=torch.float16, device="cuda"), torch.zeros(rows, B.shape[0], dtype=torch.float16, device="cuda")
    pts.gemm_run_linear(h, rows, 1, N, K, A, B, None, None, None, C, Z, code | gated, F16)
    assert (Z[0::2, :N] == INF).all() and (Z[1::2, :N] == -INF).all() and (C[0::2] == INF).all() and (C[1::2] == 0).all()
    dC, dZ = torch.full_like(C, 0.25), torch.full_like(Z, 7.0)
    pts.gemm_linear_grad(h, rows, 1, N, dC, Z, None, dZ, None, code | gated, F16)
    up = Z[:, N:] if gated else torch.ones_like(C)
    assert (dZ[1::2, :N] == 0).all()
    assert (dZ[0::2, :N] == INF).all() if code == 2 else torch.equal(dZ[0::2, :N], (dC * up)[0::2])
    if gated:
        assert (dZ[0::2, N:] == INF).all() and (dZ[1::2, N:] == 0).all()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES)
@pytest.mark.parametrize("gated", [0, GATED], ids=["plain", "gated"])
@pytest.mark.parametrize("code", range(1, 6), ids=ref.ACTS[1:])
def test_a_nan_stays_one(h, code, gated, dtype):
    """A NaN in Z, in either place of a pair, reaches its own gradients, dbias with them, and no others; forward too."""
    t, N, rows = TORCH[dtype], 48, 6
    z = torch.linspace(-3, 3, rows * N).view(rows, N).to(t).cuda()
    z[1, 6], z[4, 7] = NAN, NAN
    Z = torch.cat([z, torch.full_like(z, 1.5)], 1)[:, :N * (2 if gated else 1)].contiguous()
    dC, dZ, dbias = torch.full_like(z, 0.5), torch.zeros_like(Z), torch.zeros(1, Z.shape[1], device="cuda")
    pts.gemm_linear_grad(h, rows, 1, N, dC, Z, None, dZ, dbias, code | gated, dtype)
    bad, cols = torch.zeros_like(Z, dtype=torch.bool), [6, 7, N + 6, N + 7] if gated else [6, 7]
    for r, c in ((1, 6), (4, 7)):
        bad[r, c::N] = True
    assert torch.equal(torch.isnan(dZ), bad) and torch.isfinite(dZ[~bad]).all()
    assert torch.isnan(dbias[0, cols]).all() and int(torch.isnan(dbias).sum()) == len(cols)
    K = 16
    A, B, C = torch.zeros(rows, K, dtype=t, device="cuda"), torch.zeros(Z.shape[1], K, dtype=t, device="cuda"), torch.zeros(rows, N, dtype=t, device="cuda")
    pts.gemm_run_linear(h, rows, 1, N, K, A, B, Z[1:2].contiguous(), None, None, C, None, code | gated, dtype)
    assert torch.isnan(C[:, 6]).all() and int(torch.isnan(C).sum()) == rows
