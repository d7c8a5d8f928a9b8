"""The product with bias, activation and residual, and its gradient, against plain forms in 64 bits (layer_reference.py)."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu

F16, BF16, E4M3 = pts.GEMM_F16, pts.GEMM_BF16, pts.GEMM_E4M3
TORCH = {F16: torch.float16, BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn}
OUT = {F16: torch.float16, BF16: torch.bfloat16, E4M3: torch.bfloat16}
NAMES = {F16: "f16", BF16: "bf16", E4M3: "e4m3"}.get
GATED = pts.GEMM_ACT_GATED


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
    """Handles that take every variant, and several tiles per cluster."""
    h = pts.gemm_create(0, pts.make_opts(**request.param))
    yield h
    st, dev = pts.gemm_check(h)
    pts.gemm_destroy(h)
    assert st == 0, f"device status {dev:#x}"


def rand(shape, dtype, seed, scale=1.0):
    x = torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale
    return (x.clamp(-448, 448) if dtype == torch.float8_e4m3fn else x).to(dtype).cuda()


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def spans(counts):
    at = np.concatenate([[0], np.cumsum(counts)])
    return [(e, slice(int(at[e]), int(at[e + 1]))) for e in range(len(counts))]


# rows per expert, rows behind the last, N, K
SHAPES = [([1], 0, 8, 16), ([5, 0, 3], 2, 264, 208), ([0, 0, 40, 1, 0], 0, 128, 64), ([16, 17, 15, 64, 65], 5, 392, 1008),
          ([300, 0, 1, 257, 128], 31, 520, 144), ([1025, 63], 0, 256, 336), ([3] * 45, 0, 144, 80), ([700], 0, 1000, 272),
          # few tiles and a long contraction
          ([1], 0, 136, 4112), ([0, 0, 1, 0], 0, 2056, 2064), ([3, 0, 0, 2], 4, 128, 8208), ([20, 9, 0], 3, 1000, 2000)]
# activation, bias, residual, Z kept
OPTIONS = [(0, True, True, False), (5, False, False, True), (3 | GATED, True, True, True), (5 | GATED, False, True, False),
           (2, True, True, True), (4 | GATED, True, False, True), (1, False, True, False), (4, True, False, False), (0 | GATED, False, False, False)]


def run_linear(h, counts, spare, N, K, dtype, option, one_matrix=False, in_place=False):
    act, has_bias, has_residual, keep = option
    rows, E, all_, out = sum(counts) + spare, len(counts), N * (2 if act & GATED else 1), OUT[dtype]
    A, B = rand((rows, K), TORCH[dtype], 11), rand((E, all_, K), TORCH[dtype], 12, 2.0 / K ** 0.5 if dtype != E4M3 else 1.0)
    if dtype != E4M3:
        A[sum(counts):] = float("nan")
    scale = (8.0, K ** 0.5 / 16) if dtype == E4M3 else (1.0, 1.0)
    scale = tuple(float(np.float32(s)) for s in scale)
    bias, residual = rand((E, all_), out, 13) if has_bias else None, rand((rows, N), out, 14) if has_residual else None
    C = torch.full((rows, N), 7.0, dtype=out, device="cuda")
    if in_place and has_residual:
        C.copy_(residual)
    Z = torch.full((rows, all_), 7.0, dtype=out, device="cuda") if keep else None
    before = C.clone()
    pts.gemm_run_linear(h, rows, E, N, K, A, B, bias, C if in_place and has_residual else residual, None if one_matrix else offsets_of(counts),
                        C, Z, act, dtype, *scale)
    for e, r in spans(counts):
        (c, dc), (z, dz) = ref.linear(act, A[r], B[e], None if bias is None else bias[e], None if residual is None else residual[r], scale[0] * scale[1])
        ref.close(C[r], c, dc, ("C", e))
        if keep:
            ref.close(Z[r], z, dz, ("Z", e))
    assert torch.equal(C[sum(counts):], before[sum(counts):])   # rows of no expert are not written
    assert Z is None or (Z[sum(counts):] == 7.0).all()


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids=NAMES)
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_linear(hv, case, dtype):
    """Every shape with a third of the options, so that each option meets each type and variant in several shapes."""
    for option in OPTIONS[case % 3::3]:
        run_linear(hv, *SHAPES[case], dtype, option)


@pytest.mark.parametrize("option", OPTIONS, ids=str)
@pytest.mark.parametrize("rows,N,K", [(1, 64, 128), (17, 520, 264), (130, 1032, 520), (515, 264, 1040), (1, 2048, 4096), (24, 512, 8192)])
def test_one_matrix_without_offsets(hv, rows, N, K, option):
    run_linear(hv, [rows], 0, N, K, BF16, option, one_matrix=True)


@pytest.mark.parametrize("option", [o for o in OPTIONS if o[2]], ids=str)
@pytest.mark.parametrize("case", [3, 4, 7, 8, 10])
def test_residual_in_place(hv, case, option):
    run_linear(hv, *SHAPES[case], F16, option, in_place=True)


@pytest.mark.parametrize("act", range(6), ids=ref.ACTS)
@pytest.mark.parametrize("gated", [0, GATED])
def test_every_activation(h, act, gated):
    run_linear(h, [150, 20], 3, 272, 144, F16, (act | gated, True, True, True))
    run_linear(h, [2, 0, 1], 0, 272, 144, BF16, (act | gated, True, False, True))


@pytest.mark.parametrize("counts,N,K", [([300, 20], 264, 72), ([2, 1], 136, 2048), ([3], 128, 40)])
def test_small_integers_are_exact(hv, counts, N, K):
    rows, E = sum(counts), len(counts)
    gen = torch.Generator().manual_seed(1)
    ints = lambda *s: torch.randint(-1, 2, s, generator=gen).half().cuda()  # noqa: E731
    A, B, bias, residual = ints(rows, K), ints(E, N, K), ints(E, N) * 5, ints(rows, N) * 3
    C, Z = (torch.zeros(rows, N, dtype=torch.float16, device="cuda") for _ in range(2))
    pts.gemm_run_linear(hv, rows, E, N, K, A, B, bias, residual, offsets_of(counts), C, Z, pts.GEMM_ACT_RELU, F16)
    z = torch.cat([A[r].double() @ B[e].double().T + bias[e].double() for e, r in spans(counts)])
    assert torch.equal(Z.double(), z) and torch.equal(C.double(), z.clamp(min=0) + residual.double())


def test_without_a_contraction(h):
    """K = 0: the sums are the bias."""
    bias, residual = rand((2, 64), torch.bfloat16, 1), rand((5, 32), torch.bfloat16, 2)
    C, Z = torch.zeros(5, 32, dtype=torch.bfloat16, device="cuda"), torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda")
    pts.gemm_run_linear(h, 5, 2, 32, 0, None, None, bias, residual, offsets_of([3, 2]), C, Z, pts.GEMM_ACT_SILU | GATED, BF16)
    z = bias.double()[[0, 0, 0, 1, 1]]
    assert torch.equal(Z.double(), z)
    ref.close(C, ref.hidden(5 | GATED, z, 0 * z)[0] + residual.double(), 2.0 ** -14 * z[:, :32].abs() * z[:, 32:].abs() + 2.0 ** -22)


def test_empty_calls(h):
    x = torch.zeros(64, dtype=torch.float16, device="cuda")
    assert pts.gemm_run_linear(h, 0, 1, 8, 8, x, x, None, None, None, x, None, 0, F16) == 0
    assert pts.gemm_run_linear(h, 8, 0, 8, 8, x, x, None, None, None, x, None, 0, F16) == 0
    assert pts.gemm_run_linear(h, 8, 1, 0, 8, x, x, None, None, None, x, None, 0, F16) == 0
    assert pts.gemm_linear_grad(h, 0, 1, 8, x, x, None, x, None, 0, F16) == 0
    assert (x == 0).all()


def test_values_stay_with_their_row_and_feature(hv):
    """NaN and infinity in a row, a feature's weights, a bias or a residual reach their own outputs alone."""
    counts, N, K = [40, 30], 264, 136
    A, B, bias, residual = rand((70, K), torch.float16, 1), rand((2, N, K), torch.float16, 2), rand((2, N), torch.float16, 3), rand((70, N), torch.float16, 4)
    A[5, 3], B[0, 17, 9], bias[1, 40], residual[60, 41] = float("nan"), float("inf"), float("nan"), float("inf")
    C = torch.zeros(70, N, dtype=torch.float16, device="cuda")
    pts.gemm_run_linear(hv, 70, 2, N, K, A, B, bias, residual, offsets_of(counts), C, None, pts.GEMM_ACT_NONE, F16)
    bad = torch.zeros(70, N, dtype=torch.bool, device="cuda")
    bad[5], bad[:40, 17], bad[40:, 40], bad[60, 41] = True, True, True, True
    assert torch.equal(~torch.isfinite(C), bad)


def test_hostile_offsets(hv):
    """Offsets that go back and forth or lie outside the rows lead nowhere outside the arrays."""
    rows, N, K = 50, 128, 64
    A, B, residual = rand((rows, K), torch.float16, 1), rand((4, N, K), torch.float16, 2), rand((rows, N), torch.float16, 3)
    for off in ([0, 90, -4, 60, 20], [40, 10, 30, 20, 1 << 30], [-9, -8, -7, -6, -5]):
        buf = torch.full((3, rows, N), 7.0, dtype=torch.float16, device="cuda")
        pts.gemm_run_linear(hv, rows, 4, N, K, A, B, None, residual, torch.tensor(off, dtype=torch.int32, device="cuda"), buf[1], None, 1, F16)
        grad = torch.full((3, rows, N), 7.0, dtype=torch.float16, device="cuda")
        pts.gemm_linear_grad(hv, rows, 4, N, A.new_zeros(rows, N), residual, torch.tensor(off, dtype=torch.int32, device="cuda"), grad[1],
                             torch.zeros(4, N, device="cuda"), 1, F16)
        for b in (buf, grad):
            assert (b[0] == 7.0).all() and (b[2] == 7.0).all()


# ---- gradient --------------------------------------------------------------------

GRAD = [([1], 0, 16), ([5, 0, 3], 2, 272), ([0, 0, 40, 1, 0], 0, 128), ([300, 0, 1, 257, 128], 31, 528), ([1025, 63], 0, 256), ([3] * 45, 0, 144),
        ([2500], 0, 48), ([3000, 10], 5, 1040), ([777], 0, 4112)]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES)
@pytest.mark.parametrize("gated", [0, GATED], ids=["plain", "gated"])
@pytest.mark.parametrize("case", range(len(GRAD)))
def test_linear_grad(h, case, gated, dtype):
    counts, spare, N = GRAD[case]
    N += 8 * (case % 2)
    rows, E, all_ = sum(counts) + spare, len(counts), N * (2 if gated else 1)
    dC, Z = rand((rows, N), TORCH[dtype], 1), rand((rows, all_), TORCH[dtype], 2, 2.0)
    Z[0, 0], Z[0, 1], Z[0, 2] = 0.0, 30.0, -30.0
    dC[sum(counts):], Z[sum(counts):] = float("nan"), float("inf")
    for act in range(6):
        dZ = torch.full((rows + 1, all_), 7.0, dtype=TORCH[dtype], device="cuda")
        dbias = torch.full((E + 1, all_), 7.0, device="cuda") if act != 1 else None
        off = None if E == 1 and act % 2 else offsets_of(counts)
        pts.gemm_linear_grad(h, rows if off is not None else sum(counts), E, N, dC, Z, off, dZ, dbias, act | gated, dtype)
        for e, r in spans(counts):
            d, z = dC[r].double(), Z[r].double()
            a, s, sa = ref.act(act, z[:, :N])
            want, err = d * s, d.abs() * sa * 2 * ref.EPS_ACT
            if gated:
                want = torch.cat([want * z[:, N:], d * a], 1)
                err = torch.cat([err * z[:, N:].abs(), d.abs() * a.abs() * 2 * ref.EPS_ACT], 1)
            ref.close(dZ[r], want, err, ("dZ", act, e))
            if dbias is not None:
                ref.close(dbias[e], want.sum(0), err.sum(0) + want.shape[0] * 2.0 ** -23 * want.abs().sum(0), ("dbias", act, e))
        assert (dZ[sum(counts):] == 7.0).all() and (dbias is None or (dbias[E] == 7.0).all())


@pytest.mark.parametrize("act", range(6), ids=ref.ACTS)
@pytest.mark.parametrize("gated", [0, GATED])
def test_gradient_is_that_of_the_forward_form(h, act, gated):
    """Against differences of the 64-bit forward form: (f(z + t) - f(z - t)) / 2t is off by t^2 f'''/6 <= 2^-20 (t = 2^-10, |f'''| < 6)
    and by f's rounding, 2^-52 |f| / t; relu and relu^2 are not differentiable at 0, so z stays away from it."""
    N, t = 64, 2.0 ** -10
    z = rand((9, N * (2 if gated else 1)), torch.float16, 3, 2.0)
    z = torch.where(z.abs() < 0.01, torch.ones_like(z), z)
    dC, dZ = torch.ones(9, N, dtype=torch.float16, device="cuda"), torch.zeros_like(z)
    pts.gemm_linear_grad(h, 9, 1, N, dC, z, None, dZ, None, act | gated, F16)
    for half in range(2 if gated else 1):
        step = torch.zeros_like(z, dtype=torch.float64)
        step[:, half * N:(half + 1) * N] = t
        f = lambda v: ref.hidden(act | gated, v, 0 * v)[0]  # noqa: E731
        want = (f(z.double() + step) - f(z.double() - step)) / (2 * t)
        scale = 1.0 + z.double()[:, N:].abs() if gated else 1.0
        ref.close(dZ[:, half * N:(half + 1) * N], want, (2.0 ** -20 + 4 * ref.EPS_ACT * (1.0 + z.double()[:, :N].abs())) * scale, half)


def test_dbias_repeats_itself_and_is_zero_without_rows(h):
    dC, Z = rand((5000, 1024), torch.bfloat16, 1), rand((5000, 1024), torch.bfloat16, 2)
    off, got = offsets_of([0, 5000, 0]), []
    for _ in range(3):
        dZ, dbias = torch.zeros_like(Z), torch.full((3, 1024), float("nan"), device="cuda")
        pts.gemm_linear_grad(h, 5000, 3, 1024, dC, Z, off, dZ, dbias, 5, BF16)
        got.append((dZ, dbias))
    assert all(torch.equal(a, b) for g in got[1:] for a, b in zip(g, got[0]))
    assert (got[0][1][[0, 2]] == 0).all()
    dbias = torch.full((2, 16), float("nan"), device="cuda")
    pts.gemm_linear_grad(h, 0, 2, 16, None, None, offsets_of([0, 0]), None, dbias, 0, BF16)
    assert (dbias == 0).all()


# ---- as they are used ---------------------------------------------------------------


def test_a_graph_follows_new_values(h):
    """Captured once (after a first call), replayed under other rows, counts and residuals."""
    E, N, K, rows = 3, 264, 136, 90
    A, B, residual = (torch.zeros(s, dtype=torch.float16, device="cuda") for s in ((rows, K), (E, N, K), (rows, N)))
    off, C, Z = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(rows, N, dtype=torch.float16, device="cuda"), torch.zeros(rows, N, dtype=torch.float16, device="cuda")
    dC, dZ, dbias = rand((rows, N), torch.float16, 9), torch.zeros(rows, N, dtype=torch.float16, device="cuda"), torch.zeros(E, N, device="cuda")

    def step(s):
        pts.gemm_run_linear(h, rows, E, N, K, A, B, None, residual, off, C, Z, 5, F16, stream=s)
        pts.gemm_linear_grad(h, rows, E, N, dC, Z, off, dZ, dbias, 5, F16, stream=s)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    for seed, counts in ((1, [30, 60, 0]), (2, [1, 0, 80]), (3, [0, 0, 0])):
        A.copy_(rand((rows, K), torch.float16, seed))
        B.copy_(rand((E, N, K), torch.float16, seed + 10, 0.1))
        residual.copy_(rand((rows, N), torch.float16, seed + 20))
        off.copy_(offsets_of(counts))
        graph.replay()
        torch.cuda.synchronize()
        for e, r in spans(counts):
            (c, dc), (z, dz) = ref.linear(5, A[r], B[e], None, residual[r])
            ref.close(C[r], c, dc)
            ref.close(Z[r], z, dz)
            _, slope, sa = ref.act(5, Z[r].double())
            ref.close(dbias[e], (dC[r].double() * slope).sum(0), ((dC[r].double().abs() * sa).sum(0)) * (2 * ref.EPS_ACT + rows * 2.0 ** -23))


HANDLES = {"auto": {}, "single": dict(cta_group=1), "pair": dict(cta_group=2), "pair2": dict(cta_group=2, max_clusters=2)}


@pytest.mark.parametrize("opts", HANDLES)
@pytest.mark.parametrize("counts,N,K,load", [([5, 0, 70], 272, 128, 0), ([40], 144, 200, 0), ([300, 33], 528, 208, 1), ([700, 90], 1008, 1040, 5), ([1], 1024, 4096, 3)])
@pytest.mark.parametrize("act,keep", [(1, False), (1, True), (GATED, True)])
def test_a_wait_that_runs_out(opts, counts, N, K, load, act, keep):
    """A stage load that does not come in full: reported, every residual box that was asked for lands, and the next call is exact."""
    rows, E, all_ = sum(counts), len(counts), N * (2 if act & GATED else 1)
    gen = torch.Generator().manual_seed(2)
    ints = lambda *s: torch.randint(-1, 2, s, generator=gen).half().cuda()  # noqa: E731
    A, B, residual, off = ints(rows, K) * (torch.rand(rows, K, generator=gen) < 0.05).cuda(), ints(E, all_, K), ints(rows, N), offsets_of(counts)
    z = torch.cat([A[r].double() @ B[e].double().T for e, r in spans(counts)])
    want = z[:, :N] * z[:, N:] if act & GATED else z.clamp(min=0)
    for flags in (pts.GEMM_DEBUG_FAULT_SKIP_TMA, 0):
        h = pts.gemm_create(0, pts.make_opts(debug_flags=flags, fault_arg=load, timeout_ns=20_000_000, **HANDLES[opts]))
        C, Z = torch.zeros(rows, N, dtype=torch.float16, device="cuda"), torch.zeros(rows, all_, dtype=torch.float16, device="cuda")
        pts.gemm_run_linear(h, rows, E, N, K, A, B, None, residual, off, C, Z if keep else None, act, F16)
        st, dev = pts.gemm_check(h)
        pts.gemm_destroy(h)
        if flags:
            assert st == pts.gemm.GEMM_ERR_TIMEOUT and dev >> 24 == 1
    assert st == 0 and torch.equal(C.double(), want + residual.double())


# ---- extremes -----------------------------------------------------------------------

EXTREMES = [-float("inf"), -3e38, -1e30, -1e10, -65504.0, -5000.0, -300.0, -90.0, -60.0, -44.0, -41.0, -20.0, -6.7, -0.0, 0.0, 2.0 ** -20, 5.0, 20.0, 90.0,
            5000.0, 65504.0, 1e10, 1e18]


def extreme(dtype, N, seed):
    """N values, each of EXTREMES next to each other one sometimes; f: their activation in 64 bits, whose limit at -infinity is 0."""
    x = torch.tensor(EXTREMES)
    x = x[(x.abs() <= torch.finfo(dtype).max) | torch.isinf(x)]
    return x[torch.randint(0, len(x), (N,), generator=torch.Generator().manual_seed(seed))].to(dtype).cuda()


def at_limits(code, z):
    a, s, sa = ref.act(code, z.double().clamp(min=-1e300))
    return torch.where(torch.isnan(a), 0.0, a), torch.where(torch.isnan(s), (z > 0).double(), s), torch.where(torch.isnan(sa), (z > 0).double(), sa)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES)
@pytest.mark.parametrize("rows,K", [(1, 16), (1, 8192), (30, 16), (12, 4096), (300, 16)])
@pytest.mark.parametrize("code", range(1, 6), ids=ref.ACTS[1:])
def test_extreme_sums(hv, code, rows, K, dtype):
    """Sums from -infinity up to 1e18 (the bias; the operands are 0): the activation's limits, without a NaN, beside a NaN."""
    N, t = 272, TORCH[dtype]
    A, B = torch.zeros(rows, K, dtype=t, device="cuda"), torch.zeros(2 * N, K, dtype=t, device="cuda")
    for gated in (0, GATED):
        bias = torch.cat([extreme(t, N, 1), torch.full((N,), -0.75, dtype=t, device="cuda")])[None, :N * (2 if gated else 1)].contiguous()
        bias[0, 5] = float("nan")
        A[rows // 2, 3] = float("nan") if rows > 1 else 0.0
        C = torch.zeros(rows, N, dtype=t, device="cuda")
        pts.gemm_run_linear(hv, rows, 1, N, K, A, B, bias, None, None, C, None, code | gated, dtype)
        if rows > 1:
            assert torch.isnan(C[rows // 2]).all()
            C[rows // 2] = C[0]
        a = at_limits(code, bias[0, :N])[0] * (-0.75 if gated else 1.0)
        assert torch.isnan(C[:, 5]).all()
        a = a.to(t).double().expand(rows, N).clone()   # (rounded: what overflows is infinite on both sides)
        a[:, 5], C[:, 5] = 0.0, 0.0
        same = C.double() == a
        assert (same | ((C.double() - a).abs() <= 2 * ref.U[t] * a.abs() + 2 * ref.EPS_ACT * a.abs() + ref.TINY)).all()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES)
@pytest.mark.parametrize("code", range(1, 6), ids=ref.ACTS[1:])
def test_extreme_gradients(h, code, dtype):
    rows, N, t = 9, 272, TORCH[dtype]
    for gated in (0, GATED):
        g = torch.stack([extreme(t, N, r) for r in range(rows)])
        Z = torch.cat([g, torch.full_like(g, -0.75)], 1)[:, :N * (2 if gated else 1)].contiguous()
        dC, dZ = torch.full_like(g, 0.5), torch.zeros_like(Z)
        dC[3, 7], Z[4, 8] = float("nan"), float("nan")
        pts.gemm_linear_grad(h, rows, 1, N, dC, Z, None, dZ, None, code | gated, dtype)
        a, s, sa = at_limits(code, g)
        want = torch.cat([s * 0.5 * -0.75, a * 0.5], 1) if gated else s * 0.5
        err = 2 * ref.EPS_ACT * (torch.cat([sa * 0.5 * 0.75, a.abs() * 0.5], 1) if gated else sa * 0.5)
        want = want.to(t).double()   # (rounded: what overflows is infinite on both sides)
        err = torch.where(torch.isinf(want), 0.0, err)
        for half in (dZ[:, :N], want[:, :N], dZ[:, N:], want[:, N:]):
            if half.shape[1]:
                if half.dtype == t and code > 2:   # (of relu the slope at NaN is 0)
                    assert torch.isnan(half[[3, 4], [7, 8]]).all()
                half[[3, 4], [7, 8]] = 0.0
        same = dZ.double() == want
        assert (same | ((dZ.double() - want).abs() <= 2 * ref.U[t] * want.abs() + 2 * err + ref.TINY)).all(), code
