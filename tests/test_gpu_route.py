"""A router's choice and its gradient against plain forms in 64 bits.

Ids have to be equal.  Weights: the scores are exact or, of the sigmoid, off by 2 steps of 2^-24 of themselves and of 1; exp and
the division are off by 2 steps each, the sum of n of them by n: (2 |u_max - u| + 2 |u| + n + 16) 2^-24 of the weight covers it."""
import pytest
import torch

import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu

TYPES = {"f32": (pts.GEMM_F32, torch.float32, 2.0 ** -24), "f16": (pts.GEMM_F16, torch.float16, 2.0 ** -11), "bf16": (pts.GEMM_BF16, torch.bfloat16, 2.0 ** -8)}
SELECTED, ALL, SIGMOID = pts.GEMM_ROUTE_SELECTED, pts.GEMM_ROUTE_ALL, pts.GEMM_ROUTE_SIGMOID
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def h():
    h = pts.gemm_create(0)
    yield h
    pts.gemm_destroy(h)


def chosen(logits, k):
    """ids (-1 where nothing is left) on the host: a stable sort keeps the lower index first, -0 and 0 are equal."""
    x = torch.where(torch.isnan(logits), -INF, logits.double())
    v, ids = torch.sort(x, dim=1, descending=True, stable=True)
    return torch.where(v[:, :k] > -INF, ids[:, :k], -1)


def weights(logits, ids, mode):
    """(w of the chosen, w of all experts) in 64 bits; differentiable."""
    x = logits.clamp(max=torch.finfo(torch.float32).max)
    u = torch.nn.functional.logsigmoid(x) if mode == SIGMOID else x
    pool = ~torch.isnan(x) & (x > -INF)
    if mode != ALL:
        inside = torch.zeros_like(pool).scatter_(1, ids.clamp(min=0), True)
        inside[(ids < 0).all(1)] = False
        pool = pool & inside
    p = torch.softmax(torch.where(pool, u, torch.full_like(u, -1e300)), dim=1) * pool
    return torch.where(ids >= 0, torch.gather(p, 1, ids.clamp(min=0)), 0.0), p


def make(tokens, experts, kind, seed, spread=2.0):
    x = (torch.randn(tokens, experts, generator=torch.Generator().manual_seed(seed)) * spread).to(TYPES[kind][1])
    if tokens > 3:   # masked experts, padded tokens, one left, NaN
        x[torch.rand(tokens, experts, generator=torch.Generator().manual_seed(seed + 1)) < 0.2] = -INF
        x[1] = -INF
        x[2] = -INF
        x[2, experts // 2] = 0.5
        x[3, 0] = NAN
    return x


SIZES = [(1, 1, 1), (1, 2, 2), (5, 8, 2), (16, 64, 4), (33, 31, 31), (7, 33, 8), (300, 128, 8), (64, 250, 6), (9, 257, 32), (130, 1024, 8), (5, 1000, 1), (2049, 16, 3)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("mode", [SELECTED, ALL, SIGMOID], ids=["selected", "all", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,k", SIZES)
def test_route_and_gradient(h, tokens, experts, k, mode, kind):
    code, dtype, u = TYPES[kind]
    x = make(tokens, experts, kind, tokens + experts)
    want = chosen(x, k)
    ids = torch.full((tokens + 1, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((tokens + 1, k), 9.0, device="cuda")
    xd = x.cuda()
    pts.gemm_expert_route(h, tokens, k, experts, xd, ids, w, mode, code)
    assert torch.equal(ids[:tokens].cpu().long(), want) and (ids[tokens] == -9).all() and (w[tokens] == 9.0).all()
    leaf = x.double().requires_grad_()
    w64, p64 = weights(leaf, want, mode)
    n = experts if mode == ALL else k
    reach = 2 * 2 * 8 * 2.0   # |u| and |u_max - u| of values within 8 spreads
    assert ((w[:tokens].cpu().double() - w64).abs() <= (4 * reach + n + 16) * 2.0 ** -24 * w64 + 1e-37).all()
    if mode != ALL:
        full = (want >= 0).any(1)
        assert ((w[:tokens].cpu().double().sum(1) - 1.0).abs()[full] <= k * 2.0 ** -22).all()

    dw = torch.randn(tokens, k, generator=torch.Generator().manual_seed(7))
    dl = torch.full((tokens + 1, experts), 9.0, dtype=dtype, device="cuda")
    pts.gemm_expert_route_grad(h, tokens, k, experts, xd, ids, dw.cuda(), dl, mode, code)
    (g,) = torch.autograd.grad((w64 * dw.double()).sum(), leaf)
    g = torch.where(torch.isnan(x) | (x == -INF), 0.0, g)
    # p (d - sum w d): p is off as above, the difference by n + 4 roundings of its terms
    size = p64.detach() * (dw.double().abs().max(1, keepdim=True).values * 2)
    err = (4 * reach + 2 * n + 40) * 2.0 ** -24 * size
    assert ((dl[:tokens].cpu().double() - g).abs() <= u * g.abs() + 2 * err + 2.0 ** -25).all()
    assert (dl[tokens] == 9.0).all()


@pytest.mark.parametrize("mode", [SELECTED, ALL, SIGMOID])
def test_gradient_against_differences(h, mode):
    """(f(l + t) - f(l - t)) / 2t, t = 2^-8, is off by t^2 / 6 times a third derivative below 2 of each of the weights, times dw."""
    T, E, k, t = 3, 12, 4, 2.0 ** -8
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(5)).double() * 2
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(6))
    ids = chosen(x.float(), k)
    dl = torch.zeros(T, E, device="cuda")
    pts.gemm_expert_route_grad(h, T, k, E, x.float().cuda(), ids.int().cuda(), dw.cuda(), dl, mode, pts.GEMM_F32)
    for e in range(E):
        step = torch.zeros_like(x)
        step[:, e] = t
        f = lambda v: (weights(v, ids, mode)[0] * dw.double()).sum(1)  # noqa: E731
        diff = (f(x.float().double() + step) - f(x.float().double() - step)) / (2 * t)
        assert ((dl[:, e].cpu().double() - diff).abs() <= t * t / 3 * dw.double().abs().sum(1) + 2.0 ** -18).all()


@pytest.mark.parametrize("kind", TYPES)
def test_equal_logits_go_to_the_lower_index(h, kind):
    code, dtype, _ = TYPES[kind]
    gen = torch.Generator().manual_seed(3)
    x = torch.randint(-1, 2, (500, 70), generator=gen).to(dtype)
    x[torch.rand(500, 70, generator=gen) < 0.3] *= -0.0   # zeros of both signs
    x[0], x[1] = 0.0, -INF
    ids, w = torch.zeros(500, 9, dtype=torch.int32, device="cuda"), torch.zeros(500, 9, device="cuda")
    pts.gemm_expert_route(h, 500, 9, 70, x.cuda(), ids, w, SELECTED, code)
    assert torch.equal(ids.cpu().long(), chosen(x, 9))
    assert torch.equal(ids[0].cpu(), torch.arange(9, dtype=torch.int32)) and (w[0] - 1 / 9).abs().max() < 1e-7
    assert (ids[1] == -1).all() and (w[1] == 0).all()


def test_infinite_and_extreme_logits(h):
    big = torch.finfo(torch.float32).max
    x = torch.tensor([[INF, 0.0, INF, -INF], [big, INF, -big, 1.0], [-big, -big, -INF, NAN], [-200.0, -300.0, -250.0, -199.0], [NAN, NAN, NAN, NAN]], device="cuda")
    for mode in (SELECTED, ALL, SIGMOID):
        ids, w = torch.zeros(5, 3, dtype=torch.int32, device="cuda"), torch.zeros(5, 3, device="cuda")
        pts.gemm_expert_route(h, 5, 3, 4, x, ids, w, mode, pts.GEMM_F32)
        dl, dw = torch.zeros(5, 4, device="cuda"), torch.ones(5, 3, device="cuda") * torch.tensor([1.0, 2.0, 3.0], device="cuda")
        pts.gemm_expert_route_grad(h, 5, 3, 4, x, ids, dw, dl, mode, pts.GEMM_F32)
        assert ids.tolist() == [[0, 2, 1], [0, 1, 3], [0, 1, -1], [3, 0, 2], [-1, -1, -1]]
        assert torch.isfinite(w).all() and torch.isfinite(dl).all()
        assert (w[:4].sum(1) - 1.0).abs().max() < 1e-6 and (w[4] == 0).all() and (dl[4] == 0).all() and w[2, 2] == 0
        if mode != SIGMOID:   # (of the sigmoid all large ones are 1)
            assert w[0].tolist() == [0.5, 0.5, 0.0] and w[1].tolist() == [0.5, 0.5, 0.0]
        else:   # far below 0 it falls as exp does
            assert (w[3].double().cpu() - torch.softmax(torch.tensor([-199.0, -200.0, -250.0]).double(), 0)).abs().max() < 1e-6


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("experts,k", [(4, 3), (10, 3), (40, 9), (130, 3), (300, 3)])
def test_infinite_and_extreme_16_bit_logits(h, kind, experts, k):
    """Rows of a type's extremes among zeros (masked ones where fewer are wanted), in every kernel: with 8 and 16 lanes and a warp to
    a token, rows that can and cannot be loaded at once, more than 8 choices."""
    code, dtype, _ = TYPES[kind]
    big = torch.finfo(dtype).max
    x = torch.full((5, experts), -INF, dtype=dtype)
    x[0, :4] = torch.tensor([INF, 0.0, INF, -INF], dtype=dtype)
    x[1, :4] = torch.tensor([big, INF, -big, 1.0], dtype=dtype)
    x[2, :4] = torch.tensor([-big, -big, -INF, NAN], dtype=dtype)
    x[3, :4] = torch.tensor([-200.0, -300.0, -250.0, -199.0], dtype=dtype)
    x[4] = NAN
    pad = [-1] * (k - 3)
    want = [[0, 2, 1], [1, 0, 3], [0, 1, -1], [3, 0, 2], [-1, -1, -1]]
    if k > 3:
        want = [[0, 2, 1, -1], [1, 0, 3, 2], [0, 1, -1, -1], [3, 0, 2, 1], [-1] * 4]
        pad = [-1] * (k - 4)
    for mode in (SELECTED, ALL, SIGMOID):
        ids, w = torch.zeros(5, k, dtype=torch.int32, device="cuda"), torch.full((5, k), NAN, device="cuda")
        pts.gemm_expert_route(h, 5, k, experts, x.cuda(), ids, w, mode, code)
        dl, dw = torch.full((5, experts), NAN, dtype=dtype, device="cuda"), torch.arange(1.0, k + 1, device="cuda").expand(5, k).contiguous()
        pts.gemm_expert_route_grad(h, 5, k, experts, x.cuda(), ids, dw, dl, mode, code)
        assert ids.tolist() == [row + pad for row in want]
        assert torch.isfinite(w).all() and torch.isfinite(dl).all()
        assert (w[:4].sum(1) - 1.0).abs().max() < (1e-6 if mode != ALL or k > 3 else 1e-3) and (w[4] == 0).all() and (dl[4] == 0).all()
        if mode != SIGMOID:
            assert w[0, :3].tolist() == [0.5, 0.5, 0.0]
            assert w[1, 0] == 1.0   # (+infinity counts as more than the largest finite value)


def test_ids_that_lead_nowhere_have_no_gradient(h):
    x = torch.randn(4, 8, generator=torch.Generator().manual_seed(1)).cuda()
    x[2, 5] = -INF
    ids = torch.tensor([[1, 99], [-7, 3], [5, 2], [1 << 30, -1 << 31]], dtype=torch.int32, device="cuda")
    fixed = torch.tensor([[1, -1], [-1, 3], [-1, 2], [-1, -1]], dtype=torch.int32, device="cuda")
    dw = torch.randn(4, 2, generator=torch.Generator().manual_seed(2)).cuda()
    for mode in (SELECTED, ALL, SIGMOID):
        a, b = (torch.full((4, 8), 9.0, device="cuda") for _ in range(2))
        pts.gemm_expert_route_grad(h, 4, 2, 8, x, ids, dw, a, mode, pts.GEMM_F32)
        pts.gemm_expert_route_grad(h, 4, 2, 8, x, fixed, dw, b, mode, pts.GEMM_F32)
        assert torch.equal(a, b) and torch.isfinite(a).all()


def test_rows_at_odd_addresses(h):
    """fp16 rows of an odd length, from an odd element on."""
    T, E, k = 50, 37, 5
    buf = torch.randn(T * E + 1, generator=torch.Generator().manual_seed(4)).half()
    x = buf[1:].view(T, E)
    ids, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    dev = buf.cuda()
    pts.gemm_expert_route(h, T, k, E, dev[1:].view(T, E), ids, w, SELECTED, pts.GEMM_F16)
    assert torch.equal(ids.cpu().long(), chosen(x, k))
    out = torch.full((T * E + 2,), 9.0, dtype=torch.float16, device="cuda")
    pts.gemm_expert_route_grad(h, T, k, E, dev[1:].view(T, E), ids, w, out[1:-1].view(T, E), ALL, pts.GEMM_F16)
    assert out[0] == 9.0 and out[-1] == 9.0 and torch.isfinite(out).all()


def test_no_tokens(h):
    assert pts.gemm_expert_route(h, 0, 2, 8, None, None, None, SELECTED, pts.GEMM_F32) == 0
    assert pts.gemm_expert_route_grad(h, 0, 2, 8, None, None, None, None, SELECTED, pts.GEMM_F32) == 0


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("mode", [SELECTED, ALL, SIGMOID], ids=["selected", "all", "sigmoid"])
@pytest.mark.parametrize("experts", [7, 128, 1000])
def test_infinite_dweights_reach_what_depends_on_them(h, experts, mode, kind):
    """A token with infinite or NaN dweights: zeros where a logit was masked or, but for the softmax over all, not chosen; the other
    tokens' gradients are as without it."""
    code, dtype, _ = TYPES[kind]
    x = (torch.randn(6, experts, generator=torch.Generator().manual_seed(5))).to(dtype)
    x[:, 3] = -INF
    ids = chosen(x, 3)
    dw = torch.randn(6, 3, generator=torch.Generator().manual_seed(6))
    got = []
    for bad in (0.0, INF, NAN):
        d = dw.clone()
        if bad:
            d[1, 0], d[4, 2] = bad, bad
        dl = torch.full((6, experts), 9.0, dtype=dtype, device="cuda")
        pts.gemm_expert_route_grad(h, 6, 3, experts, x.cuda(), ids.int().cuda(), d.cuda(), dl, mode, code)
        got.append(dl.cpu())
    free = torch.ones(6, experts, dtype=torch.bool)
    if mode == ALL:
        free[:] = False
    free.scatter_(1, ids, False)
    free[:, 3] = True
    for dl in got[1:]:
        assert (dl[free] == 0).all() and torch.equal(dl[[0, 2, 3, 5]], got[0][[0, 2, 3, 5]])
        assert not torch.isfinite(dl[[1, 4]].gather(1, ids[[1, 4]])).any(1).all()


def test_an_id_that_is_there_twice_adds_up(h):
    x = torch.randn(3, 40, generator=torch.Generator().manual_seed(1)).cuda()
    for mode in (SELECTED, ALL, SIGMOID):
        out = []
        for ids, dw in (([5, 9, 5], [0.5, -2.0, 0.75]), ([5, 9, -1], [1.25, -2.0, 3.0])):
            dl = torch.zeros(3, 40, device="cuda")
            pts.gemm_expert_route_grad(h, 3, 3, 40, x, torch.tensor([ids] * 3, dtype=torch.int32, device="cuda"), torch.tensor([dw] * 3, device="cuda"),
                                       dl, mode, pts.GEMM_F32)
            out.append(dl)
        assert torch.equal(*out)


def test_calls_that_are_refused(h):
    x, ids, w = torch.zeros(4096, device="cuda"), torch.zeros(4096, dtype=torch.int32, device="cuda"), torch.zeros(4096, device="cuda")
    route = lambda T, k, E, mode=0, dtype=pts.GEMM_F32, X=x.data_ptr(), i=ids.data_ptr(), v=w.data_ptr(): pts.gemm_expert_route(h, T, k, E, X, i, v, mode, dtype)  # noqa: E731
    back = lambda T, k, E, mode=0, dtype=pts.GEMM_F32, X=x.data_ptr(), i=ids.data_ptr(), v=w.data_ptr(), o=x.data_ptr(): pts.gemm_expert_route_grad(h, T, k, E, X, i, v, o, mode, dtype)  # noqa: E731
    for f in (route, back):
        assert f(2, 2, 8) == 0
        for bad in ((-1, 2, 8), (2, 0, 8), (2, 9, 8), (2, 33, 64), (2, 2, 0), (2, 2, 1025), (1 << 31, 2, 8), (2, 2, 8, 3), (2, 2, 8, -1), (2, 2, 8, 0, pts.GEMM_E4M3),
                    (2, 2, 8, 0, pts.GEMM_F32, x.data_ptr() + 2), (2, 2, 8, 0, pts.GEMM_F16, x.data_ptr() + 1), (2, 2, 8, 0, pts.GEMM_F32, None),
                    (2, 2, 8, 0, pts.GEMM_F32, x.data_ptr(), ids.data_ptr() + 2), (2, 2, 8, 0, pts.GEMM_F32, x.data_ptr(), ids.data_ptr(), None)):
            with pytest.raises(pts.GemmError) as err:
                f(*bad)
            assert err.value.status == 1, bad
    with pytest.raises(pts.GemmError):
        back(2, 2, 8, 0, pts.GEMM_F32, x.data_ptr(), ids.data_ptr(), w.data_ptr(), x.data_ptr() + 2)
