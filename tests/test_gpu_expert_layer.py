"""A whole layer of experts for a few tokens against the same layer token by token in 64 bits (layer_reference.py)."""
import pytest
import torch

import layer_reference as ref
import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu

F16, BF16 = pts.GEMM_F16, pts.GEMM_BF16
TORCH = {F16: torch.float16, BF16: torch.bfloat16}
GATED = pts.GEMM_ACT_GATED


@pytest.fixture(scope="module")
def h():
    h = pts.gemm_create(0)
    yield h
    st, dev = pts.gemm_check(h)
    pts.gemm_destroy(h)
    assert st == 0, f"device status {dev:#x}"


def rand(shape, dtype, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def weights_of(E, D, H, act, dtype, bias):
    all_ = H * (2 if act & GATED else 1)
    up, down = rand((E, all_, D), dtype, 1, 1 / max(D, 1) ** 0.5), rand((E, D, H), dtype, 2, 1 / max(H, 1) ** 0.5)
    return up, rand((E, all_), dtype, 3) if bias else None, down, rand((E, D), dtype, 4) if bias else None


def run(h, T, k, E, D, H, act, dtype, ids, bias=True, residual=True, in_place=False, seed=5):
    t = TORCH[dtype]
    up, up_bias, down, down_bias = weights_of(E, D, H, act, t, bias)
    x, res = rand((T, D), t, seed), rand((T, D), t, seed + 1) if residual else None
    w = torch.randn(T, k, generator=torch.Generator().manual_seed(seed + 2)).cuda()
    Hs = torch.full((T * k + 1, H), 7.0, dtype=t, device="cuda")
    Y = torch.full((T + 1, D), 7.0, dtype=t, device="cuda")
    if in_place:
        Y[:T] = res
    pts.gemm_expert_layer(h, T, k, E, D, H, x, ids, w, up, up_bias, down, down_bias, Y if in_place else res, Hs, Y, act, dtype)
    y, err = ref.layer(act, x, ids.cpu(), w.cpu(), up, up_bias, down, down_bias, res, t)
    ref.close(Y[:T], y, err)
    assert (Y[T] == 7.0).all() and (Hs[T * k] == 7.0).all()
    return Y[:T]


def choose(T, k, E, seed=8, lo=-1):
    return torch.randint(lo, E + 1, (T, k), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()


# tokens, top_k, experts, dim, hidden
SIZES = [(1, 1, 1, 8, 8), (1, 2, 8, 136, 264), (2, 3, 5, 520, 72), (7, 2, 4, 1032, 272), (16, 2, 8, 256, 512), (17, 1, 2, 264, 136), (33, 4, 64, 128, 264),
         (64, 8, 16, 72, 144), (64, 1, 1, 272, 96), (13, 4, 32, 512, 1024), (5, 6, 1024, 24, 40), (3, 2, 4, 4104, 16), (3, 2, 4, 16, 4104), (1, 64, 3, 80, 88)]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_layer(h, case, dtype):
    T, k, E, D, H = SIZES[case]
    ids = choose(T, k, E)   # some outside the experts, some twice
    for i, act in enumerate((5 | GATED, 2, 3 | GATED, 4, 0, 1 | GATED)):
        if (i + case) % 2 == 0 or D * H < 40000:
            run(h, T, k, E, D, H, act, dtype, ids, bias=i % 2 == 0, residual=i % 3 != 1)


def test_residual_in_place(h):
    run(h, 9, 2, 4, 136, 72, 5 | GATED, BF16, choose(9, 2, 4), in_place=True)


@pytest.mark.parametrize("T,k", [(1, 1), (40, 3), (64, 8)])
def test_all_tokens_choose_one_expert(h, T, k):
    """Blocks of 16 of one expert's tokens, the same expert named top_k times."""
    run(h, T, k, 6, 264, 152, 5 | GATED, BF16, torch.full((T, k), 4, dtype=torch.int32, device="cuda"))


def test_no_token_has_an_expert(h):
    ids = torch.tensor([[-1, 99], [1 << 30, -1 << 31], [4, -5]], dtype=torch.int32, device="cuda")
    Y = run(h, 3, 2, 4, 136, 72, 5, BF16, ids, residual=True)
    assert torch.equal(Y, rand((3, 136), torch.bfloat16, 6))
    assert (run(h, 3, 2, 4, 136, 72, 5, BF16, ids, residual=False) == 0).all()


def test_without_hidden_features(h):
    """hidden = 0: the residual and the down bias alone."""
    run(h, 5, 2, 3, 40, 0, 0, F16, choose(5, 2, 3))


def test_values_stay_with_the_tokens_that_meet_them(h):
    T, E, D, H = 20, 4, 136, 264
    ids = (torch.arange(T, dtype=torch.int32, device="cuda") % 4)[:, None].contiguous()
    w, t = torch.ones(T, 1, device="cuda"), torch.float16
    up, _, down, _ = weights_of(E, D, H, GATED | 5, t, False)
    x = rand((T, D), t, 5)
    clean, Hs = torch.zeros(T, D, dtype=t, device="cuda"), torch.zeros(T, H, dtype=t, device="cuda")
    pts.gemm_expert_layer(h, T, 1, E, D, H, x, ids, w, up, None, down, None, None, Hs, clean, 5 | GATED, F16)
    x[6, 3], down[1, 17, 5], up[3, 9, 2] = float("nan"), float("inf"), float("nan")
    Y = torch.zeros_like(clean)
    pts.gemm_expert_layer(h, T, 1, E, D, H, x, ids, w, up, None, down, None, None, Hs, Y, 5 | GATED, F16)
    bad = torch.zeros(T, D, dtype=torch.bool, device="cuda")
    bad[6], bad[1::4, 17], bad[3::4] = True, True, True
    assert torch.equal(~torch.isfinite(Y), bad) and torch.equal(Y[~bad], clean[~bad])


def test_an_unchosen_expert_is_not_read(h):
    """NaN everywhere in experts that no token chose."""
    T, E, D, H, t = 6, 5, 72, 88, torch.bfloat16
    up, _, down, _ = weights_of(E, D, H, 2, t, False)
    ids = torch.tensor([[1, 3]] * T, dtype=torch.int32, device="cuda")
    up[[0, 2, 4]], down[[0, 2, 4]] = float("nan"), float("nan")
    x, w = rand((T, D), t, 5), torch.ones(T, 2, device="cuda")
    Y, Hs = torch.zeros(T, D, dtype=t, device="cuda"), torch.full((T * 2, H), float("nan"), dtype=t, device="cuda")
    pts.gemm_expert_layer(h, T, 2, E, D, H, x, ids, w, up, None, down, None, None, Hs, Y, 2, BF16)
    assert torch.isfinite(Y).all()


def test_small_integers_are_exact_and_it_repeats_itself(h):
    T, k, E, D, H = 30, 2, 6, 264, 136
    gen = torch.Generator().manual_seed(1)
    ints = lambda *s: torch.randint(-1, 2, s, generator=gen).half().cuda()  # noqa: E731
    x, up, down = ints(T, D), ints(E, H, D) * (torch.rand(E, H, D, generator=gen) < 0.1).half().cuda(), ints(E, D, H) * (torch.rand(E, D, H, generator=gen) < 0.1).half().cuda()
    ids, w = torch.randint(0, E, (T, k), generator=gen, dtype=torch.int32).cuda(), torch.ones(T, k, device="cuda")
    Hs = torch.zeros(T * k, H, dtype=torch.float16, device="cuda")
    got = [torch.zeros(T, D, dtype=torch.float16, device="cuda") for _ in range(3)]
    for Y in got:
        pts.gemm_expert_layer(h, T, k, E, D, H, x, ids, w, up, None, down, None, None, Hs, Y, 1, F16)
    want = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            want[t] += down[e].double() @ (up[e].double() @ x[t].double()).clamp(min=0)
    assert want.abs().max() < 2048 and all(torch.equal(Y.double(), want) for Y in got)


def test_routing_layer_and_the_calls_around_them(h):
    """As a decoding step uses them, queued without waiting and captured: the logits' product, the choice, the layer; each with new
    values, on the same buffers, against the layer made of the single operators."""
    T, k, E, D, H, t = 11, 3, 12, 136, 264, torch.bfloat16
    up, up_bias, down, down_bias = weights_of(E, D, H, 5 | GATED, t, True)
    gate = rand((1, 16, D), t, 20, 0.3)   # (of 16 rows 12 are experts; the others are masked by their bias)
    gate_bias = torch.zeros(1, 16, dtype=t, device="cuda")
    gate_bias[0, 12:] = float("-inf")
    x, logits = torch.zeros(T, D, dtype=t, device="cuda"), torch.zeros(T, 16, dtype=t, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, w, off, row_of, src_of = i32(T, k), torch.zeros(T, k, device="cuda"), i32(E + 1), i32(T, k), i32(T * k)
    Hs, y = torch.zeros(T * k, H, dtype=t, device="cuda"), torch.zeros(T, D, dtype=t, device="cuda")
    xs, a, ys, y2 = (torch.zeros(n, c, dtype=t, device="cuda") for n, c in ((T * k, D), (T * k, H), (T * k, D), (T, D)))

    def step(s):
        pts.gemm_run_linear(h, T, 1, 16, D, x, gate, gate_bias, None, None, logits, None, pts.GEMM_ACT_NONE, BF16, stream=s)
        pts.gemm_expert_route(h, T, k, 16, logits, ids, w, pts.GEMM_ROUTE_SELECTED, BF16, stream=s)
        pts.gemm_expert_layer(h, T, k, E, D, H, x, ids, w, up, up_bias, down, down_bias, x, Hs, y, 5 | GATED, BF16, stream=s)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    for seed in range(4):
        x.copy_(rand((T, D), t, 30 + seed))
        if seed % 2:
            graph.replay()
        else:
            with torch.cuda.stream(s):
                step(s)
                step(s)
        torch.cuda.synchronize()
        assert ((ids >= 0) & (ids < E)).all()
        want, err = ref.layer(5 | GATED, x, ids.cpu(), w.cpu(), up, up_bias, down, down_bias, x, t)
        ref.close(y, want, err)
        pts.gemm_expert_sort(h, T, k, E, ids, off, row_of, src_of)
        pts.gemm_expert_gather(h, T, k, D, x, row_of, xs, BF16)
        pts.gemm_run_linear(h, T * k, E, H, D, xs, up, up_bias, None, off, a, None, 5 | GATED, BF16)
        pts.gemm_run_linear(h, T * k, E, D, H, a, down, down_bias, None, off, ys, None, 0, BF16)
        pts.gemm_expert_combine(h, T, k, D, ys, row_of, w, y2, BF16)
        # (ys and y2 are rounded once more each than in the layer)
        assert float((y2.double() + x.double() - y.double()).norm()) <= 2.0 ** -7 * float(y.double().norm())


def test_layers_back_to_back_see_their_own_values(h):
    """Queued one after another on the same buffers, with other ids and weights each time, written by the calls before."""
    T, k, E, D, n, t = 8, 2, 4, 64, 40, torch.float16
    up = torch.stack([torch.eye(D) * (e + 1) for e in range(E)]).half().cuda()
    down = torch.eye(D).expand(E, D, D).half().contiguous().cuda()
    logits = torch.randn(n, T, E, generator=torch.Generator().manual_seed(2)).cuda()
    x = torch.randint(0, 4, (T, D), generator=torch.Generator().manual_seed(3)).half().cuda()
    ids, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    ones = torch.ones(T, k, device="cuda")
    Hs, y = torch.zeros(T * k, D, dtype=t, device="cuda"), torch.zeros(n, T, D, dtype=t, device="cuda")
    torch.cuda.synchronize()
    for i in range(n):
        pts.gemm_expert_route(h, T, k, E, logits[i], ids, w, pts.GEMM_ROUTE_SELECTED, pts.GEMM_F32)
        pts.gemm_expert_layer(h, T, k, E, D, D, x, ids, ones, up, None, down, None, None, Hs, y[i], 1, F16)
    torch.cuda.synchronize()
    factor = (logits.topk(k, dim=2).indices + 1).sum(2).double()
    assert torch.equal(y.double(), factor[..., None] * x.double())


def test_sizes_that_are_refused(h):
    x, ids, w = torch.zeros(1 << 16, dtype=torch.float16, device="cuda"), torch.zeros(4096, dtype=torch.int32, device="cuda"), torch.zeros(4096, device="cuda")
    call = lambda T, k, E, D, H, act=0, X=x: pts.gemm_expert_layer(h, T, k, E, D, H, X, ids, w, x, None, x, None, None, x, x, act, F16)  # noqa: E731
    assert call(1, 1, 1, 8, 8) == 0
    for bad in ((65, 1, 1, 8, 8), (64, 9, 1, 8, 8), (1, 513, 1, 8, 8), (1, 1, 1025, 8, 8), (1, 1, 1, 12, 8), (1, 1, 1, 8, 4), (1, 0, 1, 8, 8), (-1, 1, 1, 8, 8),
                (1, 1, 1, 8, 8, 6), (1, 1, 1, 8, 8, -1), (1, 1, 1, 8, 8, 0x20)):
        with pytest.raises(pts.GemmError) as err:
            call(*bad)
        assert err.value.status == 1, bad
    with pytest.raises(pts.GemmError):
        call(1, 1, 1, 8, 8, 0, x[1:])   # not 16-byte aligned
    assert call(0, 1, 1, 8, 8) == 0 and call(1, 1, 1, 0, 8) == 0


@pytest.mark.parametrize("T,k,E,D,H,act", [(64, 8, 16, 520, 1048, 5 | GATED), (40, 8, 6, 1032, 520, 3 | GATED), (64, 8, 36, 72, 7600, 2), (33, 4, 1, 2056, 1000, 4),
                                           (64, 2, 3, 5160, 552, 1 | GATED), (20, 3, 4, 4096, 1032, 0)])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
def test_many_tokens_an_expert(h, T, k, E, D, H, act, dtype):
    """Blocks of 32 tokens, teams of 2, 4 and 8 warps, ragged; ids outside the experts and twice."""
    run(h, T, k, E, D, H, act, dtype, choose(T, k, E))
    run(h, T, k, E, D, H, act, dtype, torch.full((T, k), E - 1, dtype=torch.int32, device="cuda"), bias=False, in_place=True)
