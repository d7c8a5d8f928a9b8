"""Calls around the products, queued behind kernels of the library that write what they read and let the next one start early: every
array new each time, each of them the last one written in turn, against the same calls one after another."""
import pytest
import torch

import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu

F16, F32, t = pts.GEMM_F16, pts.GEMM_F32, torch.float16
GATED, SILU, SELECTED = pts.GEMM_ACT_GATED, pts.GEMM_ACT_SILU, pts.GEMM_ROUTE_SELECTED


@pytest.fixture(scope="module")
def h():
    h = pts.gemm_create(0)
    yield h
    st, dev = pts.gemm_check(h)
    pts.gemm_destroy(h)
    assert st == 0, f"device status {dev:#x}"


def rand(shape, seed, scale=1.0, dtype=t):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def queued(h, values, call, outputs, times):
    """values: name -> (two or more versions of an array, each a multiple of 16 bytes, the same size); call(arrays) uses the arrays that
    gemm_expert_gather copies them to, as one row of bits."""
    arrays = {name: torch.zeros_like(v[0]) for name, v in values.items()}
    zero = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    names = list(values)

    def go(i):
        for j in range(len(names)):
            name = names[(i + j) % len(names)]
            src, dst = values[name][i % len(values[name])], arrays[name]
            n = src.numel() * src.element_size() // 2
            pts.gemm_expert_gather(h, 1, 1, n, src.view(-1).view(t), zero, dst.view(-1).view(t), F16)
        call(arrays)

    def run(wait):
        out = []
        for i in range(times):
            go(i)
            if wait:
                torch.cuda.synchronize()
            out.append([o.clone() for o in outputs])
        torch.cuda.synchronize()
        return out

    want = run(True)
    assert any(not torch.equal(a, b) for a, b in zip(want[0], want[1]))
    # (without torch's copies in between, whose launches would wait: all calls first, then the outputs of the last)
    for n in range(1, times + 1):
        for i in range(n):
            go(i)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outputs, want[n - 1])), n
    assert all(torch.equal(a, b) for x, y in zip(run(False), want) for a, b in zip(x, y))


@pytest.mark.parametrize("T,k,E,D,H,act", [(8, 2, 4, 64, 64, 1), (1, 2, 8, 1024, 64, SILU | GATED), (4, 2, 8, 2048, 16, SILU | GATED), (16, 4, 8, 512, 1024, 3 | GATED),
                                           (64, 8, 16, 520, 1048, SILU | GATED)])
def test_layer(h, T, k, E, D, H, act):
    """The down kernel reads ids, weights, biases, the residual and its matrices before it waits."""
    all_, n = H * (2 if act & GATED else 1), 3
    each = lambda shape, seed, scale=1.0, dtype=t: [rand(shape, seed + 100 * i, scale, dtype) for i in range(n)]  # noqa: E731
    ids = [torch.randint(0, E, (T, max(k, 4)), generator=torch.Generator().manual_seed(i), dtype=torch.int32).cuda() for i in range(n)]
    values = dict(ids=ids, w=each((T, max(k, 4)), 1, 1.0, torch.float32), x=each((T, D), 2), res=each((T, D), 3), up=each((E, all_, D), 4, D ** -0.5),
                  up_bias=each((E, all_), 5), down=each((E, D, H), 6, H ** -0.5), down_bias=each((E, D), 7))
    Hs, Y = torch.zeros(T * k, H, dtype=t, device="cuda"), torch.zeros(T, D, dtype=t, device="cuda")

    def call(a):
        pts.gemm_expert_layer(h, T, k, E, D, H, a["x"], a["ids"], a["w"], a["up"], a["up_bias"], a["down"], a["down_bias"], a["res"], Hs, Y, act, F16)

    queued(h, values, call, [Y], 10)


@pytest.mark.parametrize("rows,N,K,act", [(1, 1024, 1024, SILU | GATED), (3, 264, 4096, 2), (8, 4096, 256, 0), (24, 1024, 2048, 3), (40, 512, 4096, SILU | GATED), (300, 520, 264, 4),
                                          (24, 19464, 1536, 1), (16, 9736, 1536, SILU | GATED)])
def test_linear_and_its_gradient(h, rows, N, K, act):
    """A few rows, tiles that CTAs share, whole tiles, and a wave and a part, whose second launch does not wait for the first."""
    all_, n = N * (2 if act & GATED else 1), 2
    each = lambda shape, seed, scale=1.0: [rand(shape, seed + 100 * i, scale) for i in range(n)]  # noqa: E731
    values = dict(A=each((rows, K), 1), B=each((1, all_, K), 2, K ** -0.5), bias=each((1, all_), 3), res=each((rows, N), 4))
    C, Z, dZ = (torch.zeros(rows, m, dtype=t, device="cuda") for m in (N, all_, all_))
    db = torch.zeros(1, all_, device="cuda")

    def call(a):
        pts.gemm_run_linear(h, rows, 1, N, K, a["A"], a["B"], a["bias"], a["res"], None, C, Z, act, F16)
        pts.gemm_linear_grad(h, rows, 1, N, C, Z, None, dZ, db, act, F16)

    queued(h, values, call, [C, Z, dZ, db], 8)


@pytest.mark.parametrize("tokens,k,E,dtype", [(16, 4, 64, F32), (300, 8, 128, F16), (40, 12, 1024, F16)])
def test_route_and_its_gradient(h, tokens, k, E, dtype):
    n, kind = 2, torch.float32 if dtype == F32 else t
    values = dict(x=[rand((tokens, E), 1 + i, 2.0, kind) for i in range(n)], dw=[rand((tokens, k), 5 + i, 1.0, torch.float32) for i in range(n)])
    ids, w, dl = torch.zeros(tokens, k, dtype=torch.int32, device="cuda"), torch.zeros(tokens, k, device="cuda"), torch.zeros(tokens, E, dtype=kind, device="cuda")

    def call(a):
        pts.gemm_expert_route(h, tokens, k, E, a["x"], ids, w, SELECTED, dtype)
        pts.gemm_expert_route_grad(h, tokens, k, E, a["x"], ids, a["dw"], dl, SELECTED, dtype)

    queued(h, values, call, [ids, w, dl], 12)
