"""Order between the stream that arrays are filled on and a stream that a test makes (conftest.py), and the two launches that share a
product's tiles, captured and replayed between kernels that write what they read."""
import pytest
import torch

import layer_reference as ref
import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu


def test_a_new_stream_follows_what_was_filled_before():
    """torch's streams do not wait for the default stream: without the fixture the copy runs beside the sleep, before the fill."""
    x, y = (torch.zeros(1 << 20, device="cuda") for _ in range(2))
    with torch.cuda.stream(torch.cuda.Stream()):   # (what a first copy and a first stream wait for is behind them)
        y.copy_(x)
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)   # (cycles, some 20 ms)
    x.fill_(1.0)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y.copy_(x)
    torch.cuda.synchronize()
    assert (y == 1.0).all()


def test_streams_are_otherwise_as_torch_makes_them():
    a, b = torch.cuda.Stream(), torch.cuda.Stream(0, priority=-1)
    assert isinstance(a, torch.cuda.Stream) and a != b and a.cuda_stream != b.cuda_stream and b.priority < a.priority
    with torch.cuda.stream(a):
        assert torch.cuda.current_stream() == a
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


@pytest.mark.parametrize("N,act", [(19464, pts.GEMM_ACT_NONE), (9736, pts.GEMM_ACT_SILU | pts.GEMM_ACT_GATED)])
def test_a_wave_and_a_part_in_a_graph(N, act):
    """More tiles than SMs, fewer than twice as many: X goes through the product, which adds to C, and C back to X, three times, each
    product held to what it read; then replayed, with equal bits."""
    rows, K, t, n = 16, 1600, torch.float16, 3
    gen = torch.Generator("cuda").manual_seed(3)
    fill = lambda *s, scale=1.0: torch.empty(s, dtype=t, device="cuda").normal_(0.0, scale, generator=gen)  # noqa: E731
    A, B = fill(rows, K), fill(N * (2 if act & pts.GEMM_ACT_GATED else 1), K, scale=K ** -0.5)
    back, res = fill(K, N, scale=N ** -0.5), fill(rows, N)
    X, C = torch.zeros_like(A), torch.zeros_like(res)
    xs, cs = torch.zeros(n + 1, rows, K, dtype=t, device="cuda"), torch.zeros(n + 1, rows, N, dtype=t, device="cuda")
    h, s = pts.gemm_create(0), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        X.copy_(A)
        C.copy_(res)
        for i in range(n + 1):
            xs[i].copy_(X)
            cs[i].copy_(C)
            if i < n:
                pts.gemm_run_linear(h, rows, 1, N, K, X, B, None, C, None, C, None, act, pts.GEMM_F16, stream=s)
                pts.gemm_run_linear(h, rows, 1, K, N, C, back, None, None, None, X, None, 0, pts.GEMM_F16, stream=s)
        X.zero_()
        C.zero_()

    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    first = xs.clone(), cs.clone()
    assert torch.equal(xs[0], A) and torch.equal(cs[0], res)
    for i in range(n):
        (c, dc), _ = ref.linear(act, xs[i], B, None, cs[i])
        ref.close(cs[i + 1], c, dc, ("C", i))
        (x, dx), _ = ref.linear(0, cs[i + 1], back)
        ref.close(xs[i + 1], x, dx, ("X", i))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for _ in range(5):
        xs.zero_()
        cs.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(xs, first[0]) and torch.equal(cs, first[1])
    st, dev = pts.gemm_check(h)
    pts.gemm_destroy(h)
    assert st == 0, f"device status {dev:#x}"
