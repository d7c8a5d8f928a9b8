"""What stands around the products at its limits: many experts, arrays of more than 2^31 elements, calls on several streams at once,
and what is refused."""
import pytest
import torch

import layer_reference as ref
import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu

F16, BF16 = pts.GEMM_F16, pts.GEMM_BF16
GATED, SILU = pts.GEMM_ACT_GATED, pts.GEMM_ACT_SILU


@pytest.fixture(scope="module")
def h():
    h = pts.gemm_create(0)
    yield h
    st, dev = pts.gemm_check(h)
    pts.gemm_destroy(h)
    assert st == 0, f"device status {dev:#x}"


def rand(shape, dtype, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def large(shape, dtype, seed, scale=1.0):
    """Made on the GPU."""
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=torch.Generator("cuda").manual_seed(seed))


def offsets_of(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("counts", [[1, 0, 2] * 200, [9, 1, 0] * 200, [0] * 599 + [1000], [1000] + [0] * 203], ids=["600", "600 more", "the last", "the first of 204"])
@pytest.mark.parametrize("act", [SILU | GATED, 2])
def test_many_experts(h, counts, act):
    rows, E, N, K = sum(counts), len(counts), 40, 72
    all_ = N * (2 if act & GATED else 1)
    A, B, bias, off = rand((rows + 2, K), torch.bfloat16, 1), rand((E, all_, K), torch.bfloat16, 2, 0.2), rand((E, all_), torch.bfloat16, 3), offsets_of(counts)
    C, Z = torch.full((rows + 2, N), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((rows + 2, all_), 7.0, dtype=torch.bfloat16, device="cuda")
    pts.gemm_run_linear(h, rows + 2, E, N, K, A, B, bias, None, off, C, Z, act, BF16)
    dZ, dbias = torch.full_like(Z, 7.0), torch.full((E, all_), 7.0, device="cuda")
    dC = rand((rows + 2, N), torch.bfloat16, 4)
    pts.gemm_linear_grad(h, rows + 2, E, N, dC, Z, off, dZ, dbias, act, BF16)
    at = off.tolist()
    for e in range(E):
        r = slice(at[e], at[e + 1])
        (c, dc), (z, dz) = ref.linear(act, A[r], B[e], bias[e])
        ref.close(C[r], c, dc, ("C", e))
        ref.close(Z[r], z, dz, ("Z", e))
        d, z = dC[r].double(), Z[r].double()
        a, s, sa = ref.act(act, z[:, :N])
        want, err = d * s, d.abs() * sa * 2 * ref.EPS_ACT
        if act & GATED:
            want, err = torch.cat([want * z[:, N:], d * a], 1), torch.cat([err * z[:, N:].abs(), d.abs() * a.abs() * 2 * ref.EPS_ACT], 1)
        ref.close(dZ[r], want, err, ("dZ", e))
        ref.close(dbias[e], want.sum(0), err.sum(0) + want.shape[0] * 2.0 ** -23 * want.abs().sum(0), ("dbias", e))
    assert all((t[rows:] == 7.0).all() for t in (C, Z, dZ))


def test_the_largest_layer(h):
    """As many tokens, assignments and experts as it takes."""
    T, k, E, D, H = 64, 8, 1024, 72, 40
    up, down, x = rand((E, 2 * H, D), torch.float16, 1, 0.2), rand((E, D, H), torch.float16, 2, 0.2), rand((T, D), torch.float16, 3)
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k] for t in range(T)]).int().cuda()
    ids[0] = torch.arange(E - k, E)
    w, Hs, Y = rand((T, k), torch.float32, 4), torch.zeros(T * k, H, dtype=torch.float16, device="cuda"), torch.zeros(T, D, dtype=torch.float16, device="cuda")
    pts.gemm_expert_layer(h, T, k, E, D, H, x, ids, w, up, None, down, None, None, Hs, Y, SILU | GATED, F16)
    ref.close(Y, *ref.layer(SILU | GATED, x, ids.cpu(), w.cpu(), up, None, down, None, None, torch.float16))


def test_more_than_2_31_outputs(h):
    """70016 rows of 32776 columns: C passes 2^31 elements, Z 2^32."""
    rows, N, K, act = 70016, 32776, 16, SILU | GATED
    A, B, bias = rand((rows, K), torch.bfloat16, 1), rand((1, 2 * N, K), torch.bfloat16, 2, 0.3), rand((1, 2 * N), torch.bfloat16, 3)
    C, Z = (torch.empty(rows, n, dtype=torch.bfloat16, device="cuda") for n in (N, 2 * N))
    pts.gemm_run_linear(h, rows, 1, N, K, A, B, bias, None, None, C, Z, act, BF16)
    dZ, dbias = torch.empty_like(Z), torch.empty(1, 2 * N, device="cuda")
    pts.gemm_linear_grad(h, rows, 1, N, C, Z, None, dZ, dbias, act, BF16)
    for r in (slice(0, 20), slice(32760, 32780), slice(65510, 65540), slice(rows - 20, rows)):
        (c, dc), (z, dz) = ref.linear(act, A[r], B[0], bias[0])
        ref.close(C[r], c, dc, r)
        ref.close(Z[r], z, dz, r)
        d, z = C[r].double(), Z[r].double()
        a, s, sa = ref.act(act, z[:, :N])
        ref.close(dZ[r], torch.cat([d * s * z[:, N:], d * a], 1), 2 * ref.EPS_ACT * torch.cat([d.abs() * sa * z[:, N:].abs(), (d * a).abs()], 1), r)
    cols = torch.tensor([0, 1, N - 1], device="cuda")
    d, g, u = C[:, cols].double(), Z[:, cols].double(), Z[:, cols + N].double()
    a, s, sa = ref.act(act, g)
    for at, want, err in ((cols, d * s * u, (d * u).abs() * sa), (cols + N, d * a, (d * a).abs())):
        ref.close(dbias[0, at], want.sum(0), 2 * ref.EPS_ACT * err.sum(0) + rows * 2.0 ** -23 * want.abs().sum(0))


def test_more_than_2_31_weights(h):
    """33 experts of 8192 x 8192, the last behind 2^31 elements: a row each, more rows each, and the whole layer."""
    E, D = 33, 8192
    W = large((E, D, D), torch.bfloat16, 1, D ** -0.5)
    for each in (1, 8):
        A, C = rand((E * each, D), torch.bfloat16, 2), torch.zeros(E * each, D, dtype=torch.bfloat16, device="cuda")
        pts.gemm_run_linear(h, E * each, E, D, D, A, W, None, None, offsets_of([each] * E), C, None, 1, BF16)
        for e in (0, 31, 32):
            r = slice(e * each, (e + 1) * each)
            (c, dc), _ = ref.linear(1, A[r], W[e])
            ref.close(C[r], c, dc, (each, e))
    ids, w, x = torch.tensor([[32, 0], [5, 32], [31, 32]], dtype=torch.int32), rand((3, 2), torch.float32, 3), rand((3, D), torch.bfloat16, 4)
    Hs, Y = torch.zeros(6, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, D, dtype=torch.bfloat16, device="cuda")
    pts.gemm_expert_layer(h, 3, 2, E, D, D, x, ids.cuda(), w, W, None, W, None, x, Hs, Y, 1, BF16)
    ref.close(Y, *ref.layer(1, x, ids, w.cpu(), W, None, W, None, x, torch.bfloat16))


def test_more_than_2_31_logits(h):
    T, E, k = (1 << 21) + 77, 1024, 4
    x = large((T, E), torch.bfloat16, 1)
    ids, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    pts.gemm_expert_route(h, T, k, E, x, ids, w, pts.GEMM_ROUTE_SELECTED, BF16)
    dl = torch.full_like(x, 9.0)
    pts.gemm_expert_route_grad(h, T, k, E, x, ids, w, dl, pts.GEMM_ROUTE_SELECTED, BF16)
    for r in (slice(0, 50), slice((1 << 21) - 20, T)):
        v, at = torch.sort(x[r].double(), dim=1, descending=True, stable=True)
        assert torch.equal(ids[r].long(), at[:, :k])
        p = torch.softmax(v[:, :k], 1)
        # values within 8 of another: as in the routing's tests
        assert ((w[r].double() - p).abs() <= 200 * 2.0 ** -24 * p).all()
        g = torch.zeros(p.shape[0], E, dtype=torch.float64, device="cuda").scatter_(1, at[:, :k], p * (w[r].double() - (p * w[r].double()).sum(1, keepdim=True)))
        assert ((dl[r].double() - g).abs() <= 2.0 ** -8 * g.abs() + 704 * 2.0 ** -24).all()


def test_calls_on_several_streams_at_once(h):
    """One handle, three streams, each its own arrays, eager and captured: as one after another."""
    T, k, E, D, H, n = 20, 2, 8, 520, 264, 12
    t, act = torch.bfloat16, SILU | GATED
    up, down, gate = rand((E, 2 * H, D), t, 1, D ** -0.5), rand((E, D, H), t, 2, H ** -0.5), rand((1, E, D), t, 3, D ** -0.5)
    wide = rand((1, 1032, D), t, 4, D ** -0.5)

    class Arrays:
        def __init__(self, seed):
            self.x, self.big = rand((T, D), t, seed), rand((700, D), t, seed + 50)
            self.logits, self.ids, self.w = torch.zeros(T, E, dtype=t, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
            self.Hs, self.Y = torch.zeros(T * k, H, dtype=t, device="cuda"), torch.zeros(T, D, dtype=t, device="cuda")
            self.C, self.Z = torch.zeros(700, 1032, dtype=t, device="cuda"), torch.zeros(700, 1032, dtype=t, device="cuda")
            self.dZ, self.db = torch.zeros_like(self.C), torch.zeros(1, 1032, device="cuda")
            self.dl = torch.zeros_like(self.logits)

        def step(self, s):
            pts.gemm_run_linear(h, 700, 1, 1032, D, self.big, wide, None, None, None, self.C, self.Z, SILU, BF16, stream=s)
            pts.gemm_run_linear(h, T, 1, E, D, self.x, gate, None, None, None, self.logits, None, 0, BF16, stream=s)
            pts.gemm_expert_route(h, T, k, E, self.logits, self.ids, self.w, pts.GEMM_ROUTE_ALL, BF16, stream=s)
            pts.gemm_expert_layer(h, T, k, E, D, H, self.x, self.ids, self.w, up, None, down, None, self.x, self.Hs, self.Y, act, BF16, stream=s)
            pts.gemm_linear_grad(h, 700, 1, 1032, self.C, self.Z, None, self.dZ, self.db, SILU, BF16, stream=s)
            pts.gemm_expert_route_grad(h, T, k, E, self.logits, self.ids, self.w, self.dl, pts.GEMM_ROUTE_ALL, BF16, stream=s)

        def results(self):
            return [v.clone() for v in (self.logits, self.ids, self.w, self.Hs, self.Y, self.C, self.Z, self.dZ, self.db, self.dl)]

        def clear(self):
            for v in (self.logits, self.ids, self.w, self.Hs, self.Y, self.C, self.Z, self.dZ, self.db, self.dl):
                v.zero_()

    sets, streams = [Arrays(10 + i) for i in range(3)], [torch.cuda.Stream() for _ in range(3)]
    want = []
    for a in sets:
        a.step(None)
        torch.cuda.synchronize()
        want.append(a.results())
    graphs = []
    for a, s in zip(sets, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            a.step(s)
    for captured in (False, True):
        for a in sets:
            a.clear()
        torch.cuda.synchronize()
        for _ in range(n):
            for a, s, g in zip(sets, streams, graphs):
                with torch.cuda.stream(s):
                    if captured:
                        g.replay()
                    else:
                        a.step(s)
        torch.cuda.synchronize()
        for a, results in zip(sets, want):
            assert all(torch.equal(x, y) for x, y in zip(a.results(), results))


@pytest.mark.parametrize("dtype", [F16, BF16, pts.GEMM_E4M3], ids=["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("counts,N,K", [([33], 264, 8192), ([64], 2048, 4096), ([65], 1000, 1536), ([100], 136, 2048), ([300], 128, 4096), ([1000], 136, 1024),
                                        ([0, 100, 3], 264, 2048), ([70, 0, 0, 64], 520, 4096), ([17, 130], 128, 8192)])
@pytest.mark.parametrize("act,keep", [(3, False), (SILU | GATED, True)])
def test_row_tiles_that_ctas_share(h, counts, N, K, act, keep, dtype):
    """Several tiles of rows, ragged, whose contraction 2, 4 or 8 CTAs share: two runs have equal bits."""
    rows, E, all_, out = sum(counts) + 2, len(counts), N * (2 if act & GATED else 1), torch.float16 if dtype == F16 else torch.bfloat16
    t = {F16: torch.float16, BF16: torch.bfloat16, pts.GEMM_E4M3: torch.float8_e4m3fn}[dtype]
    A, B = rand((rows, K), torch.float32, 1).clamp(-448, 448).to(t), rand((E, all_, K), torch.float32, 2, 1.0 if dtype == pts.GEMM_E4M3 else K ** -0.5).clamp(-448, 448).to(t)
    scale = float(torch.tensor(K ** 0.5 if dtype == pts.GEMM_E4M3 else 1.0).float())
    bias, res, off = rand((E, all_), out, 3), rand((rows, N), out, 4), offsets_of(counts)
    got = []
    for _ in range(2):
        C, Z = torch.full((rows, N), 7.0, dtype=out, device="cuda"), torch.full((rows, all_), 7.0, dtype=out, device="cuda") if keep else None
        pts.gemm_run_linear(h, rows if E > 1 else rows - 2, E, N, K, A, B, bias, res, off if E > 1 else None, C, Z, act, dtype, 1.0, scale)
        got.append((C, Z))
    assert torch.equal(got[0][0], got[1][0]) and (not keep or torch.equal(got[0][1], got[1][1]))
    at = off.tolist()
    for e in range(E):
        r = slice(at[e], at[e + 1])
        (c, dc), (z, dz) = ref.linear(act, A[r], B[e], bias[e], res[r], scale)
        ref.close(C[r], c, dc, ("C", e))
        if keep:
            ref.close(Z[r], z, dz, ("Z", e))
    assert (C[-2:] == 7.0).all() and (not keep or (Z[-2:] == 7.0).all())


@pytest.mark.parametrize("N,act,dtype", [(19456 + 8, 2, F16), (22528, SILU, BF16), (28000, 0, F16), (9736, SILU | GATED, BF16), (14336, 3 | GATED, F16), (22528, 1, pts.GEMM_E4M3)])
@pytest.mark.parametrize("rows", [9, 24, 32])
def test_a_wave_and_a_part(h, rows, N, act, dtype):
    """Tiles that are more than the SMs but less than twice as many, as one of two products queued one after the other: the second
    reads all that the first has written, and neither writes before the call in front has read."""
    K = 2048 if dtype != pts.GEMM_E4M3 else 4096
    all_, out = N * (2 if act & GATED else 1), torch.bfloat16 if dtype != F16 else torch.float16
    t = {F16: torch.float16, BF16: torch.bfloat16, pts.GEMM_E4M3: torch.float8_e4m3fn}[dtype]
    A, B = rand((rows, K), torch.float32, 1).clamp(-448, 448).to(t), large((all_, K), torch.float32, 2, 1.0 if dtype == pts.GEMM_E4M3 else K ** -0.5).clamp(-448, 448).to(t)
    scale = K ** 0.5 if dtype == pts.GEMM_E4M3 else 1.0
    bias, res = rand((1, all_), out, 3), rand((rows, N), out, 4)
    back = large((64, N), out, 5, N ** -0.5)
    C, Z, D = torch.zeros(rows, N, dtype=out, device="cuda"), torch.zeros(rows, all_, dtype=out, device="cuda"), torch.zeros(8, rows, 64, dtype=out, device="cuda")
    torch.cuda.synchronize()
    for i in range(8):   # C starts as the residual, so every call changes it
        C.copy_(res) if i % 4 == 0 else None
        pts.gemm_run_linear(h, rows, 1, N, K, A, B, bias, C, None, C, Z, act, dtype, 1.0, float(torch.tensor(scale).float()))
        pts.gemm_run_linear(h, rows, 1, 64, N, C, back, None, None, None, D[i], None, 0, F16 if out == torch.float16 else BF16)
    torch.cuda.synchronize()
    assert torch.equal(D[:4], D[4:])
    last = C.clone()
    C.copy_(res)
    pts.gemm_run_linear(h, rows, 1, N, K, A, B, bias, C, None, C, Z, act, dtype, 1.0, float(torch.tensor(scale).float()))
    (c, dc), (z, dz) = ref.linear(act, A, B, bias[0], res, float(torch.tensor(scale).float()))
    ref.close(C, c, dc, "C")
    ref.close(Z, z, dz, "Z")
    (d, dd), _ = ref.linear(0, last, back)
    ref.close(D[3], d, dd, "D")


def test_a_wave_and_a_part_captured(h):
    """The two launches in a graph, between kernels that write what they read and read what they write: as eagerly."""
    rows, N, K, t = 24, 20000, 1600, torch.float16
    A, B, back = rand((rows, K), t, 1), large((N, K), t, 2, K ** -0.5), large((K, N), t, 3, N ** -0.5)
    X, C, Y = torch.zeros_like(A), torch.zeros(rows, N, dtype=t, device="cuda"), torch.zeros(rows, K, dtype=t, device="cuda")

    def step(s):
        X.copy_(A)
        for _ in range(3):
            pts.gemm_run_linear(h, rows, 1, N, K, X, B, None, None, None, C, None, SILU, F16, stream=s)
            pts.gemm_run_linear(h, rows, 1, K, N, C, back, None, X, None, X, None, 0, F16, stream=s)
        Y.copy_(X)
        C.zero_()

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(s)
    torch.cuda.synchronize()
    want = Y.clone()
    x = A.double()
    for _ in range(3):
        c = torch.nn.functional.silu(x @ B.double().T).to(t).double()
        x = (c @ back.double().T + x).to(t).double()
    assert float((want.double() - x).norm()) <= 3 * 2.0 ** -10 * float(x.norm())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    for _ in range(5):
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)


def test_products_that_are_refused(h):
    x = torch.zeros(1 << 16, dtype=torch.float16, device="cuda").data_ptr()
    off = offsets_of([8, 0]).data_ptr()
    linear = lambda rows, E, N, K, act=0, dtype=F16, A=x, B=x, bias=None, res=None, o=off, C=x, Z=None, sa=1.0: pts.gemm_run_linear(  # noqa: E731
        h, rows, E, N, K, A, B, bias, res, o, C, Z, act, dtype, sa, 1.0)
    grad = lambda rows, E, N, act=0, dtype=F16, dC=x, Z=x, o=off, dZ=x, db=None: pts.gemm_linear_grad(h, rows, E, N, dC, Z, o, dZ, db, act, dtype)  # noqa: E731
    most = pts.gemm.GEMM_EXPERT_MAX_SIZE
    for bad in ((-1, 2, 8, 8), (8, -1, 8, 8), (8, 2, -8, 8), (8, 2, 8, -8), (8, 2, 12, 8), (8, 2, 8, 12), (8, 2, 8, 8, 0, pts.GEMM_E4M3), (most + 8, 2, 8, 8), (8, 2, most + 8, 8),
                (8, 2, 8, most + 8), (8, 2, (most // 16 + 1) * 8, 8, GATED), (8, 2, 8, 8, 6), (8, 2, 8, 8, -1), (8, 2, 8, 8, 0x20), (8, 2, 8, 8, 0x16)):
        with pytest.raises(pts.GemmError) as err:
            linear(*bad)
        assert err.value.status == 1, bad
    for bad in (dict(A=None), dict(B=None), dict(C=None), dict(o=None), dict(A=x + 8), dict(B=x + 2), dict(C=x + 8), dict(bias=x + 4), dict(res=x + 8), dict(Z=x + 2), dict(o=off + 2)):
        with pytest.raises(pts.GemmError) as err:
            linear(8, 2, 8, 8, **bad)
        assert err.value.status == 1, bad
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(pts.GemmError):
            linear(8, 2, 8, 16, dtype=pts.GEMM_E4M3, sa=scale)
    for bad in ((-1, 2, 8), (8, -1, 8), (8, 2, -8), (8, 2, 12), (most + 8, 2, 8), (8, 2, most + 8), (8, 2, 8, 6), (8, 2, 8, -1), (8, 2, 8, 0x20), (8, 2, 8, 0, pts.GEMM_E4M3),
                (8, 2, (most // 16 + 1) * 8, GATED)):
        with pytest.raises(pts.GemmError) as err:
            grad(*bad)
        assert err.value.status == 1, bad
    for bad in (dict(dC=None), dict(Z=None), dict(dZ=None), dict(o=None), dict(dC=x + 8), dict(Z=x + 2), dict(dZ=x + 8), dict(o=off + 2), dict(db=x + 2)):
        with pytest.raises(pts.GemmError) as err:
            grad(8, 2, 8, **bad)
        assert err.value.status == 1, bad
