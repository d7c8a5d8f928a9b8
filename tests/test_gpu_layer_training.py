"""The operators around the products run together, as examples/expert_layer.py uses them: a router, a layer of experts and their
gradients, against the same layer in 64 bits and its autograd; decoding against the trained layer's forward pass."""
import os
import sys

import pytest
import torch

import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def make(D, H, E, k):
    import expert_layer as ex
    quantise, ex.quantise = ex.quantise, lambda w, group: None   # (sizes that are no multiple of a group)
    try:
        return ex.ExpertLayer(D, H, E, k)
    finally:
        ex.quantise = quantise


@pytest.fixture(scope="module")
def layer():
    layer = make(72, 136, 5, 2)
    yield layer
    st, dev = pts.gemm_check(layer.h)
    layer.close()
    assert st == 0, f"device status {dev:#x}"


def layer64(x, gate, up, down, ids):
    """y with ids given (the choice has no gradient) and weights from the gate."""
    logits = x @ gate.T
    w = torch.softmax(torch.gather(logits, 1, ids), 1)
    hidden = torch.einsum("tkhd,td->tkh", up[ids], x).clamp(min=0) ** 2
    return (torch.einsum("tkdh,tkh->tkd", down[ids], hidden) * w[..., None]).sum(1)


def near(a, b, what):
    """Each 16-bit tensor between two operators is rounded to 2^-8 of itself and a product keeps that relative to the root of its
    sum of squares: at most 8 roundings in a row are below 2^-5 of the result's norm."""
    assert float((a.double() - b.double()).norm()) <= 2.0 ** -5 * float(b.double().norm()), what


@pytest.mark.parametrize("tokens", [1, 100])
def test_training_step(layer, tokens):
    gen = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, layer.dim, generator=gen).to(torch.bfloat16).cuda()
    dy = torch.randn(tokens, layer.dim, generator=gen).to(torch.bfloat16).cuda()
    ids, w, routed = layer.route(x)
    y, saved = layer.forward(x, ids, w)
    dx, dw, dup, ddown = layer.backward(dy, saved)
    dx_route, dgate = layer.route_backward(dw, routed)

    leaves = [t.double().requires_grad_() for t in (x, layer.gate[0, :layer.experts], layer.up, layer.down)]
    y64 = layer64(*leaves, ids.long())
    want = torch.autograd.grad((y64 * dy.double()).sum(), leaves)
    assert ((ids >= 0) & (ids < layer.experts)).all()
    near(y, y64.detach(), "y")
    for a, b, what in ((dup, want[2], "up"), (ddown, want[3], "down")):
        near(a, b, what)
    # A weight's gradient is dy . ys, where ys is off by 2 roundings of 2^-8: by 2^-7 |dy| |ys| at most, however small the sum is.  The
    # softmax's gradient halves that at least, and the product with x takes it times x's largest singular value.
    row_of, ys = saved[2].long(), saved[-1].double()
    off = (dy.double().norm(dim=1)[:, None] * ys[row_of].norm(dim=2)).norm() * 2.0 ** -7 * torch.linalg.matrix_norm(x.double(), 2)
    assert float((dgate[0, :layer.experts].double() - want[1]).norm()) <= 2.0 ** -5 * float(want[1].norm()) + float(off)
    assert (dgate[0, layer.experts:] == 0).all()
    near(dx.double() + dx_route.double(), want[0], "x")


def test_gradients_against_differences(layer):
    """Along a random direction of the router's and the experts' matrices: the 64-bit layer's central difference of step 2^-12 (off by
    2^-24 of a third derivative, far below the 16-bit roundings) and the gradients' inner product with the direction."""
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(40, layer.dim, generator=gen).to(torch.bfloat16).cuda()
    dy = torch.randn(40, layer.dim, generator=gen).to(torch.bfloat16).cuda()
    ids, w, routed = layer.route(x)
    y, saved = layer.forward(x, ids, w)
    _, dw, dup, ddown = layer.backward(dy, saved)
    base = [x.double(), layer.gate[0, :layer.experts].double(), layer.up.double(), layer.down.double()]
    for i, g in ((2, dup), (3, ddown)):
        d = torch.randn(base[i].shape, generator=gen).double().cuda()
        f = lambda t: float((layer64(*[b + t * d if j == i else b for j, b in enumerate(base)], ids.long()) * dy.double()).sum())  # noqa: E731
        diff = (f(2.0 ** -12) - f(-2.0 ** -12)) / 2.0 ** -11
        # (an inner product of random signs: an error of 2^-5 of the gradient's norm moves it by 2^-5 |g| |d| / sqrt(n) times a normal
        # deviate, 6 of which are not met by chance)
        assert abs(float((g.double() * d).sum()) - diff) <= 6 * 2.0 ** -5 * float(g.double().norm()) * float(d.norm()) / g.numel() ** 0.5


@pytest.mark.parametrize("tokens", [1, 7, 64])
def test_decoding_in_two_launches_is_the_forward_pass(layer, tokens):
    x = torch.randn(tokens, layer.dim, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    ids, w, _ = layer.route(x)
    y, _ = layer.forward(x, ids, w)
    near(layer.decode16(x, ids, w), y, "decode16")
