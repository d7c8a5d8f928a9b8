"""Plain 64-bit forms of what stands around the products, with the bounds their results are held to.

Bounds.  u is half a step of the output's type (2^-8 bf16, 2^-11 fp16, 2^-24 fp32), relative to the value.
  sums of K products in fp32   K 2^-23 sum |a||b| (a tensor core may truncate), and 2^-22 of the sum for scale and bias
  activations                  2^-15 of their value.  2^y in its fast form is off by 4 steps of 2^-24, and y by as many roundings
                               of 2^-24 |y| as it has operations and constants, which moves the power by 0.7 times that.
                               gelu: y = -z^2 log2(e) / 2 has 3; behind |z| = 13.5, |y| = 132, less than 2^-127 is left.  With
                               the polynomial's 1.1e-6 (19 steps) and 4 roundings of the products around it that is
                               (4 + 0.7 * 3 * 132 + 19 + 4) 2^-24 < 2^-15.  silu and the tanh form: y has at most 8, and behind
                               |y| = 60 the power is cut off, the value then below 44 * 2^-60: (4 + 0.7 * 8 * 60 + 8) 2^-24.
  an error d of a sum          slope * d behind the activation; |slope| <= 1.13 (gelu and silu), 2 |z| + 2 d (relu^2)
and 2^-25, half the smallest fp16 subnormal (bf16's are smaller), for each rounding to 16 bits."""
import math

import torch

ACTS = ("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")   # GEMM_ACT_NONE ... GEMM_ACT_SILU
GATED = 0x10
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 2.0 ** -25
EPS_ACT = 2.0 ** -15


def act(code, z):
    """act(z), its slope, and the sum of the absolute terms that the slope is made of."""
    name = ACTS[code & 15]
    if name == "none":
        return z, torch.ones_like(z), torch.ones_like(z)
    if name in ("relu", "relu2"):
        p = z.clamp(min=0.0)
        s = (z > 0).double() if name == "relu" else 2.0 * p
        return (p if name == "relu" else p * p), s, s
    if name == "gelu":
        s, d = torch.special.ndtr(z), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    elif name == "gelu_tanh":
        y = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        s = torch.sigmoid(y)
        d = z * s * torch.sigmoid(-y) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    else:
        s = torch.sigmoid(z)
        d = z * s * torch.sigmoid(-z)
    return z * s, s + d, s.abs() + d.abs()


def act_error(code, z, dz):
    """What act(z) may be off by where z is off by dz."""
    a, _, _ = act(code, z)
    if ACTS[code & 15] == "none":
        return dz
    slope = 2 * z.abs() + 2 * dz if ACTS[code & 15] == "relu2" else 1.13
    return slope * dz + EPS_ACT * a.abs()


def hidden(code, z, dz):
    """act(z), gated act(gate) * up, and what it may be off by."""
    if not code & GATED:
        return act(code, z)[0], act_error(code, z, dz)
    n = z.shape[-1] // 2
    (g, u), (dg, du) = (z[..., :n], z[..., n:]), (dz[..., :n], dz[..., n:])
    a, da = act(code, g)[0], act_error(code, g, dg)
    return a * u, da * (u.abs() + du) + a.abs() * du + 2.0 ** -23 * (a * u).abs()


def linear(code, A, B, bias=None, residual=None, scale=1.0):
    """(C, its bound before rounding), (Z, its bound): one matrix."""
    a, b = A.double(), B.double()
    z = a @ b.T / scale
    dz = (a.shape[1] + 2) * 2.0 ** -23 * (a.abs() @ b.abs().T) / scale
    if bias is not None:
        z = z + bias.double()
    dz = dz + 2.0 ** -22 * z.abs()
    c, dc = hidden(code, z, dz)
    if residual is not None:
        dc = dc + 2.0 ** -23 * (c.abs() + residual.double().abs())
        c = c + residual.double()
    return (c, dc), (z, dz)


def close(got, ref, err, what=""):
    """got (rounded once to its type) against ref, which the computation may have missed by err before that."""
    bound = U[got.dtype] * (ref.abs() + err) + err + TINY
    off = (got.double() - ref).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), got.shape, float((off / bound).nan_to_num(9e9).max()), bad.nonzero()[:4].tolist())


def layer(code, x, ids, w, up, up_bias, down, down_bias, residual, dtype):
    """A layer of experts token by token: y and what it may be off by before its rounding."""
    T, D = x.shape
    y = torch.zeros(T, D, dtype=torch.float64, device=x.device) if residual is None else residual.double().clone()
    terms, err = y.abs(), torch.zeros_like(y)
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < up.shape[0]:
                continue
            (h, dh), _ = linear(code, x[t:t + 1], up[e], None if up_bias is None else up_bias[e])
            dh = dh + U[dtype] * (h.abs() + dh) + TINY
            W, f = down[e].double(), float(w[t, j])
            o, oa = (h @ W.T)[0], (h.abs() @ W.abs().T)[0]
            if down_bias is not None:
                o, oa = o + down_bias[e].double(), oa + down_bias[e].double().abs()
            y[t] += f * o
            terms[t] += abs(f) * oa
            err[t] += abs(f) * ((dh @ W.abs().T)[0] + (h.shape[1] + 2) * 2.0 ** -23 * oa)
    # (the sums over warps, assignments, bias and residual: fewer than 64 more additions)
    return y, err + 64 * 2.0 ** -23 * terms
