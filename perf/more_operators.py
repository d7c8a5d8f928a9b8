"""What stands around the products of a feed-forward layer, as cases that can be timed and compared.

  linear         C = act(A . B^T + bias) + residual in one launch
                 (gemm_run_linear): one matrix, or rows sorted by expert with the
                 counts on the device; gated, B holds a gate and an up matrix and
                 C = act(gate) * up; `keep` also writes Z, the sum before act
  linear_grad    from dC and Z: dZ and the bias's gradient (gemm_linear_grad)
  route          expert ids and weights from a router's logits
                 (gemm_expert_route), and the gradient of the logits
                 (gemm_expert_route_grad) where `backward` is set
  layer          a layer of experts for a few tokens: up (gated or not), act,
                 down, weighted sum, residual (gemm_expert_layer)

`run` computes a case in its plain form, or with the framework's kernels where
`own` is set.  Sizes are those of this repository's benchmark and of its expert
layer's cases (4096, 8192, 4224, 2048, 1024 and their kind) or generic.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "f32": torch.float32}
_library = None


def listed():
    return [
        # one token against a gate and an up projection: latency and the weights' bytes
        dict(name="linear_token", op="linear", rows=1, experts=1, N=4096, K=4096, act="silu", gated=True, bias=False,
             residual=False, keep=False, skew=0.0, dtype="bf16"),
        # the down projection of a decoding batch, added to the residual stream
        dict(name="linear_decode", op="linear", rows=24, experts=1, N=4096, K=8192, act="none", gated=False, bias=True,
             residual=True, keep=False, skew=0.0, dtype="f16"),
        # a prompt of odd length through a projection with everything in its epilogue
        dict(name="linear_prompt", op="linear", rows=4101, experts=1, N=4224, K=4096, act="gelu", gated=False, bias=True,
             residual=True, keep=False, skew=0.0, dtype="f16"),
        # a training step's gated projection, the sums kept for the backward pass
        dict(name="linear_train", op="linear", rows=8192, experts=1, N=8192, K=4096, act="silu", gated=True, bias=False,
             residual=False, keep=True, skew=0.0, dtype="bf16"),
        # experts' up projections in 8 bits, unevenly filled
        dict(name="linear_experts_e4m3", op="linear", rows=2047, experts=8, N=4096, K=8192, act="relu2", gated=False,
             bias=True, residual=False, keep=False, skew=0.3, dtype="e4m3"),
        # the backward pass through an activation and a bias, a training step's rows
        dict(name="linear_grad_train", op="linear_grad", rows=16384, experts=1, N=8192, act="gelu_tanh", gated=False,
             bias=True, skew=0.0, dtype="bf16"),
        # the same of gated experts, odd row counts
        dict(name="linear_grad_experts", op="linear_grad", rows=4101, experts=16, N=2048, act="silu", gated=True, bias=True,
             skew=0.4, dtype="f16"),
        # a decoding batch's routing: latency
        dict(name="route_decode", op="route", tokens=16, experts=64, top_k=4, mode="selected", backward=False, masked=0.0,
             dtype="f32"),
        # a training step's routing and its gradient, padded tokens among them
        dict(name="route_train", op="route", tokens=16384, experts=128, top_k=8, mode="all", backward=True, masked=0.1,
             dtype="bf16"),
        # one token through a layer of experts
        dict(name="layer_one", op="layer", tokens=1, top_k=2, experts=8, of=8, dim=4096, hidden=4096, act="silu", gated=True,
             bias=False, residual=True, dtype="bf16"),
        # a decoding batch that reaches every expert of a wide layer
        dict(name="layer_batch", op="layer", tokens=16, top_k=2, experts=8, of=8, dim=4096, hidden=8192, act="silu", gated=True,
             bias=False, residual=False, dtype="bf16"),
        # an odd batch over many small experts, half of which are on another device
        dict(name="layer_many", op="layer", tokens=13, top_k=4, experts=32, of=64, dim=2048, hidden=1024, act="relu2", gated=False,
             bias=True, residual=True, dtype="f16"),
    ]


_ACTS = ["none", "relu", "relu2", "gelu", "gelu_tanh", "silu"]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, lo), hi // step * step)


def _draw_one(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "route", "layer", "layer"])
    if op == "route":
        experts = _log(rng, 2, 512)
        return dict(op=op, tokens=_log(rng, 8, 20000), experts=experts, top_k=min(rng.choice([1, 2, 3, 4, 6, 8]), experts),
                    mode=rng.choice(["selected", "all", "sigmoid"]), backward=rng.random() < 0.5, masked=rng.choice([0.0, 0.2]),
                    dtype=rng.choice(["f32", "f16", "bf16"]))
    gated = rng.random() < 0.5
    c = dict(op=op, act=rng.choice(_ACTS), gated=gated, bias=rng.random() < 0.5)
    step = 16 if gated else 8
    if op == "layer":
        experts = _log(rng, 2, 64)
        return dict(c, tokens=_log(rng, 1, 64), top_k=min(rng.choice([1, 2, 4, 8]), experts), experts=experts,
                    of=experts * rng.choice([1, 1, 2]), dim=_log(rng, 256, 8192, 8), hidden=_log(rng, 256, 8192, step),
                    residual=rng.random() < 0.5, dtype=rng.choice(["f16", "bf16"]))
    experts = 1 if rng.random() < 0.5 else _log(rng, 2, 32)
    c.update(rows=_log(rng, 1, 16384), experts=experts, N=_log(rng, 128, 8192, step), skew=round(rng.uniform(0.0, 0.6), 2) if experts > 1 else 0.0)
    if op == "linear_grad":
        return dict(c, dtype=rng.choice(["f16", "bf16"]))
    return dict(c, K=_log(rng, 256, 8192, 16), residual=rng.random() < 0.4, keep=rng.random() < 0.4,
                dtype=rng.choice(["f16", "bf16", "bf16", "e4m3"]))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        c = _draw_one(rng)
        weights = c.get("experts", 1) * c.get("N", 0) * c.get("K", 0) + c.get("experts", 1) * c.get("dim", 0) * c.get("hidden", 0)
        if weights > 1 << 28 or _cost(c) > most or (c["op"] == "layer" and c["of"] > c["experts"] and c["tokens"] * c["top_k"] < 8):
            continue   # (too large, or likely to have nothing on this device)
        return c


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 280)


# ---- inputs -----------------------------------------------------------------


def _normal(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * scale


def _ids(gen, rows, experts, skew, top_k=1):
    """top_k different experts for each row, expert e preferred by -skew * log(e + 1)."""
    u = torch.rand(rows, experts, generator=gen, device="cuda").clamp_(1e-7, 1.0 - 1e-7)
    score = -torch.log(-torch.log(u)) - skew * torch.log(torch.arange(1, experts + 1, device="cuda", dtype=torch.float32))
    return torch.topk(score, top_k, dim=1).indices


def _zeros(shape, dtype):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dt = case["op"], _DT[case["dtype"]]
    s = {"case": case}
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        logits = _normal(gen, T, E, scale=2.0)
        if case["masked"]:   # experts that a token may not go to, and padded tokens, which may go to none
            u = torch.rand(T, E, generator=gen, device="cuda") + (torch.rand(T, 1, generator=gen, device="cuda") < case["masked"]) * -2.0
            logits = torch.where(u < case["masked"], -math.inf, logits)
        s.update(logits=logits.to(dt), ids=_zeros((T, k), torch.int32), w=_zeros((T, k), torch.float32))
        if case["backward"]:
            s.update(dw=_normal(gen, T, k), dlogits=_zeros((T, E), dt))
        return s
    half = 2 if case["gated"] else 1
    if op == "layer":
        T, k, E, D, H = case["tokens"], case["top_k"], case["experts"], case["dim"], case["hidden"]
        # the router ranks all `of` experts; this device holds E of them, from `base` on
        base = (case["of"] - E) // 2
        s.update(ids=(_ids(gen, T, case["of"], 0.0, k) - base).to(torch.int32).contiguous(),
                 w=torch.softmax(_normal(gen, T, k), dim=1).contiguous(), X=_normal(gen, T, D).to(dt),
                 up=_normal(gen, E, half * H, D, scale=1.0 / math.sqrt(D)).to(dt),
                 down=_normal(gen, E, D, H, scale=1.0 / math.sqrt(H)).to(dt),
                 up_bias=_normal(gen, E, half * H, scale=0.1).to(dt) if case["bias"] else None,
                 down_bias=_normal(gen, E, D, scale=0.1).to(dt) if case["bias"] else None,
                 residual=_normal(gen, T, D).to(dt) if case["residual"] else None, Hs=_zeros((T * k, H), dt), Y=_zeros((T, D), dt))
        return s
    rows, E, N = case["rows"], case["experts"], case["N"]
    if E > 1:
        counts = torch.bincount(_ids(gen, rows, E, case["skew"]).reshape(-1), minlength=E)
        s["offsets"] = _zeros(E + 1, torch.int32)
        s["offsets"][1:] = torch.cumsum(counts, 0)
        s["most"] = int(counts.max())
    else:
        s.update(offsets=None, most=rows)
    if op == "linear_grad":
        s.update(dC=_normal(gen, rows, N, scale=1.0 / 16).to(dt), Z=_normal(gen, rows, half * N).to(dt), dZ=_zeros((rows, half * N), dt),
                 dbias=_zeros((E, half * N), torch.float32) if case["bias"] else None)
        return s
    K, out = case["K"], torch.bfloat16 if case["dtype"] == "e4m3" else dt
    a, b = _normal(gen, rows, K), _normal(gen, E, half * N, K, scale=1.0 / math.sqrt(K))
    s.update(scale_a=1.0, scale_b=1.0)
    if case["dtype"] == "e4m3":   # scaled so that the largest value is the type's largest
        s.update(scale_a=448.0 / float(a.abs().max()), scale_b=448.0 / float(b.abs().max()))
        a, b = (a * s["scale_a"]).clamp_(-448, 448), (b * s["scale_b"]).clamp_(-448, 448)
    s.update(A=a.to(dt), B=b.to(dt), bias=_normal(gen, E, half * N, scale=0.1).to(out) if case["bias"] else None,
             residual=_normal(gen, rows, N).to(out) if case["residual"] else None, C=_zeros((rows, N), out),
             Z=_zeros((rows, half * N), out) if case["keep"] else None)
    return s


# ---- one pass ---------------------------------------------------------------


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    global _library
    if _library is None:
        import persistent_tile_scheduled_gb300 as pts
        _library = (pts, pts.gemm_create(0), {"f16": pts.GEMM_F16, "bf16": pts.GEMM_BF16, "e4m3": pts.GEMM_E4M3, "f32": pts.GEMM_F32},
                    {"none": pts.GEMM_ACT_NONE, "relu": pts.GEMM_ACT_RELU, "relu2": pts.GEMM_ACT_RELU2, "gelu": pts.GEMM_ACT_GELU,
                     "gelu_tanh": pts.GEMM_ACT_GELU_TANH, "silu": pts.GEMM_ACT_SILU},
                    {"selected": pts.GEMM_ROUTE_SELECTED, "all": pts.GEMM_ROUTE_ALL, "sigmoid": pts.GEMM_ROUTE_SIGMOID})
    pts, h, types, acts, modes = _library
    c = s["case"]
    op, dt = c["op"], types[c["dtype"]]
    if op == "route":
        T, k, E, mode = c["tokens"], c["top_k"], c["experts"], modes[c["mode"]]
        pts.gemm_expert_route(h, T, k, E, s["logits"], s["ids"], s["w"], mode, dt)
        if not c["backward"]:
            return {"ids": s["ids"], "w": s["w"]}
        pts.gemm_expert_route_grad(h, T, k, E, s["logits"], s["ids"], s["dw"], s["dlogits"], mode, dt)
        return {"ids": s["ids"], "w": s["w"], "dlogits": s["dlogits"]}
    act = acts[c["act"]] | (pts.GEMM_ACT_GATED if c["gated"] else 0)
    if op == "layer":
        pts.gemm_expert_layer(h, c["tokens"], c["top_k"], c["experts"], c["dim"], c["hidden"], s["X"], s["ids"], s["w"], s["up"],
                              s["up_bias"], s["down"], s["down_bias"], s["residual"], s["Hs"], s["Y"], act, dt)
        return {"Y": s["Y"]}
    if op == "linear_grad":
        pts.gemm_linear_grad(h, c["rows"], c["experts"], c["N"], s["dC"], s["Z"], s["offsets"], s["dZ"], s["dbias"], act, dt)
        return {"dZ": s["dZ"], "dbias": s["dbias"]} if c["bias"] else {"dZ": s["dZ"]}
    pts.gemm_run_linear(h, c["rows"], c["experts"], c["N"], c["K"], s["A"], s["B"], s["bias"], s["residual"], s["offsets"], s["C"],
                        s["Z"], act, dt, s["scale_a"], s["scale_b"])
    return {"C": s["C"], "Z": s["Z"]} if c["keep"] else {"C": s["C"]}


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _act(name, z):
    if name == "relu":
        return z.clamp(min=0.0)
    if name == "relu2":
        return z.clamp(min=0.0) ** 2
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * _sigmoid(z) if name == "silu" else z


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "relu2":
        return 2.0 * z.clamp(min=0.0)
    if name == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if name == "silu":
        g = _sigmoid(z)
        return g * (1.0 + z * (1.0 - g))
    return torch.ones_like(z)


def _padded(x, offsets, most):
    """Rows sorted by expert -> (experts, most, columns) in 32 bits, zeros behind each expert's last row."""
    at = offsets[:-1, None].long() + torch.arange(most, device="cuda")
    there = at < offsets[1:, None]
    return torch.where(there[..., None], x.float()[at.clamp_(max=x.shape[0] - 1)], 0.0)


def _expert_of(offsets, rows):
    return (torch.arange(rows, device="cuda")[:, None] >= offsets[None, 1:]).sum(1)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        k, mode = c["top_k"], c["mode"]
        x = s["logits"].float()
        v, ids = torch.sort(x, dim=1, descending=True, stable=True)
        there = torch.isfinite(v[:, :k])
        ids = torch.where(there, ids[:, :k], 0)
        u = torch.minimum(x, torch.zeros_like(x)) - torch.log1p(torch.exp(-x.abs())) if mode == "sigmoid" else x
        best = v[:, :1].clamp(min=-1e30) if mode != "sigmoid" else torch.gather(u, 1, ids[:, :1]).clamp(min=-1e30)
        e = torch.exp(u - best)
        picked = torch.where(there, torch.gather(e, 1, ids), 0.0)
        total = (e if mode == "all" else picked).sum(1, keepdim=True).clamp(min=1e-30)
        w = picked / total
        out = {"ids": torch.where(there, ids, -1).int(), "w": w}
        if c["backward"]:
            d = torch.zeros_like(x).scatter_add_(1, ids, torch.where(there, s["dw"], 0.0))
            p = e / total if mode == "all" else torch.zeros_like(x).scatter_add_(1, ids, w)
            g = p * (d - (d * p).sum(1, keepdim=True))
            out["dlogits"] = (g * _sigmoid(-x) if mode == "sigmoid" else g).nan_to_num_(0.0).to(s["logits"].dtype)
        return out
    act, gated = c["act"], c["gated"]
    if op == "layer":
        T, H = c["tokens"], c["hidden"]
        held = (s["ids"] >= 0) & (s["ids"] < c["experts"])
        used = torch.unique(s["ids"][held]).long()
        cw = ((s["ids"][None] == used[:, None, None]) * s["w"][None]).sum(2)          # (used, T): a token's weight for an expert
        z = torch.bmm(s["X"].float().expand(used.numel(), -1, -1), s["up"][used].float().transpose(1, 2))
        z = z if s["up_bias"] is None else z + s["up_bias"][used].float()[:, None]
        hid = _act(act, z[..., :H]) * z[..., H:] if gated else _act(act, z)
        y = torch.bmm(hid, s["down"][used].float().transpose(1, 2))
        y = y if s["down_bias"] is None else y + s["down_bias"][used].float()[:, None]
        y = (y * cw[..., None]).sum(0)
        return {"Y": (y if s["residual"] is None else y + s["residual"].float()).to(s["Y"].dtype)}
    rows, N, off = c["rows"], c["N"], s["offsets"]
    if op == "linear_grad":
        d, z = s["dC"].float(), s["Z"].float()
        if gated:
            dz = torch.cat([d * z[:, N:] * _act_grad(act, z[:, :N]), d * _act(act, z[:, :N])], dim=1)
        else:
            dz = d * _act_grad(act, z)
        out = {"dZ": dz.to(s["dZ"].dtype)}
        if c["bias"]:
            if off is None:
                out["dbias"] = dz.sum(0, keepdim=True, dtype=torch.float64).float()
            else:
                e = _expert_of(off, rows)
                out["dbias"] = torch.zeros(c["experts"], dz.shape[1], dtype=torch.float64, device="cuda").index_add_(0, e, dz.double()).float()
        return out
    if off is None:
        z = s["A"].float() @ s["B"][0].float().T
        bias = None if s["bias"] is None else s["bias"].float()
    else:
        e = _expert_of(off, rows)
        z = torch.bmm(_padded(s["A"], off, s["most"]), s["B"].float().transpose(1, 2))[e, torch.arange(rows, device="cuda") - off[e].long()]
        bias = None if s["bias"] is None else s["bias"].float()[e]
    z = z / (s["scale_a"] * s["scale_b"])
    z = z if bias is None else z + bias
    y = _act(act, z[:, :N]) * z[:, N:] if gated else _act(act, z)
    y = y if s["residual"] is None else y + s["residual"].float()
    out = {"C": y.to(s["C"].dtype)}
    return dict(out, Z=z.to(s["C"].dtype)) if c["keep"] else out


# ---- what a pass cannot do without ------------------------------------------


def work(case):
    op = case["op"]
    es = {"e4m3": 1, "f32": 4}.get(case["dtype"], 2)
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": T * E * es + 8 * T * k + (T * E * 2 * es + 8 * T * k if case["backward"] else 0), "flops": 0}
    half = 2 if case["gated"] else 1
    if op == "layer":
        T, k, E, D, H = case["tokens"], case["top_k"], case["experts"], case["dim"], case["hidden"]
        used = E * (1.0 - (1.0 - k / case["of"]) ** T)   # experts that some token chose, evenly routed
        held = T * k * E / case["of"]
        bias = used * (half * H + D) * es if case["bias"] else 0
        return {"bytes": int(used * (half + 1) * D * H * es + bias + T * D * es * (3 if case["residual"] else 2) + 8 * T * k),
                "flops": int(2 * held * (half + 1) * D * H)}
    rows, E, N = case["rows"], case["experts"], case["N"]
    if op == "linear_grad":
        return {"bytes": rows * N * es * (1 + 2 * half) + (4 * E * half * N if case["bias"] else 0), "flops": 4 * rows * half * N}
    K = case["K"]
    used = E * (1.0 - (1.0 - 1.0 / E) ** rows) if E > 1 else 1.0   # experts with a row, evenly routed
    outs = rows * N * (1 + (1 if case["residual"] else 0) + (half if case["keep"] else 0))
    return {"bytes": int(used * half * N * K * es + rows * K * es + 2 * outs + (2 * used * half * N if case["bias"] else 0)),
            "flops": 2 * rows * half * N * K}


# ---- the definition, in 64 bits ---------------------------------------------


def _f(name, z):
    """act(z) and its derivative, in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name in ("relu", "relu2"):
        pos = torch.where(z > 0, z, 0.0)
        return (pos, (z > 0).double()) if name == "relu" else (pos * pos, 2.0 * pos)
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    if name == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    c = 2.0 * math.sqrt(2.0 / math.pi)   # 0.5 (1 + tanh(u)) = sigmoid(2 u)
    p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
    q = torch.sigmoid(-c * (z + 0.044715 * z ** 3))
    return z * p, p + z * p * q * c * (1.0 + 0.134145 * z * z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        k, mode = case["top_k"], case["mode"]
        x = s["logits"].double().cpu()
        w, dl = torch.zeros(x.shape[0], k, dtype=torch.float64), torch.zeros_like(x)
        # order by value, then by index: the values' distinct ranks and the indexes make one integer key
        ranks = torch.unique(x, return_inverse=True)[1]
        order = torch.argsort(-(ranks * x.shape[1] + (x.shape[1] - 1 - torch.arange(x.shape[1]))), dim=1)[:, :k]
        ok = torch.gather(x, 1, order) > -math.inf
        inside = torch.zeros_like(x).scatter_(1, order, ok.double()) > 0
        u = torch.nn.functional.logsigmoid(x) if mode == "sigmoid" else x
        pool = (x > -math.inf) if mode == "all" else inside
        p = torch.softmax(torch.where(pool, u, -math.inf), dim=1)
        p = torch.where(pool, p, 0.0)
        w = torch.where(ok, torch.gather(p, 1, order), 0.0)
        out = {"ids": None, "w": w}
        if case["backward"]:
            dw = torch.zeros_like(x).scatter_add_(1, order, torch.where(ok, s["dw"].double().cpu(), 0.0))
            dl = p * (dw - (p * dw).sum(1, keepdim=True))
            out["dlogits"] = torch.where(pool, dl * torch.sigmoid(-x), 0.0) if mode == "sigmoid" else dl
        return out
    act, gated = case["act"], case["gated"]
    if op == "layer":
        H = case["hidden"]
        Y = s["residual"].double() if case["residual"] else torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            t, j = (s["ids"] == e).nonzero(as_tuple=True)
            if t.numel():
                z = s["X"][t].double() @ s["up"][e].double().T + (s["up_bias"][e].double() if case["bias"] else 0.0)
                hid = _f(act, z[:, :H])[0] * z[:, H:] if gated else _f(act, z)[0]
                y = hid @ s["down"][e].double().T + (s["down_bias"][e].double() if case["bias"] else 0.0)
                Y.index_add_(0, t, y * s["w"][t, j].double()[:, None])
        return {"Y": Y}
    rows, N, half = case["rows"], case["N"], 2 if gated else 1
    off = [0, rows] if s["offsets"] is None else s["offsets"].tolist()
    spans = [(e, a, b) for e, (a, b) in enumerate(zip(off[:-1], off[1:])) if b > a]
    if op == "linear_grad":
        dZ = torch.empty(rows, half * N, dtype=torch.float64, device="cuda")
        db = torch.zeros(case["experts"], half * N, dtype=torch.float64, device="cuda")
        for e, a, b in spans:
            d, z = s["dC"][a:b].double(), s["Z"][a:b].double()
            f, g = _f(act, z[:, :N])
            dZ[a:b, :N] = d * g * (z[:, N:] if gated else 1.0)
            if gated:
                dZ[a:b, N:] = d * f
            db[e] = dZ[a:b].sum(0)
        return {"dZ": dZ, "dbias": db} if case["bias"] else {"dZ": dZ}
    C = torch.empty(rows, N, dtype=torch.float64, device="cuda")
    Z = torch.empty(rows, half * N, dtype=torch.float64, device="cuda")
    for e, a, b in spans:
        z = s["A"][a:b].double() @ s["B"][e].double().T / (s["scale_a"] * s["scale_b"])
        Z[a:b] = z + s["bias"][e].double() if case["bias"] else z
        f = _f(act, Z[a:b, :N])[0]
        C[a:b] = f * Z[a:b, N:] if gated else f
    C = C + s["residual"].double() if case["residual"] else C
    return {"C": C, "Z": Z} if case["keep"] else {"C": C}
