"""The operators of a sparse expert layer, as cases that can be timed and compared.

A layer with E experts sends each of T tokens to top_k of them.  The operators:

  dispatch      assignments sorted by expert (gemm_expert_sort) and the tokens'
                rows copied into that order (gemm_expert_gather)
  combine       the experts' rows back in token order, summed with the router's
                weights (gemm_expert_combine); without weights it is the
                gradient of the copy above
  combine_grad  its gradient: rows and weights (gemm_expert_combine_grad)
  experts       C[r] = A[r] . B_e^T for every row r of expert e
                (gemm_run_experts), rows sorted by expert, counts on the device
  experts_dx    its gradient for the rows (gemm_run_experts_dgrad)
  experts_dw    its gradient for the weights (gemm_run_experts_wgrad)
  nibble        the same product for few rows with 4-bit weights and a scale
                (and zero) per group of `group` of them (gemm_run_nibble);
                experts = 1 is one ordinary weight matrix

`run` computes a case in its plain form, or with the framework's kernels where
`own` is set.  Sizes are those of this repository's benchmark (4096, 8192,
5120, 4224, 2048, 1024 and their kind) or generic.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_CODE = {"f16": 0, "bf16": 1, "e4m3": 2}
_library = None


def listed():
    return [
        # a decoding step of a small batch: latency
        dict(name="dispatch_decode", op="dispatch", tokens=16, top_k=2, experts=8, of=8, dim=4096, skew=0.0, dtype="bf16"),
        # a long prefill on a device that holds half of the experts
        dict(name="dispatch_prefill", op="dispatch", tokens=16384, top_k=4, experts=32, of=64, dim=4096, skew=0.5, dtype="bf16"),
        # the way back of an odd number of tokens
        dict(name="combine_ragged", op="combine", tokens=4101, top_k=2, experts=8, of=8, dim=4224, skew=0.3, dtype="f16", weighted=True),
        # the same in a training step, backward
        dict(name="combine_grad_train", op="combine_grad", tokens=8192, top_k=4, experts=64, of=64, dim=5120, skew=0.5, dtype="bf16"),
        # experts' products of a decoding batch: a few rows each, the weights' bytes count
        dict(name="experts_decode", op="experts", rows=40, spare=0, experts=8, N=4096, K=4096, skew=0.0, dtype="bf16"),
        # a training step's products: few large experts, unevenly filled
        dict(name="experts_train", op="experts", rows=16384, spare=0, experts=8, N=8192, K=4096, skew=0.4, dtype="bf16"),
        # prefill in 8 bits: more experts, odd row counts
        dict(name="experts_prefill_e4m3", op="experts", rows=8191, spare=65, experts=16, N=4096, K=8192, skew=0.3, dtype="e4m3"),
        # the backward products of a training step
        dict(name="experts_dx_train", op="experts_dx", rows=8192, spare=0, experts=16, N=4096, K=5120, skew=0.4, dtype="bf16"),
        dict(name="experts_dw_train", op="experts_dw", rows=16384, spare=0, experts=8, N=4096, K=4096, skew=0.4, dtype="f16"),
        # one token against one projection: latency
        dict(name="nibble_one", op="nibble", rows=1, experts=1, N=4096, K=4096, group=128, zeros=False, skew=0.0, dtype="f16"),
        # a small batch against a wide projection, fine groups with zeros
        dict(name="nibble_wide", op="nibble", rows=8, experts=1, N=16384, K=8192, group=32, zeros=True, skew=0.0, dtype="bf16"),
        # a decoding batch's experts in 4 bits
        dict(name="nibble_experts", op="nibble", rows=16, experts=32, N=2048, K=4096, group=64, zeros=False, skew=0.0, dtype="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, lo), hi // step * step)


def _draw_one(rng):
    op = rng.choice(["dispatch", "combine", "combine_grad", "experts", "experts", "experts_dx", "experts_dw", "nibble", "nibble"])
    skew = round(rng.uniform(0.0, 0.6), 2)
    if op in ("dispatch", "combine", "combine_grad"):
        experts = _log(rng, 2, 128)
        c = dict(op=op, tokens=_log(rng, 1, 20000), top_k=min(rng.choice([1, 2, 3, 4, 6, 8]), experts), experts=experts,
                 of=experts * rng.choice([1, 1, 2, 4]), dim=_log(rng, 256, 8192, 8), skew=skew, dtype=rng.choice(["f16", "bf16"]))
        return dict(c, weighted=rng.random() < 0.6) if op == "combine" else c
    if op == "nibble":
        few = rng.random() < 0.5
        return dict(op=op, rows=_log(rng, 1, 32), experts=1 if few else _log(rng, 2, 64), N=_log(rng, 256, 16384, 8),
                    K=_log(rng, 256, 16384, 32), group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, skew=skew,
                    dtype=rng.choice(["f16", "bf16"]))
    dtype = rng.choice(["f16", "bf16", "e4m3"] if op == "experts" else ["f16", "bf16"])
    return dict(op=op, rows=_log(rng, 1 if op == "experts" else 256, 16384), spare=rng.choice([0, 0, 37]), experts=_log(rng, 2, 64),
                N=_log(rng, 256, 8192, 16), K=_log(rng, 256, 8192, 16), skew=skew, dtype=dtype)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        c = _draw_one(rng)
        weights = c.get("experts", 1) * c.get("N", 0) * c.get("K", 0)
        copied = c.get("tokens", 0) * (c.get("top_k", 0) + 1) * c.get("dim", 0)
        some_held = c["op"] not in ("dispatch", "combine", "combine_grad") or c["tokens"] * c["top_k"] * c["experts"] >= 16 * c["of"] or c["of"] == c["experts"]
        if not some_held or 3072 in c.values() or weights > 1 << 28 or copied > 8192 * 9 * 5120 or _cost(c) > most:
            continue
        return c


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


# ---- inputs -----------------------------------------------------------------


def _ids(gen, rows, experts, skew, top_k=1):
    """top_k different experts for each row, expert e preferred by -skew * log(e + 1)."""
    u = torch.rand(rows, experts, generator=gen, device="cuda").clamp_(1e-7, 1.0 - 1e-7)
    score = -torch.log(-torch.log(u)) - skew * torch.log(torch.arange(1, experts + 1, device="cuda", dtype=torch.float32))
    return torch.topk(score, top_k, dim=1).indices


def _normal(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dt = case["op"], _DT[case["dtype"]]
    s = {"case": case}
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, E, D = case["tokens"], case["top_k"], case["experts"], case["dim"]
        # the router ranks all `of` experts; this device holds E of them, from `base` on
        base = (case["of"] - E) // 2
        ids = (_ids(gen, T, case["of"], case["skew"], k) - base).to(torch.int32).contiguous()
        w = torch.softmax(_normal(gen, T, k), dim=1).contiguous()
        if op == "dispatch":
            s.update(ids=ids, X=_normal(gen, T, D).to(dt), offsets=_zeros(E + 1, torch.int32), row_of=_zeros((T, k), torch.int32),
                     src_of=_zeros(T * k, torch.int32), Xs=_zeros((T * k, D), dt))
            return s
        held = (ids >= 0) & (ids < E)
        order = torch.sort(torch.where(held, ids, E).reshape(-1), stable=True).indices
        row_of = torch.empty(T * k, dtype=torch.int32, device="cuda")
        row_of[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
        s.update(row_of=torch.where(held, row_of.view(T, k), -1).contiguous(), Ys=_normal(gen, T * k, D).to(dt),
                 w=w if case.get("weighted", True) else None)
        if op == "combine":
            s.update(Y=_zeros((T, D), dt))
        else:
            s.update(dY=_normal(gen, T, D).to(dt), dYs=_zeros((T * k, D), dt), dw=_zeros((T, k), torch.float32))
        return s
    rows, E, N, K = case["rows"], case["experts"], case["N"], case["K"]
    counts = torch.bincount(_ids(gen, rows, E, case["skew"]).reshape(-1), minlength=E)
    offsets = _zeros(E + 1, torch.int32)
    offsets[1:] = torch.cumsum(counts, 0)
    s.update(offsets=offsets, most=int(counts.max()))
    if op == "nibble":
        g = case["group"]
        groups = -(-K // g)
        q = (_normal(gen, E, N, K) * 2.6 + 8.0).round_().clamp_(0, 15).to(torch.uint8).view(E, N, K // 2, 2)
        s.update(A=_normal(gen, rows, K).to(dt), B=(q[..., 0] | (q[..., 1] << 4)).contiguous(),
                 scales=((torch.rand(E, N, groups, generator=gen, device="cuda") + 0.5) * (0.4 / math.sqrt(K))).to(dt),
                 zeros=torch.randint(5, 12, (E, N, groups), generator=gen, device="cuda", dtype=torch.uint8) if case["zeros"] else None,
                 C=_zeros((rows, N), dt))
        return s
    all_rows = rows + case["spare"]
    if dt == torch.float8_e4m3fn:   # scaled so that the largest value is the type's largest
        a, b = _normal(gen, all_rows, K), _normal(gen, E, N, K)
        s.update(scale_a=448.0 / float(a.abs().max()), scale_b=448.0 / float(b.abs().max()))
        s.update(A=(a * s["scale_a"]).clamp_(-448, 448).to(dt), B=(b * s["scale_b"]).clamp_(-448, 448).to(dt),
                 C=_zeros((all_rows, N), torch.bfloat16))
        return s
    if op == "experts":
        s.update(A=_normal(gen, all_rows, K).to(dt), B=_normal(gen, E, N, K, scale=1.0 / math.sqrt(K)).to(dt), C=_zeros((all_rows, N), dt))
    elif op == "experts_dx":
        s.update(dC=_normal(gen, all_rows, N).to(dt), B=_normal(gen, E, N, K, scale=1.0 / math.sqrt(K)).to(dt), dA=_zeros((all_rows, K), dt))
    else:
        s.update(dC=_normal(gen, all_rows, N, scale=1.0 / 16).to(dt), A=_normal(gen, all_rows, K).to(dt), dB=_zeros((E, N, K), dt))
    return s


def _zeros(shape, dtype):
    return torch.zeros(shape, dtype=dtype, device="cuda")


# ---- one pass ---------------------------------------------------------------


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    global _library
    if _library is None:
        import persistent_tile_scheduled_gb300 as pts
        _library = (pts, pts.gemm_create(0))
    pts, h = _library
    c = s["case"]
    op, dt = c["op"], _CODE[c["dtype"]]
    if op == "dispatch":
        pts.gemm_expert_sort(h, c["tokens"], c["top_k"], c["experts"], s["ids"], s["offsets"], s["row_of"], s["src_of"])
        pts.gemm_expert_gather(h, c["tokens"], c["top_k"], c["dim"], s["X"], s["row_of"], s["Xs"], dt)
        return {"offsets": s["offsets"], "row_of": s["row_of"], "src_of": s["src_of"], "Xs": s["Xs"]}
    if op == "combine":
        pts.gemm_expert_combine(h, c["tokens"], c["top_k"], c["dim"], s["Ys"], s["row_of"], s["w"], s["Y"], dt)
        return {"Y": s["Y"]}
    if op == "combine_grad":
        pts.gemm_expert_combine_grad(h, c["tokens"], c["top_k"], c["dim"], s["dY"], s["Ys"], s["row_of"], s["w"], s["dYs"], s["dw"], dt)
        return {"dYs": s["dYs"], "dw": s["dw"]}
    E, N, K = c["experts"], c["N"], c["K"]
    if op == "nibble":
        pts.gemm_run_nibble(h, c["rows"], E, N, K, c["group"], s["A"], s["B"], s["scales"], s["zeros"], s["offsets"], s["C"], dt)
        return {"C": s["C"]}
    rows = c["rows"] + c["spare"]
    if op == "experts":
        pts.gemm_run_experts(h, rows, E, N, K, s["A"], s["B"], s["offsets"], s["C"], dt, s.get("scale_a", 1.0), s.get("scale_b", 1.0))
        return {"C": s["C"]}
    if op == "experts_dx":
        pts.gemm_run_experts_dgrad(h, rows, E, N, K, s["dC"], s["B"], s["offsets"], s["dA"], dt)
        return {"dA": s["dA"]}
    pts.gemm_run_experts_wgrad(h, rows, E, N, K, s["dC"], s["A"], s["offsets"], s["dB"], dt)
    return {"dB": s["dB"]}


def _padded(x, offsets, most):
    """Rows sorted by expert -> (experts, most, columns) in 32 bits, zeros behind each expert's last row."""
    at = offsets[:-1, None].long() + torch.arange(most, device="cuda")
    there = at < offsets[1:, None]
    return torch.where(there[..., None], x.float()[at.clamp_(max=x.shape[0] - 1)], 0.0)


def _sorted(y, offsets, rows):
    """The way back: (experts, most, columns) -> (rows, columns), zeros behind the last expert's rows."""
    r = torch.arange(rows, device="cuda")
    e = (r[:, None] >= offsets[None, 1:]).sum(1)
    there = e < y.shape[0]
    e = e.clamp_(max=y.shape[0] - 1)
    return torch.where(there[:, None], y[e, (r - offsets[e].long()).clamp_(max=y.shape[1] - 1)], 0.0)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "dispatch":
        E, k = c["experts"], c["top_k"]
        ids, n = s["ids"].reshape(-1), s["ids"].numel()
        held = (ids >= 0) & (ids < E)
        key, order = torch.sort(torch.where(held, ids, E), stable=True)
        offsets = (key[None, :] < torch.arange(E + 1, device="cuda")[:, None]).sum(1)
        row_of = torch.empty_like(order)
        row_of[order] = torch.arange(n, device="cuda")
        src = torch.where(key < E, order, -1)
        Xs = torch.where((src >= 0)[:, None], s["X"][src.clamp(min=0) // k], 0.0)
        return {"offsets": offsets.int(), "row_of": torch.where(held, row_of, -1).int().view(-1, k), "src_of": src.int(), "Xs": Xs}
    if op == "combine":
        there = s["row_of"] >= 0
        y = torch.where(there[..., None], s["Ys"][s["row_of"].clamp(min=0)].float(), 0.0)
        y = y if s["w"] is None else y * s["w"][..., None]
        return {"Y": y.sum(1).to(s["Ys"].dtype)}
    if op == "combine_grad":
        there = s["row_of"] >= 0
        y = torch.where(there[..., None], s["Ys"][s["row_of"].clamp(min=0)].float(), 0.0)
        d = s["dY"].float()[:, None, :]
        dYs = torch.zeros_like(s["Ys"])
        dYs[s["row_of"][there]] = (d * s["w"][..., None])[there].to(dYs.dtype)
        return {"dYs": dYs, "dw": (y * d).sum(2)}
    off, most = s["offsets"], s["most"]
    if op == "nibble":
        E, N, K = c["experts"], c["N"], c["K"]
        group = torch.arange(K, device="cuda") // c["group"]
        q = torch.stack([s["B"] & 15, s["B"] >> 4], dim=-1).view(E, N, K).float()
        z = 8.0 if s["zeros"] is None else s["zeros"].float()[..., group]
        w = (q - z) * s["scales"].float()[..., group]
        return {"C": _sorted(torch.bmm(_padded(s["A"], off, most), w.transpose(1, 2)), off, c["rows"]).to(s["A"].dtype)}
    rows = c["rows"] + c["spare"]
    if op == "experts":
        y = torch.bmm(_padded(s["A"], off, most), s["B"].float().transpose(1, 2))
        y = y / (s["scale_a"] * s["scale_b"]) if "scale_a" in s else y
        return {"C": _sorted(y, off, rows).to(s["C"].dtype)}
    if op == "experts_dx":
        return {"dA": _sorted(torch.bmm(_padded(s["dC"], off, most), s["B"].float()), off, rows).to(s["dC"].dtype)}
    return {"dB": torch.bmm(_padded(s["dC"], off, most).transpose(1, 2), _padded(s["A"], off, most)).to(s["A"].dtype)}


# ---- what a pass cannot do without ------------------------------------------


def work(case):
    op = case["op"]
    es = 1 if case["dtype"] == "e4m3" else 2
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, D = case["tokens"], case["top_k"], case["dim"]
        held = T * k * case["experts"] / case["of"]
        row = D * es
        tokens = T * (1.0 - (1.0 - case["experts"] / case["of"]) ** k)   # tokens with a held expert
        if op == "dispatch":
            return {"bytes": int(12 * T * k + 4 * case["experts"] + tokens * row + held * row), "flops": 0}
        w = 4 * T * k if case.get("weighted", True) else 0
        if op == "combine":
            return {"bytes": int(4 * T * k + w + held * row + T * row), "flops": int(2 * held * D)}
        return {"bytes": int(4 * T * k + 2 * w + tokens * row + 2 * held * row), "flops": int(3 * held * D)}
    rows, E, N, K = case["rows"], case["experts"], case["N"], case["K"]
    used = E * (1.0 - (1.0 - 1.0 / E) ** rows) if E > 1 else 1.0   # experts with a row, evenly routed
    flops = 2 * rows * N * K
    if op == "nibble":
        groups = -(-K // case["group"])
        return {"bytes": int(used * N * (K // 2 + groups * (3 if case["zeros"] else 2)) + 2 * rows * (K + N)), "flops": flops}
    if op == "experts":
        return {"bytes": int(used * N * K * es + rows * K * es + 2 * rows * N), "flops": flops}
    if op == "experts_dx":
        return {"bytes": int(used * N * K * es + es * rows * (K + N)), "flops": flops}
    return {"bytes": int(E * N * K * es + es * rows * (K + N)), "flops": flops}


# ---- the definition, in 64 bits ---------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        # copies and whole numbers: row r of Xs is the token of the r-th held assignment, expert by expert
        ids, k = s["ids"].cpu().reshape(-1), case["top_k"]
        at = [i for e in range(case["experts"]) for i in (ids == e).nonzero().flatten().tolist()]
        Xs = torch.zeros(s["Xs"].shape, dtype=torch.float64, device="cuda")
        if at:
            Xs[: len(at)] = s["X"].double()[torch.tensor(at, device="cuda") // k]
        return {"offsets": None, "row_of": None, "src_of": None, "Xs": Xs}
    if op in ("combine", "combine_grad"):
        T, k, D = case["tokens"], case["top_k"], case["dim"]
        w = s["w"].double() if s["w"] is not None else torch.ones(T, k, dtype=torch.float64, device="cuda")
        Y = torch.zeros(T, D, dtype=torch.float64, device="cuda")
        dYs = torch.zeros(T * k, D, dtype=torch.float64, device="cuda") if op == "combine_grad" else None
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = (s["row_of"][:, j] >= 0).nonzero().flatten()
            r = s["row_of"][t, j].long()
            y = s["Ys"][r].double()
            if op == "combine":
                Y.index_add_(0, t, y * w[t, j, None])
            else:
                d = s["dY"][t].double()
                dYs.index_copy_(0, r, d * w[t, j, None])
                dw[t, j] = torch.einsum("td,td->t", y, d)
        return {"Y": Y} if op == "combine" else {"dYs": dYs, "dw": dw}
    off = s["offsets"].tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(case["experts"])]
    if op == "nibble":
        C = torch.zeros(case["rows"], case["N"], dtype=torch.float64, device="cuda")
        for e, a, b in spans:
            if b > a:
                x = s["A"][a:b].double()
                for j in range(s["scales"].shape[2]):
                    lo, hi = j * case["group"], min((j + 1) * case["group"], case["K"])
                    byte = s["B"][e, :, lo // 2 : hi // 2].double()
                    high = torch.floor(byte / 16)
                    zero = s["zeros"][e, :, j, None].double() if s["zeros"] is not None else 8.0
                    part = x[:, lo:hi:2] @ (byte - 16 * high - zero).T + x[:, lo + 1 : hi : 2] @ (high - zero).T
                    C[a:b] += part * s["scales"][e, :, j].double()
        return {"C": C}
    rows, N, K = case["rows"] + case["spare"], case["N"], case["K"]
    if op == "experts":
        C = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
        for e, a, b in spans:
            C[a:b] = s["A"][a:b].double() @ s["B"][e].double().T
        return {"C": C / (s["scale_a"] * s["scale_b"]) if "scale_a" in s else C}
    if op == "experts_dx":
        dA = torch.zeros(rows, K, dtype=torch.float64, device="cuda")
        for e, a, b in spans:
            dA[a:b] = s["dC"][a:b].double() @ s["B"][e].double()
        return {"dA": dA}
    dB = torch.zeros(case["experts"], N, K, dtype=torch.float64, device="cuda")
    for e, a, b in spans:
        dB[e] = s["dC"][a:b].double().T @ s["A"][a:b].double()
    return {"dB": dB}
