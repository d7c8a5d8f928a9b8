"""A layer of experts, trained and served with the library's operators.

ExpertLayer holds E pairs of matrices, up (hidden x dim) and down (dim x
hidden).  Every token goes to top_k of them:

    forward    sort -> gather -> up product -> relu^2 -> down product -> combine
    backward   combine's gradient -> down's gradients -> relu^2' -> up's
               gradients -> the gather's gradient (combine without weights)
    decode     the same forward for a few tokens with both matrices in 4 bits
               (gemm_run_nibble)

Nothing is read back in between: the experts' row counts stay on the device.

    python examples/expert_layer.py [--tokens 4096 --dim 1024 --hidden 2048 --experts 16 --top-k 2]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import persistent_tile_scheduled_gb300 as pts  # noqa: E402

DT = pts.GEMM_BF16


def _new(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def quantise(w, group):
    """(E, N, K) -> 4-bit codes (two to a byte, low half first) and a bf16 scale per group of `group` along K."""
    E, N, K = w.shape
    g = w.float().view(E, N, K // group, group)
    scale = (g.abs().amax(-1) / 7.0).clamp_(min=1e-8).to(torch.bfloat16)
    q = (g / scale.float()[..., None]).round_().clamp_(-8, 7).to(torch.int16) + 8
    q = q.to(torch.uint8).view(E, N, K // 2, 2)
    return (q[..., 0] | (q[..., 1] << 4)).contiguous(), scale.contiguous()


class ExpertLayer:
    def __init__(self, dim, hidden, experts, top_k, seed=0, group=128, device=0):
        self.dim, self.hidden, self.experts, self.top_k, self.group = dim, hidden, experts, top_k, group
        gen = torch.Generator().manual_seed(seed)
        self.up = (torch.randn(experts, hidden, dim, generator=gen) / dim ** 0.5).to(torch.bfloat16).cuda()
        self.down = (torch.randn(experts, dim, hidden, generator=gen) / hidden ** 0.5).to(torch.bfloat16).cuda()
        self.up4, self.down4 = quantise(self.up, group), quantise(self.down, group)
        self.h = pts.gemm_create(device)

    def close(self):
        pts.gemm_destroy(self.h)

    def _route(self, ids):
        T, k, E = ids.shape[0], self.top_k, self.experts
        offsets, row_of, src_of = _new(E + 1, dtype=torch.int32), _new(T, k, dtype=torch.int32), _new(T * k, dtype=torch.int32)
        pts.gemm_expert_sort(self.h, T, k, E, ids, offsets, row_of, src_of, stream=torch.cuda.current_stream())
        return offsets, row_of

    def forward(self, x, ids, weights):
        """x (T, dim) bf16, ids (T, top_k) int32 (outside [0, experts): not this layer's), weights (T, top_k) fp32."""
        T, k, D, H, E, s = x.shape[0], self.top_k, self.dim, self.hidden, self.experts, torch.cuda.current_stream()
        offsets, row_of = self._route(ids)
        # rows of no expert stay as they are: zeros keep the elementwise steps finite
        xs, a = torch.zeros(T * k, D, dtype=x.dtype, device="cuda"), torch.zeros(T * k, H, dtype=x.dtype, device="cuda")
        ys, y = _new(T * k, D), _new(T, D)
        pts.gemm_expert_gather(self.h, T, k, D, x, row_of, xs, DT, stream=s)
        pts.gemm_run_experts(self.h, T * k, E, H, D, xs, self.up, offsets, a, DT, stream=s)
        r = a.relu()
        z = r * r
        pts.gemm_run_experts(self.h, T * k, E, D, H, z, self.down, offsets, ys, DT, stream=s)
        pts.gemm_expert_combine(self.h, T, k, D, ys, row_of, weights, y, DT, stream=s)
        return y, (x, offsets, row_of, weights, xs, r, z, ys)

    def backward(self, dy, saved):
        """-> dx, d(weights), d(up), d(down)."""
        x, offsets, row_of, weights, xs, r, z, ys = saved
        T, k, D, H, E, s = x.shape[0], self.top_k, self.dim, self.hidden, self.experts, torch.cuda.current_stream()
        R = T * k
        dys, dw = torch.zeros_like(ys), torch.empty_like(weights)
        dz, da, dxs, dx = torch.zeros_like(z), None, _new(R, D), _new(T, D)
        dup, ddown = torch.empty_like(self.up), torch.empty_like(self.down)
        pts.gemm_expert_combine_grad(self.h, T, k, D, dy, ys, row_of, weights, dys, dw, DT, stream=s)
        pts.gemm_run_experts_dgrad(self.h, R, E, D, H, dys, self.down, offsets, dz, DT, stream=s)
        pts.gemm_run_experts_wgrad(self.h, R, E, D, H, dys, z, offsets, ddown, DT, stream=s)
        da = 2.0 * r * dz
        pts.gemm_run_experts_dgrad(self.h, R, E, H, D, da, self.up, offsets, dxs, DT, stream=s)
        pts.gemm_run_experts_wgrad(self.h, R, E, H, D, da, xs, offsets, dup, DT, stream=s)
        pts.gemm_expert_combine(self.h, T, k, D, dxs, row_of, None, dx, DT, stream=s)
        return dx, dw, dup, ddown

    def decode(self, x, ids, weights):
        """forward for a few tokens, the matrices in 4 bits."""
        T, k, D, H, E, s = x.shape[0], self.top_k, self.dim, self.hidden, self.experts, torch.cuda.current_stream()
        offsets, row_of = self._route(ids)
        xs, a = torch.zeros(T * k, D, dtype=x.dtype, device="cuda"), torch.zeros(T * k, H, dtype=x.dtype, device="cuda")
        ys, y = _new(T * k, D), _new(T, D)
        pts.gemm_expert_gather(self.h, T, k, D, x, row_of, xs, DT, stream=s)
        pts.gemm_run_nibble(self.h, T * k, E, H, D, self.group, xs, *self.up4, None, offsets, a, DT, stream=s)
        z = a.relu().square()
        pts.gemm_run_nibble(self.h, T * k, E, D, H, self.group, z, *self.down4, None, offsets, ys, DT, stream=s)
        pts.gemm_expert_combine(self.h, T, k, D, ys, row_of, weights, y, DT, stream=s)
        return y


def router(x, gate, top_k):
    """Expert ids and weights of the top_k largest scores, softmax over those."""
    v, ids = torch.topk(x.float() @ gate, top_k, dim=1)
    return ids.to(torch.int32).contiguous(), torch.softmax(v, dim=1).contiguous()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--dim", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=2)
    ap.add_argument("--decode-tokens", type=int, default=4)
    a = ap.parse_args()
    layer = ExpertLayer(a.dim, a.hidden, a.experts, a.top_k)
    gen = torch.Generator().manual_seed(1)
    gate = torch.randn(a.dim, a.experts, generator=gen).cuda() / a.dim ** 0.5

    def timed(what, f, flops):
        f()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        for _ in range(10):
            f()
        end.record()
        torch.cuda.synchronize()
        us = begin.elapsed_time(end) * 100.0
        print(f"{what:10} {us:9.1f} us  {flops / us / 1e6:8.1f} TFLOP/s")

    x = torch.randn(a.tokens, a.dim, generator=gen).to(torch.bfloat16).cuda()
    ids, w = router(x, gate, a.top_k)
    per_pass = 4.0 * a.tokens * a.top_k * a.dim * a.hidden
    y, saved = layer.forward(x, ids, w)
    timed("forward", lambda: layer.forward(x, ids, w), per_pass)
    timed("backward", lambda: layer.backward(y, saved), 2 * per_pass)
    xd = x[:a.decode_tokens].contiguous()
    idd, wd = router(xd, gate, a.top_k)
    timed("decode", lambda: layer.decode(xd, idd, wd), 4.0 * a.decode_tokens * a.top_k * a.dim * a.hidden)
    y4 = layer.decode(xd, idd, wd).float()
    print(f"decode in 4 bits against bf16: {float((y4 - y[:a.decode_tokens].float()).norm() / y4.norm()):.3f} of the norm")
    status, word = pts.gemm_check(layer.h)
    layer.close()
    return 0 if status == 0 else f"device status {word:#x}"


if __name__ == "__main__":
    sys.exit(main())
