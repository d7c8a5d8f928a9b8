"""Python binding of the expert layer's operators in include/pts_gemm.h.

Names and order of arguments are the C functions'.  A tensor passed where the
C call takes a pointer is checked first (on a GPU, contiguous, of the expected
type, large enough for the sizes given); a raw device address is passed on as
it is.  ``stream`` is a torch stream or a raw handle; None is the legacy
default stream, so a caller on another torch stream passes that stream.
"""
from __future__ import annotations

import torch

from .gemm import GEMM_BF16, GEMM_E4M3, GEMM_ERR_INVALID_ARG, GEMM_F16, GemmError, _stream, load

_TORCH = {GEMM_F16: torch.float16, GEMM_BF16: torch.bfloat16, GEMM_E4M3: torch.float8_e4m3fn}
_OUT = {GEMM_F16: torch.float16, GEMM_BF16: torch.bfloat16, GEMM_E4M3: torch.bfloat16}
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


class _Calls:
    """The C functions, looked up in the library at their first call (a small
    call's host time counts: the GPU work of a decoding step is as short)."""

    def __getattr__(self, name):
        f = getattr(load(), name)
        setattr(self, name, f)
        return f


_c = _Calls()


def _arg(x, dtype, count, what):
    """Address of `x`; a tensor must be a contiguous CUDA tensor of `dtype` with at least `count` elements."""
    if x is None or x.__class__ is int:
        return x
    if x.dtype is not dtype or not x.is_cuda or not x.is_contiguous() or x.numel() < count:
        raise GemmError(GEMM_ERR_INVALID_ARG,
                        f"{what}: needs a contiguous CUDA tensor of {dtype} with at least {count} elements, got "
                        f"{tuple(x.shape)} {x.dtype} on {x.device}{'' if x.is_contiguous() else ', not contiguous'}")
    return x.data_ptr()


def _type(table, dtype, what):
    if dtype not in table:
        raise GemmError(GEMM_ERR_INVALID_ARG, f"{what}: unknown dtype {dtype!r}")
    return table[dtype]


def _done(status, what):
    if status:
        raise GemmError(status, what)
    return 0


def gemm_expert_sort(h, tokens, top_k, experts, expert_ids, offsets, row_of, src_of, stream=None) -> int:
    n = tokens * top_k
    return _done(_c.gemm_expert_sort(
        h, tokens, top_k, experts, _arg(expert_ids, _I32, n, "expert_ids"), _arg(offsets, _I32, experts + 1, "offsets"),
        _arg(row_of, _I32, n, "row_of"), _arg(src_of, _I32, n, "src_of"), _stream(stream)), "gemm_expert_sort")


def gemm_expert_gather(h, tokens, top_k, dim, X, row_of, Xs, dtype, stream=None) -> int:
    t = _type(_TORCH, dtype, "gemm_expert_gather")
    n = tokens * top_k
    return _done(_c.gemm_expert_gather(
        h, tokens, top_k, dim, _arg(X, t, tokens * dim, "X"), _arg(row_of, _I32, n, "row_of"), _arg(Xs, t, n * dim, "Xs"),
        dtype, _stream(stream)), "gemm_expert_gather")


def gemm_expert_combine(h, tokens, top_k, dim, Ys, row_of, weights, Y, dtype, stream=None) -> int:
    t = _type(_TORCH, dtype, "gemm_expert_combine")
    n = tokens * top_k
    return _done(_c.gemm_expert_combine(
        h, tokens, top_k, dim, _arg(Ys, t, n * dim, "Ys"), _arg(row_of, _I32, n, "row_of"),
        _arg(weights, _F32, n, "weights"), _arg(Y, t, tokens * dim, "Y"), dtype, _stream(stream)), "gemm_expert_combine")


def gemm_expert_combine_grad(h, tokens, top_k, dim, dY, Ys, row_of, weights, dYs, dweights, dtype, stream=None) -> int:
    t = _type(_TORCH, dtype, "gemm_expert_combine_grad")
    n = tokens * top_k
    return _done(_c.gemm_expert_combine_grad(
        h, tokens, top_k, dim, _arg(dY, t, tokens * dim, "dY"), _arg(Ys, t, n * dim, "Ys"), _arg(row_of, _I32, n, "row_of"),
        _arg(weights, _F32, n, "weights"), _arg(dYs, t, n * dim, "dYs"), _arg(dweights, _F32, n, "dweights"), dtype,
        _stream(stream)), "gemm_expert_combine_grad")


def gemm_run_experts(h, rows, experts, N, K, A, B, offsets, C, dtype, scale_a=1.0, scale_b=1.0, stream=None) -> int:
    t = _type(_TORCH, dtype, "gemm_run_experts")
    return _done(_c.gemm_run_experts(
        h, rows, experts, N, K, _arg(A, t, rows * K, "A"), _arg(B, t, experts * N * K, "B"),
        _arg(offsets, _I32, experts + 1, "offsets"), _arg(C, _OUT[dtype], rows * N, "C"), dtype, scale_a, scale_b,
        _stream(stream)), "gemm_run_experts")


def gemm_run_experts_dgrad(h, rows, experts, N, K, dC, B, offsets, dA, dtype, stream=None) -> int:
    t = _type(_TORCH, dtype, "gemm_run_experts_dgrad")
    return _done(_c.gemm_run_experts_dgrad(
        h, rows, experts, N, K, _arg(dC, t, rows * N, "dC"), _arg(B, t, experts * N * K, "B"),
        _arg(offsets, _I32, experts + 1, "offsets"), _arg(dA, t, rows * K, "dA"), dtype, _stream(stream)),
        "gemm_run_experts_dgrad")


def gemm_run_experts_wgrad(h, rows, experts, N, K, dC, A, offsets, dB, dtype, stream=None) -> int:
    t = _type(_TORCH, dtype, "gemm_run_experts_wgrad")
    return _done(_c.gemm_run_experts_wgrad(
        h, rows, experts, N, K, _arg(dC, t, rows * N, "dC"), _arg(A, t, rows * K, "A"),
        _arg(offsets, _I32, experts + 1, "offsets"), _arg(dB, t, experts * N * K, "dB"), dtype, _stream(stream)),
        "gemm_run_experts_wgrad")


def gemm_run_nibble(h, rows, experts, N, K, group, A, B, scales, zeros, offsets, C, dtype, stream=None) -> int:
    t = _type(_TORCH, dtype, "gemm_run_nibble")
    groups = experts * N * (-(-K // max(group, 1)))
    return _done(_c.gemm_run_nibble(
        h, rows, experts, N, K, group, _arg(A, t, rows * K, "A"), _arg(B, _U8, experts * N * K // 2, "B"),
        _arg(scales, t, groups, "scales"), _arg(zeros, _U8, groups, "zeros"), _arg(offsets, _I32, experts + 1, "offsets"),
        _arg(C, t, rows * N, "C"), dtype, _stream(stream)), "gemm_run_nibble")
