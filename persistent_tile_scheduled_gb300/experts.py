"""Python binding of the expert layer's operators in include/pts_gemm.h.

Names and order of arguments are the C functions'.  A tensor passed where the
C call takes a pointer is checked first (on the handle's GPU, contiguous, of
the expected type, large enough for the sizes given); a raw device address is
passed on as it is.  ``stream`` is a torch stream or a raw handle; None is the legacy
default stream, so a caller on another torch stream passes that stream.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util

import torch

from . import _build
from .gemm import GEMM_ERR_INVALID_ARG, GemmError, load


def _refuse(what, x, dtype, count, device=-1):
    """Raises for an argument that the extension module does not take: not a dtype (x is None), or not such a tensor."""
    if x is None:
        raise GemmError(GEMM_ERR_INVALID_ARG, f"{what}: unknown dtype {count}")
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{what}: needs a tensor, an address or None, got {type(x).__name__}")
    where = f" on cuda:{device}" if device >= 0 else ""
    raise GemmError(GEMM_ERR_INVALID_ARG,
                    f"{what}: needs a contiguous CUDA tensor{where} of {dtype} with at least {count} elements, got "
                    f"{tuple(x.shape)} {x.dtype} on {x.device}{'' if x.is_contiguous() else ', not contiguous'}")


def _setup(module):
    module.setup(torch.Tensor, _refuse, torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.float32,
                 torch.uint8)


_FUNCTIONS = ("expert_sort", "expert_gather", "expert_combine", "expert_combine_grad", "run_experts", "run_experts_dgrad",
              "run_experts_wgrad", "run_nibble")


class _Calls:
    """The functions of the extension module, which is loaded (and built, if it has to be) at the first call."""

    def __getattr__(self, name):
        if name != "module" and name not in _FUNCTIONS:
            raise AttributeError(name)
        load()
        loader = importlib.machinery.ExtensionFileLoader("pts_experts", _build.build_experts())
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("pts_experts", loader))
        loader.exec_module(module)
        _setup(module)
        self.module = module
        for f in _FUNCTIONS:
            setattr(self, f, getattr(module, f))
        return self.__dict__[name]


_c = _Calls()


def gemm_expert_sort(h, tokens, top_k, experts, expert_ids, offsets, row_of, src_of, stream=None) -> int:
    status = _c.expert_sort(h, tokens, top_k, experts, expert_ids, offsets, row_of, src_of, stream)
    if status:
        raise GemmError(status, "gemm_expert_sort")
    return 0


def gemm_expert_gather(h, tokens, top_k, dim, X, row_of, Xs, dtype, stream=None) -> int:
    status = _c.expert_gather(dtype, h, tokens, top_k, dim, X, row_of, Xs, stream)
    if status:
        raise GemmError(status, "gemm_expert_gather")
    return 0


def gemm_expert_combine(h, tokens, top_k, dim, Ys, row_of, weights, Y, dtype, stream=None) -> int:
    status = _c.expert_combine(dtype, h, tokens, top_k, dim, Ys, row_of, weights, Y, stream)
    if status:
        raise GemmError(status, "gemm_expert_combine")
    return 0


def gemm_expert_combine_grad(h, tokens, top_k, dim, dY, Ys, row_of, weights, dYs, dweights, dtype, stream=None) -> int:
    status = _c.expert_combine_grad(dtype, h, tokens, top_k, dim, dY, Ys, row_of, weights, dYs, dweights, stream)
    if status:
        raise GemmError(status, "gemm_expert_combine_grad")
    return 0


def gemm_run_experts(h, rows, experts, N, K, A, B, offsets, C, dtype, scale_a=1.0, scale_b=1.0, stream=None) -> int:
    status = _c.run_experts(dtype, h, rows, experts, N, K, A, B, offsets, C, scale_a, scale_b, stream)
    if status:
        raise GemmError(status, "gemm_run_experts")
    return 0


def gemm_run_experts_dgrad(h, rows, experts, N, K, dC, B, offsets, dA, dtype, stream=None) -> int:
    status = _c.run_experts_dgrad(dtype, h, rows, experts, N, K, dC, B, offsets, dA, stream)
    if status:
        raise GemmError(status, "gemm_run_experts_dgrad")
    return 0


def gemm_run_experts_wgrad(h, rows, experts, N, K, dC, A, offsets, dB, dtype, stream=None) -> int:
    status = _c.run_experts_wgrad(dtype, h, rows, experts, N, K, dC, A, offsets, dB, stream)
    if status:
        raise GemmError(status, "gemm_run_experts_wgrad")
    return 0


def gemm_run_nibble(h, rows, experts, N, K, group, A, B, scales, zeros, offsets, C, dtype, stream=None) -> int:
    status = _c.run_nibble(dtype, h, rows, experts, N, K, group, A, B, scales, zeros, offsets, C, stream)
    if status:
        raise GemmError(status, "gemm_run_nibble")
    return 0
