"""The expert layer's calls on a machine without a GPU: refused without a
handle, and the binding's checks of tensors."""
import ctypes

import numpy as np
import pytest
import torch

import persistent_tile_scheduled_gb300 as pts
from persistent_tile_scheduled_gb300 import gemm as g

CALLS = {
    "gemm_expert_sort": [4, 2, 8],
    "gemm_expert_gather": [4, 2, 64],
    "gemm_expert_combine": [4, 2, 64],
    "gemm_expert_combine_grad": [4, 2, 64],
    "gemm_run_experts": [4, 2, 64, 64],
    "gemm_run_experts_dgrad": [4, 2, 64, 64],
    "gemm_run_experts_wgrad": [4, 2, 64, 64],
    "gemm_run_nibble": [4, 2, 64, 64, 32],
}


@pytest.mark.parametrize("name", CALLS)
def test_refused_without_a_handle(name):
    f = getattr(pts.load(), name)
    args = [None] + CALLS[name]
    args += [0 if t is not ctypes.c_void_p else None for t in f.argtypes[len(args):]]
    assert f(*args) == g.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("name", CALLS)
def test_tensors_are_checked_before_the_call(name):
    """A host tensor, whatever its size, is refused with the library's own error."""
    n = {"gemm_expert_sort": 4, "gemm_expert_gather": 3, "gemm_expert_combine": 4, "gemm_expert_combine_grad": 6,
         "gemm_run_nibble": 6}.get(name, 4)
    x = torch.zeros(1 << 16, dtype=torch.float16)
    with pytest.raises(pts.GemmError) as err:
        getattr(pts, name)(None, *CALLS[name], *([x] * n), *([0] if name != "gemm_expert_sort" else []))
    assert err.value.status == g.GEMM_ERR_INVALID_ARG and "contiguous CUDA tensor" in str(err.value)


def _args(name, arrays=None):
    n = {"gemm_expert_sort": 4, "gemm_expert_gather": 3, "gemm_expert_combine": 4, "gemm_expert_combine_grad": 6,
         "gemm_run_nibble": 6}.get(name, 4)
    return CALLS[name] + [arrays] * n + ([g.GEMM_F16] if name != "gemm_expert_sort" else [])


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [None, 0, 1 << 40])
def test_raw_addresses_reach_the_call(name, stream):
    """Addresses and sizes pass as they are (numpy's integers too); without a handle the C call refuses them."""
    args = [np.int64(v) if v == 4 else v for v in _args(name, 1 << 20)]
    with pytest.raises(pts.GemmError) as err:
        getattr(pts, name)(None, *args, stream=stream)
    assert err.value.status == g.GEMM_ERR_INVALID_ARG and name in str(err.value)


@pytest.mark.parametrize("name", CALLS)
def test_arguments_of_other_types_are_errors(name):
    f = getattr(pts, name)
    for args in ([None] + _args(name, "x"), [None] + _args(name, [1, 2]), ["x"] + _args(name),
                 [None, 4.5] + _args(name)[1:], [None, 1 << 70] + _args(name)[1:]):
        with pytest.raises((TypeError, OverflowError)):
            f(*args)
    with pytest.raises(AttributeError):
        f(None, *_args(name), stream="x")
    with pytest.raises(TypeError):
        f(None, 4)
    if name != "gemm_expert_sort":
        with pytest.raises(pts.GemmError, match="unknown dtype 9"):
            f(None, *_args(name)[:-1], 9)


def test_sizes_whose_product_passes_64_bits_want_more_than_any_tensor_has():
    x = torch.zeros(16, dtype=torch.float16, device="meta")
    with pytest.raises(pts.GemmError) as err:
        pts.gemm_run_experts(None, 4, 1 << 40, 1 << 40, 64, 1 << 20, x, 1 << 20, 1 << 20, g.GEMM_F16)
    assert "contiguous CUDA tensor" in str(err.value) and str((1 << 63) - 1) in str(err.value)
