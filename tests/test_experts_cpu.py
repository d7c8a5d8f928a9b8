"""The expert layer's calls on a machine without a GPU: refused without a
handle, and the binding's checks of tensors."""
import ctypes

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
