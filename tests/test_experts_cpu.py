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


class _Elsewhere:
    """A tensor as the extension module sees one, on a GPU of choice."""
    def __init__(self, device, dtype):
        self.where, self.kind = device, dtype

    dtype = property(lambda self: self.kind)
    is_cuda = property(lambda self: self.where >= 0)
    get_device = lambda self: self.where  # noqa: E731
    is_contiguous = lambda self: True  # noqa: E731
    numel = lambda self: 1 << 20  # noqa: E731
    data_ptr = lambda self: 1 << 20  # noqa: E731


def test_a_tensor_of_another_gpu_than_the_handles_is_refused():
    from persistent_tile_scheduled_gb300 import experts
    module, handle = experts._c.module, (ctypes.c_int32 * 64)(1)   # a handle begins with its device
    h = ctypes.addressof(handle)

    def refuse(what, x, dtype, count, device=None):
        raise KeyError((what, x.where, device))

    types = (torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.float32, torch.uint8)
    module.setup(_Elsewhere, refuse, *types)
    try:
        for where in ([0, 1, 1, 1], [1, 1, 1, 0], [1, 2, 1, 1], [1, 1, -1, 1]):
            at, wrong = next((i, w) for i, w in enumerate(where) if w != 1)
            with pytest.raises(KeyError) as err:
                module.expert_sort(h, 4, 2, 2000, *[_Elsewhere(w, torch.int32) for w in where], None)
            assert err.value.args[0] == (("expert_ids", "offsets", "row_of", "src_of")[at], wrong, 1)
        # all on the handle's: the C call is made, and refuses 2000 experts
        assert module.expert_sort(h, 4, 2, 2000, *[_Elsewhere(1, torch.int32)] * 4, None) == g.GEMM_ERR_INVALID_ARG
    finally:
        experts._setup(module)
