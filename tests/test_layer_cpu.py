"""What stands around the products, on a machine without a GPU: calls are refused without a handle, the binding checks tensors, and
the plain forms that the GPU tests compare with are themselves compared with differences."""
import ctypes

import pytest
import torch

import layer_reference as ref
import persistent_tile_scheduled_gb300 as pts
from persistent_tile_scheduled_gb300 import gemm as g

# sizes, arrays, what follows them
CALLS = {
    "gemm_run_linear": ([4, 2, 64, 64], 7, [0, g.GEMM_F16]),
    "gemm_linear_grad": ([4, 2, 64], 5, [0, g.GEMM_F16]),
    "gemm_expert_route": ([4, 2, 8], 3, [0, g.GEMM_F32]),
    "gemm_expert_route_grad": ([4, 2, 8], 4, [0, g.GEMM_F32]),
    "gemm_expert_layer": ([4, 2, 8, 64, 64], 10, [0, g.GEMM_F16]),
}


@pytest.mark.parametrize("name", CALLS)
def test_refused_without_a_handle(name):
    f = getattr(pts.load(), name)
    args = [None] + CALLS[name][0]
    args += [0 if t is not ctypes.c_void_p else None for t in f.argtypes[len(args):]]
    assert f(*args) == g.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("name", CALLS)
def test_tensors_are_checked_before_the_call(name):
    sizes, arrays, rest = CALLS[name]
    x = torch.zeros(1 << 16, dtype=torch.float16)
    with pytest.raises(pts.GemmError) as err:
        getattr(pts, name)(None, *sizes, *[x] * arrays, *rest)
    assert err.value.status == g.GEMM_ERR_INVALID_ARG and "contiguous CUDA tensor" in str(err.value)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [None, 0, 1 << 40])
def test_raw_addresses_reach_the_call(name, stream):
    sizes, arrays, rest = CALLS[name]
    with pytest.raises(pts.GemmError) as err:
        getattr(pts, name)(None, *sizes, *[1 << 20] * arrays, *rest, stream=stream)
    assert err.value.status == g.GEMM_ERR_INVALID_ARG and name in str(err.value)


@pytest.mark.parametrize("name", CALLS)
def test_arguments_of_other_types_are_errors(name):
    sizes, arrays, rest = CALLS[name]
    f = getattr(pts, name)
    for args in ([*sizes, *["x"] * arrays, *rest], [*sizes, *[[1]] * arrays, *rest], [4.5, *sizes[1:], *[None] * arrays, *rest],
                 [1 << 70, *sizes[1:], *[None] * arrays, *rest], [*sizes, *[None] * arrays, "x", rest[1]]):
        with pytest.raises((TypeError, OverflowError)):
            f(None, *args)
    with pytest.raises(pts.GemmError, match="unknown dtype 9"):
        f(None, *sizes, *[None] * arrays, 0, 9)
    with pytest.raises(pts.GemmError):   # an activation or mode that 32 bits do not hold
        f(None, *sizes, *[None] * arrays, 1 << 40, rest[1])
    if name in ("gemm_expert_route", "gemm_expert_route_grad"):
        return
    with pytest.raises(pts.GemmError, match="unknown dtype 3"):   # fp32 is for logits
        f(None, *sizes, *[None] * arrays, 0, g.GEMM_F32)


class _Elsewhere:
    """A tensor as the extension module sees one, of so many elements."""
    def __init__(self, dtype, count):
        self.kind, self.count = dtype, count

    dtype = property(lambda self: self.kind)
    get_device = lambda self: 1  # noqa: E731
    is_contiguous = lambda self: True  # noqa: E731
    numel = lambda self: self.count  # noqa: E731
    data_ptr = lambda self: 1 << 20  # noqa: E731


def test_the_sizes_that_tensors_need():
    """Each array with one element too few is refused, and none with just enough (the C call then refuses the missing handle)."""
    from persistent_tile_scheduled_gb300 import experts
    module = experts._c.module
    h16, f32, i32, e4m3, bf16 = torch.float16, torch.float32, torch.int32, torch.float8_e4m3fn, torch.bfloat16
    gated = g.GEMM_ACT_GATED
    rows, E, N, K, T, k, D, H = 6, 3, 16, 32, 5, 2, 24, 40
    cases = [
        ("run_linear", [0, gated, None, rows, E, N, K], [(h16, rows * K), (h16, E * 2 * N * K), (h16, E * 2 * N), (h16, rows * N), (i32, E + 1),
                                                         (h16, rows * N), (h16, rows * 2 * N)], [1.0, 1.0, None]),
        ("run_linear", [2, 1, None, rows, E, N, K], [(e4m3, rows * K), (e4m3, E * N * K), (bf16, E * N), (bf16, rows * N), (i32, E + 1),
                                                     (bf16, rows * N), (bf16, rows * N)], [1.0, 1.0, None]),
        ("linear_grad", [0, gated | 5, None, rows, E, N], [(h16, rows * N), (h16, rows * 2 * N), (i32, E + 1), (h16, rows * 2 * N), (f32, E * 2 * N)], [None]),
        ("expert_route", [3, None, T, k, E], [(f32, T * E), (i32, T * k), (f32, T * k)], [0, None]),
        ("expert_route_grad", [1, None, T, k, E], [(bf16, T * E), (i32, T * k), (f32, T * k), (bf16, T * E)], [0, None]),
        ("expert_layer", [0, gated, None, T, k, E, D, H], [(h16, T * D), (i32, T * k), (f32, T * k), (h16, E * 2 * H * D), (h16, E * 2 * H), (h16, E * D * H),
                                                           (h16, E * D), (h16, T * D), (h16, T * k * H), (h16, T * D)], [None]),
    ]

    def refuse(what, x, dtype, count, device=None):
        raise KeyError(what)

    module.setup(_Elsewhere, refuse, torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.float32, torch.uint8)
    try:
        for name, before, arrays, after in cases:
            f = getattr(module, name)
            assert f(*before, *[_Elsewhere(d, n) for d, n in arrays], *after) == g.GEMM_ERR_INVALID_ARG
            for i in range(len(arrays)):
                for wrong in ((arrays[i][0], arrays[i][1] - 1), (torch.float64, arrays[i][1])):
                    with pytest.raises(KeyError):
                        f(*before, *[_Elsewhere(*(wrong if j == i else a)) for j, a in enumerate(arrays)], *after)
    finally:
        experts._setup(module)


@pytest.mark.parametrize("code", range(6), ids=ref.ACTS)
def test_the_plain_slopes_are_the_differences(code):
    """Central differences of step 2^-13 in 64 bits: off by 2^-26 / 6 of a third derivative below 6, and 2^-52 |f| 2^13."""
    z = torch.linspace(-9, 9, 777, dtype=torch.float64) + 0.0031
    a, s, _ = ref.act(code, z)
    t = 2.0 ** -13
    d = (ref.act(code, z + t)[0] - ref.act(code, z - t)[0]) / (2 * t)
    assert ((s - d).abs() <= 2.0 ** -26 + 2.0 ** -38 * (1 + a.abs())).all()
    assert ref.ACTS[code] in ("none", "relu2") or (s.abs() <= 1.13).all()
