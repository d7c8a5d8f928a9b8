"""The routing's gradient where dweights are infinite or NaN: what depends on them shows it, in every token."""
import pytest
import torch

import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
TYPES = {"f32": (pts.GEMM_F32, torch.float32), "f16": (pts.GEMM_F16, torch.float16), "bf16": (pts.GEMM_BF16, torch.bfloat16)}
MODES = {"selected": pts.GEMM_ROUTE_SELECTED, "all": pts.GEMM_ROUTE_ALL, "sigmoid": pts.GEMM_ROUTE_SIGMOID}


@pytest.fixture(scope="module")
def h():
    h = pts.gemm_create(0)
    yield h
    pts.gemm_destroy(h)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("experts", [7, 40, 128, 250, 1000])
@pytest.mark.parametrize("place", [0, 1, 2])
def test_every_chosen_logit_of_such_a_token(h, experts, mode, kind, place):
    """dl_i = w_i (dw_i - sum_j w_j dw_j): one infinite or NaN dweight makes the sum so, and with it the gradient of each chosen logit
    (of softmax over all, of each that is not masked; those that are round to w = 0 would be 0 times infinity, NaN)."""
    code, dtype = TYPES[kind]
    x = torch.randn(5, experts, generator=torch.Generator().manual_seed(5)).to(dtype)
    x[:, 3] = -INF
    ids = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :3]
    masked = torch.zeros(5, experts, dtype=torch.bool)
    masked[:, 3] = True
    depends = ~masked if mode == "all" else torch.zeros_like(masked).scatter_(1, ids, True)
    for bad in (INF, -INF, NAN):
        dw = torch.randn(5, 3, generator=torch.Generator().manual_seed(6))
        dw[1, place], dw[2, place], dw[4, place] = bad, bad, bad
        dl = torch.full((5, experts), 9.0, dtype=dtype, device="cuda")
        pts.gemm_expert_route_grad(h, 5, 3, experts, x.cuda(), ids.int().cuda(), dw.cuda(), dl, MODES[mode], code)
        dl = dl.cpu()
        hit = torch.tensor([False, True, True, False, True])
        assert torch.equal(~torch.isfinite(dl), depends & hit[:, None])
        assert (dl[~depends] == 0).all()
