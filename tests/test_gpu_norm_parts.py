"""Layer norm's gradient without those of weight and bias: nothing is computed for
them."""
import ctypes

import pytest
import torch

from . import more_reference as M
from .model_reference import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


@pytest.mark.parametrize("D", [96, 333, 2048, 2049, 8200, 9001])
def test_no_part_of_the_sums_over_rows(scr, D):
    from scan_canonical_reduce_gb300 import model as m
    L = scr.lib()
    g = torch.Generator().manual_seed(D)
    x, dy = (torch.randn(70, D, generator=g).bfloat16() for _ in range(2))
    dx, dw = torch.empty(70, D, dtype=torch.bfloat16, device=DEV), torch.empty(D, device=DEV)
    xd, dyd = x.to(DEV), dy.to(DEV)
    size = L.cr_layer_norm_backward_workspace_bytes(1, 70, D)
    na = m._NormArgs(1, 70, D, 3, 1e-5, xd.data_ptr(), 70 * D, D, None, None)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    sums = 256 + (70 * 12 + 255) // 256 * 256  # behind the statistics
    for grad in (None, dw.data_ptr()):
        ws.fill_(0x5A)
        ng = m._NormGrads(dyd.data_ptr(), 70 * D, D, None, dx.data_ptr(), 70 * D, D, grad, None)
        before = scr.launch_count()
        assert L.cr_layer_norm_backward(ctypes.byref(na), ctypes.byref(ng), ws.data_ptr(), size,
                                        torch.cuda.current_stream(DEV).cuda_stream) == 0
        launches = scr.launch_count() - before
        if grad is None:  # statistics and dx
            assert launches == 2 and bool((ws[sums:] == 0x5A).all())
        ref = M.norm(f64(x), None, None, float(torch.tensor(1e-5)), f64(dy))
        M.near(dx, *ref["x"], "dx")
    M.near(dw, *ref["weight"], "dweight")


@pytest.mark.parametrize("D", [8200, 9001])
@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_long_rows_without_weight_or_bias(scr, D, weight, bias):
    g = torch.Generator().manual_seed(D)
    x, dy = (torch.randn(40, D, generator=g).bfloat16() for _ in range(2))
    w = torch.randn(D, generator=g) if weight else None
    b = torch.randn(D, generator=g) if bias else None
    on = [None if t is None else t.to(DEV) for t in (w, b)]
    ref = M.norm(f64(x), f64(w), f64(b), float(torch.tensor(1e-5)), f64(dy))
    M.near(scr.layer_norm(x.to(DEV), *on), *ref["y"], "y")
    got = scr.layer_norm_backward(dy.to(DEV), x.to(DEV), *on)
    assert set(got) == {"x"} | ({"weight"} if weight else set()) | ({"bias"} if bias else set())
    for k in got:
        M.near(got[k], *ref[k], "d" + k)


@pytest.mark.parametrize("shape", [(3, 0), (2, 5, 0), (0, 0)])
def test_rows_without_channels(scr, shape):
    """The statistics of nothing are NaN, not what their memory held."""
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    held = torch.full((4096,), 7.0, device=DEV)
    del held
    y, stats = scr.layer_norm(x, return_stats=True)
    assert y.shape == shape and stats.shape == (*shape[:-1], 3) and bool(stats.isnan().all())
