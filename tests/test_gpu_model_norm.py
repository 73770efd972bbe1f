"""Layer norm and its gradient against a plain 64-bit evaluation
(tests/more_reference.py derives the bounds)."""
import numpy as np
import pytest
import torch

from . import more_reference as M
from .model_reference import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def make(shape, dtype, seed, weight=True, bias=True, offset=1.0):
    g = torch.Generator().manual_seed(seed)
    D = shape[-1]
    x = torch.randn(shape, generator=g) + offset * torch.randn(*shape[:-1], 1, generator=g)
    return {"x": x.to(dtype), "weight": 1 + 0.3 * torch.randn(D, generator=g) if weight else None,
            "bias": 0.3 * torch.randn(D, generator=g) if bias else None}, \
        torch.randn(shape, generator=g).to(dtype)


def dev(s):
    return {k: v if v is None else v.to(DEV) for k, v in s.items()}


def reference(s, dy=None, eps=1e-5):
    return M.norm(f64(s["x"]), f64(s["weight"]), f64(s["bias"]), float(np.float32(eps)), f64(dy))


SHAPES = [(1, 1), (3, 2), (1, 7), (5, 8), (2, 33), (300, 64), (7, 333), (1, 1024), (3, 1000),
          (2, 5, 2048), (700, 128), (33, 2047), (4, 4096), (2, 3, 2, 520), (3, 8200), (2, 12345),
          (1, 32768), (2, 40000), (0, 16)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(scr, dtype, shape):
    s, dy = make(shape, dtype, 1)
    d = dev(s)
    y, stats = scr.layer_norm(**d, return_stats=True)
    assert y.dtype == dtype and stats.shape == (*shape[:-1], 3)
    ref = reference(s, dy)
    M.near(y, *ref["y"], "y")
    g = scr.layer_norm_backward(dy.to(DEV), **d, stats=stats)
    assert set(g) == {"x", "weight", "bias"}
    for k in g:
        M.near(g[k], *ref[k], "d" + k)
    again = scr.layer_norm_backward(dy.to(DEV), **d)  # statistics computed again
    for k in g:
        assert torch.equal(g[k], again[k]), k


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("shape", [(9, 333), (6, 2048)])
def test_without_weight_or_bias(scr, dtype, weight, bias, shape):
    s, dy = make(shape, dtype, 2, weight, bias)
    d = dev(s)
    ref = reference(s, dy)
    M.near(scr.layer_norm(**d), *ref["y"], "y")
    g = scr.layer_norm_backward(dy.to(DEV), **d)
    assert set(g) == {"x"} | ({"weight"} if weight else set()) | ({"bias"} if bias else set())
    for k in g:
        M.near(g[k], *ref[k], "d" + k)


@pytest.mark.parametrize("rows,D", [(20000, 96), (1201, 520), (5000, 1001)])
def test_many_rows(scr, rows, D):
    s, dy = make((rows, D), torch.bfloat16, 3)
    d = dev(s)
    ref = reference(s, dy)
    y, stats = scr.layer_norm(**d, return_stats=True)
    M.near(y, *ref["y"], "y")
    g = scr.layer_norm_backward(dy.to(DEV), **d, stats=stats)
    for k in g:
        M.near(g[k], *ref[k], "d" + k)


def test_large_mean_and_constant_rows(scr):
    """A mean far larger than the spread, rows of one value, and eps = 0."""
    g = torch.Generator().manual_seed(4)
    for mean, spread in ((1e4, 1.0), (-3e6, 2.0), (1e-3, 1e-12), (0.0, 1e-9), (0.0, 1e15)):
        s = {"x": mean + spread * torch.randn(7, 1500, generator=g), "weight": None, "bias": None}
        for eps in (1e-5, 0.0):
            dy = torch.randn(7, 1500, generator=g)
            if eps == 0.0 and not (s["x"] != s["x"][:, :1]).any():  # 0 / 0 by the formula
                assert scr.layer_norm(**dev(s), eps=eps).isnan().all()
                continue
            ref = reference(s, dy, eps)
            M.near(scr.layer_norm(**dev(s), eps=eps), *ref["y"], "y")
            got = scr.layer_norm_backward(dy.to(DEV), **dev(s), eps=eps)
            M.near(got["x"], *ref["x"], "dx")
    for v in (0.0, 0.1, -77777.7, 1e15):
        s = {"x": torch.full((3, 777), v), "weight": None, "bias": None}
        M.near(scr.layer_norm(**dev(s)), *reference(s)["y"], "constant")


def test_rows_stay_apart(scr):
    """NaN and infinity in one row reach that row alone (and the sums over rows)."""
    for D in (64, 2048, 5000, 40000):
        s, dy = make((9, D), torch.float32, 5)
        d = dev(s)
        want, gw = scr.layer_norm(**d), scr.layer_norm_backward(dy.to(DEV), **d)["x"]
        d["x"][4, D // 2] = float("nan")
        d["x"][7, 0] = float("inf")
        got, g = scr.layer_norm(**d), scr.layer_norm_backward(dy.to(DEV), **d)["x"]
        for r in range(9):
            if r in (4, 7):
                assert got[r].isnan().any() and g[r].isnan().any()
            else:
                assert torch.equal(got[r], want[r]) and torch.equal(g[r], gw[r])


def test_strides_and_alignment(scr):
    """The same bits from strided, misaligned, transposed and repeated inputs."""
    for D in (24, 2048):
        s, dy = make((3, 40, D), torch.bfloat16, 6)
        d, dyd = dev(s), dy.to(DEV)
        want, gw = scr.layer_norm(**d), scr.layer_norm_backward(dyd, **d)

        def placed(v, offset, pad):
            big = torch.full((3 * 41 * (D + pad) + offset,), float("nan"), dtype=v.dtype, device=DEV)
            t = big[offset:].as_strided((3, 40, D), (41 * (D + pad), D + pad, 1))
            return t.copy_(v)

        for offset, pad in ((0, 8), (1, 0), (3, 5), (8, 0), (2, 2)):
            x, g = placed(d["x"], offset, pad), placed(dyd, offset, pad)
            out = placed(torch.zeros_like(want), offset, pad)
            assert torch.equal(scr.layer_norm(x, d["weight"], d["bias"]), want)
            assert scr.layer_norm(x, d["weight"], d["bias"], out=out) is out
            assert torch.equal(out, want)
            got = scr.layer_norm_backward(g, x, d["weight"], d["bias"])
            assert all(torch.equal(got[k], gw[k]) for k in gw)
            w = torch.empty(D + 1, device=DEV)[1:].copy_(d["weight"])  # 4-byte aligned
            assert torch.equal(scr.layer_norm(x, w, d["bias"]), want)
        turned = d["x"].transpose(0, 1)
        assert torch.equal(scr.layer_norm(turned, d["weight"], d["bias"]), want.transpose(0, 1))
        last = d["x"].transpose(1, 2).contiguous().transpose(1, 2)
        assert torch.equal(scr.layer_norm(last, d["weight"], d["bias"]), want)
        one = d["x"][:, :1].expand(3, 40, D)
        assert torch.equal(scr.layer_norm(one, d["weight"], d["bias"]),
                           want[:, :1].expand(3, 40, D))
        wide = d["x"].reshape(3, 2, 20, D).transpose(1, 2)
        assert torch.equal(scr.layer_norm(wide, d["weight"], d["bias"]),
                           want.reshape(3, 2, 20, D).transpose(1, 2))


def test_rows_do_not_change_each_other(scr):
    """A row's bits are the same alone and among others."""
    for D in (100, 2048, 4096, 9000):
        s, dy = make((50, D), torch.bfloat16, 7)
        d, dyd = dev(s), dy.to(DEV)
        y, g = scr.layer_norm(**d), scr.layer_norm_backward(dyd, **d)["x"]
        for r in (0, 13, 49):
            one = {**d, "x": d["x"][r:r + 1]}
            assert torch.equal(scr.layer_norm(**one)[0], y[r])
            assert torch.equal(scr.layer_norm_backward(dyd[r:r + 1], **one)["x"][0], g[r])


def test_gradient_matches_differences(scr):
    """A direction's derivative against central differences of the 64-bit formula,
    whose error eps^2 / 6 of the third derivative leaves the gradient's own binary32
    rounding as the largest."""
    s, dy = make((6, 40), torch.float32, 8)
    got = scr.layer_norm_backward(dy.to(DEV), **dev(s))
    gen = torch.Generator().manual_seed(9)
    for name in got:
        v = torch.randn(s[name].shape, generator=gen, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            m = {k: f64(t) for k, t in s.items()}
            m[name] = m[name] + sign * 1e-4 * v.numpy()
            ends.append((M.norm(m["x"], m["weight"], m["bias"], 1e-5)["y"][0] * f64(dy)).sum())
        want = (ends[0] - ends[1]) / 2e-4
        have = (f64(got[name]) * v.numpy()).sum()
        size = (np.abs(f64(got[name])) * np.abs(v.numpy())).sum()
        assert abs(have - want) <= 1e-5 * size, name


def test_autograd(scr):
    s, dy = make((4, 30, 72), torch.float32, 10)
    d, dyd = dev(s), dy.to(DEV)
    want = scr.layer_norm_backward(dyd, **d)
    leaves = {k: v.clone().requires_grad_(True) for k, v in d.items()}
    y = scr.layer_norm(**leaves)
    assert torch.equal(y.detach(), scr.layer_norm(**d))
    y.backward(dyd)
    assert all(torch.equal(leaves[k].grad, want[k]) for k in want)
    y, stats = scr.layer_norm(**leaves, return_stats=True)
    assert not stats.requires_grad
    w = leaves["weight"].detach().requires_grad_(True)  # one argument alone
    (gw,) = torch.autograd.grad(scr.layer_norm(d["x"], w), w, dyd)
    assert torch.equal(gw, scr.layer_norm_backward(dyd, d["x"], d["weight"])["weight"])
    with pytest.raises(RuntimeError):
        scr.layer_norm(**leaves, out=torch.empty_like(d["x"]))
    y = scr.layer_norm(**leaves)
    (gx,) = torch.autograd.grad(y, leaves["x"], dyd, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()


def test_refusals(scr):
    x = torch.zeros(4, 16, device=DEV)
    w = torch.ones(16, device=DEV)
    for bad, error in ((dict(x=x.double()), TypeError), (dict(weight=w.bfloat16()), TypeError),
                       (dict(weight=w[:5]), ValueError), (dict(bias=w[None]), ValueError),
                       (dict(eps=-1e-5), ValueError), (dict(eps=float("nan")), ValueError),
                       (dict(weight=w.cpu()), ValueError), (dict(out=x[:2]), ValueError),
                       (dict(out=x.bfloat16()), TypeError), (dict(x=x.cpu()), ValueError),
                       (dict(out=x), scr.CrError), (dict(x=x[0, 0]), ValueError)):
        with pytest.raises(error):
            scr.layer_norm(**{"x": x, **bad})
    for bad, error in ((dict(dy=x[:2]), ValueError), (dict(dy=x.half()), TypeError),
                       (dict(stats=x), ValueError)):
        with pytest.raises(error):
            scr.layer_norm_backward(**{"dy": x + 1, "x": x, **bad})


def test_no_rows_and_no_channels(scr):
    w = torch.ones(16, device=DEV)
    x = torch.zeros(0, 16, device=DEV)
    assert scr.layer_norm(x, w).shape == x.shape
    g = scr.layer_norm_backward(x, x, w, w)
    assert not g["weight"].any() and not g["bias"].any() and g["weight"].shape == (16,)
    x = torch.zeros(5, 0, device=DEV)
    assert scr.layer_norm(x, w[:0]).shape == x.shape
    assert scr.layer_norm_backward(x, x, w[:0])["weight"].shape == (0,)
