"""Sampling: the token is that of the definition in 64 bits
(tests/more_reference.py)."""
import numpy as np
import pytest
import torch

from . import more_reference as M
from .model_reference import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def logits(rows, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(rows, V, generator=g)).to(dtype), torch.rand(rows, generator=g)


def want(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    rows = x.shape[0]

    def each(v):
        return f64(v) if isinstance(v, torch.Tensor) else np.full(rows, v, dtype=np.float64)
    return M.sample(f64(x), f64(u), each(temperature), each(top_k), each(top_p), each(min_p))


def check(scr, x, u, **settings):
    on = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in settings.items()}
    got = scr.sample(x.to(DEV), u.to(DEV), **on)
    assert got.dtype == torch.int64 and got.shape == u.shape
    assert got.cpu().tolist() == want(x, u, **settings).tolist()
    return got


SETTINGS = [dict(), dict(temperature=0.0), dict(temperature=0.7, top_k=5), dict(top_k=1),
            dict(top_p=0.9), dict(top_p=0.0), dict(top_p=1e-7), dict(min_p=0.1), dict(min_p=1.0),
            dict(temperature=1.7, top_k=40, top_p=0.8, min_p=0.02), dict(temperature=30.0),
            dict(temperature=1e-3), dict(top_k=10 ** 6), dict(temperature=0.9, top_p=0.999999)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 33, 1000, 10007])
@pytest.mark.parametrize("settings", SETTINGS)
def test_settings(scr, dtype, V, settings):
    check(scr, *logits(9, V, dtype, V), **settings)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,V", [(1, 65536), (3, 100003), (2, 262144), (300, 2000)])
def test_sizes(scr, dtype, rows, V):
    x, u = logits(rows, V, dtype, 2)
    check(scr, x, u)
    check(scr, x, u, temperature=0.8, top_k=50, top_p=0.95)
    check(scr, x, u, top_k=min(V, 30000), top_p=0.99, min_p=1e-4)


def test_settings_of_their_own(scr):
    g = torch.Generator().manual_seed(3)
    x, u = logits(64, 5000, torch.float32, 3)
    r = lambda: torch.rand(64, generator=g)  # noqa: E731
    s = dict(temperature=torch.where(r() < 0.3, torch.zeros(64), 0.3 + r()),
             top_k=(300 * r()).int() - 50, top_p=1.2 * r(), min_p=0.3 * r())
    check(scr, x, u, **s)
    check(scr, x, u, **{**s, "top_k": s["top_k"].long()})
    s["top_p"][::3] = NAN
    s["min_p"][::4] = NAN
    s["temperature"][::5] = NAN
    s["temperature"][1::5] = INF
    check(scr, x, u, **s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [50, 3000, 40000])
def test_masked(scr, dtype, V):
    x, u = logits(8, V, dtype, 4)
    g = torch.Generator().manual_seed(5)
    x[torch.rand(8, V, generator=g) < 0.7] = -INF
    x[:, ::5] = torch.finfo(dtype).min
    x[:, ::11] = NAN
    x[1] = -INF
    x[2] = NAN
    x[3] = torch.finfo(dtype).min  # all alike: all of them candidates
    x[4] = -INF
    x[4, V // 2] = -5.0  # the only one
    x[5, 7] = INF
    x[5, V - 1] = INF
    for s in (dict(), dict(top_k=20), dict(top_p=0.7), dict(min_p=0.05), dict(temperature=0.0),
              dict(temperature=2.0, top_k=100, top_p=0.9, min_p=0.01), dict(temperature=INF)):
        got = check(scr, x, u, **s)
        assert got[1] == -1 and got[2] == -1 and got[4] == V // 2 and int(got[5]) in (7, V - 1)


@pytest.mark.parametrize("V", [100, 3001, 70000])
def test_equal_logits(scr, V):
    """Many of one value: their order is that of the index."""
    g = torch.Generator().manual_seed(6)
    u = torch.rand(40, generator=g)
    u[0], u[1] = 0.0, 1 - 2.0 ** -24
    flat = torch.full((40, V), 1.25)
    for s in (dict(), dict(top_k=V // 2), dict(top_p=0.5), dict(temperature=0.3, top_k=7)):
        check(scr, flat, u, **s)
    few = torch.randint(0, 4, (40, V), generator=g).float()
    few[:, 3] = -0.0
    for s in (dict(), dict(top_k=V // 3), dict(top_p=0.77), dict(min_p=0.1),
              dict(temperature=0.5, top_k=V - 2, top_p=0.95)):
        check(scr, few, u, **s)
        check(scr, few.bfloat16(), u, **s)


def test_nearly_equal_logits(scr):
    """Values that differ by less than a weight shows, and ones around zero."""
    g = torch.Generator().manual_seed(7)
    u = torch.rand(30, generator=g)
    V = 9000
    for base, step in ((1.0, 2.0 ** -23), (0.0, 1e-30), (0.0, 2.0 ** -149), (-7.0, 2.0 ** -21)):
        x = base + step * torch.randint(-20, 20, (30, V), generator=g).float()
        for s in (dict(), dict(top_k=1000), dict(top_p=0.3), dict(top_k=4500, top_p=0.9)):
            check(scr, x, u, **s)


def test_u_at_its_ends(scr):
    x, _ = logits(6, 700, torch.float32, 8)
    u = torch.tensor([0.0, -1.0, NAN, 1.0, 7.0, 1 - 2.0 ** -24])
    for s in (dict(), dict(top_k=10), dict(top_p=0.6)):
        check(scr, x, u, **s)


def test_shares(scr):
    """Over evenly spaced u each token comes as often as its probability says."""
    x = torch.tensor([1.0, 3.0, -2.0, 0.5, 3.0, 0.0])
    n = 4096
    u = (torch.arange(n) + 0.5) / n
    got = scr.sample(x.to(DEV).expand(n, 6), u.to(DEV), temperature=1.5)
    p = torch.softmax(x.double() / 1.5, 0)
    share = torch.bincount(got.cpu(), minlength=6).double() / n
    # a token's interval of u holds its length times n of the points, give or take one
    assert (share - p).abs().max() <= 1.0 / n


def test_shapes_strides_and_alignment(scr):
    x, u = logits(6, 1001, torch.float16, 9)
    d, ud = x.to(DEV), u.to(DEV)
    s = dict(temperature=0.8, top_k=100, top_p=0.9)
    base = check(scr, x, u, **s)
    assert torch.equal(scr.sample(d.view(2, 3, 1001), ud.view(2, 3), **s), base.view(2, 3))
    assert scr.sample(d[2], ud[2], **s).shape == () and scr.sample(d[2], ud[2], **s) == base[2]
    pad = torch.full((6, 1100), NAN, dtype=x.dtype, device=DEV)
    for at in (0, 1, 3, 8):
        pad[:, at:at + 1001] = d
        assert torch.equal(scr.sample(pad[:, at:at + 1001], ud, **s), base)
    assert torch.equal(scr.sample(d.t().contiguous().t(), ud, **s), base)
    assert torch.equal(scr.sample(d[:1].expand(6, 1001), ud[:1].expand(6), **s), base[:1].expand(6))
    out = torch.zeros(6, dtype=torch.int64, device=DEV)
    assert scr.sample(d, ud, **s, out=out) is out and torch.equal(out, base)
    assert scr.sample(d[:0], ud[:0]).shape == (0,)
    assert scr.sample(d[:, :0], ud).tolist() == [-1] * 6


def test_refusals(scr):
    x, u = logits(4, 50, torch.float32, 10)
    d, ud = x.to(DEV), u.to(DEV)
    for bad, error in ((dict(logits=d.double()), TypeError), (dict(logits=x), ValueError),
                       (dict(u=ud.double()), TypeError), (dict(u=ud[:2]), ValueError),
                       (dict(u=u), ValueError), (dict(u=None), TypeError),
                       (dict(temperature=-1.0), ValueError), (dict(temperature=NAN), ValueError),
                       (dict(top_k=-1), ValueError), (dict(top_p=-0.1), ValueError),
                       (dict(min_p=1.5), ValueError), (dict(min_p=-0.5), ValueError),
                       (dict(temperature=ud[:1]), ValueError), (dict(top_k=ud), TypeError),
                       (dict(top_p=ud.half()), TypeError), (dict(temperature="hot"), TypeError),
                       (dict(out=torch.zeros(4, dtype=torch.int32, device=DEV)), TypeError),
                       (dict(out=torch.zeros(5, dtype=torch.int64, device=DEV)), ValueError)):
        with pytest.raises(error):
            scr.sample(**{"logits": d, "u": ud, **bad})
    with pytest.raises(scr.CrError):
        scr.sample(d[:1, :1].expand(1, (1 << 20) + 1), ud[:1])
