"""Sampling where a setting lies close to a border, next to the ends of the bins
in which the kernel finds it: the token is that of the definition in 64 bits
(tests/more_reference.py)."""
import numpy as np
import pytest
import torch

from . import more_reference as M
from .model_reference import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LAST = 1 - 2.0 ** -24  # the largest u


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def each(v, rows):
    return f64(v) if isinstance(v, torch.Tensor) else np.full(rows, v, dtype=np.float64)


def check(scr, x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    s = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    got = scr.sample(x.to(DEV), u.to(DEV), **{k: v.to(DEV) if isinstance(v, torch.Tensor) else v
                                              for k, v in s.items()})
    want = M.sample(f64(x), f64(u), *(each(v, len(x)) for v in s.values()))
    bad = np.flatnonzero(got.cpu().numpy() != want)
    assert not len(bad), (len(bad), bad[:5], got[bad[:5]].tolist(), want[bad[:5]])
    return got


# ------------------------------------------------------------------ min_p
def test_min_p_beside_the_end_of_a_bin(scr):
    """Two tokens, the second of weight 2^-21 (1 + 4.4e-7), min_p 2^-21 (1 + 1.2e-7)."""
    x = torch.tensor([[14.55609, 0.0]])
    for min_p in (4.768372e-07, torch.tensor([4.768372e-07])):
        assert check(scr, x, torch.tensor([LAST]), min_p=min_p).tolist() == [1]


def min_p_rows(seed, above):
    """Logits [top, l] with l next to a bin's end, weights 2^(-b / 16) (1 +- 2^-18),
    b up to 22 octaves (u can still tell that the second is kept), and a min_p a
    rounding or a few above or below the weight, 2^-30 of it away at least."""
    rng = np.random.default_rng(seed)
    b = np.repeat(np.arange(1, 353), 24)
    top = (rng.standard_normal(len(b)) * 10).astype(np.float32)
    low = (top.astype(np.float64) - b / 16 * np.log(2)).astype(np.float32)
    for _ in range(2):
        low = np.where(rng.random(len(b)) < 0.5, np.nextafter(low, np.float32(above)), low)
    w = np.exp(low.astype(np.float64) - top)
    min_p = w.astype(np.float32)
    for _ in range(2):
        step = rng.integers(-1, 2, len(b)).astype(np.float32)
        min_p = np.where(step == 0, min_p, np.nextafter(min_p, step))
    clear = (np.abs(min_p.astype(np.float64) / w - 1) > 2.0 ** -30) & (min_p > 0) & (w < 1)
    return (torch.from_numpy(np.stack([top, low], 1)[clear]),
            torch.from_numpy(min_p[clear].astype(np.float32)))


@pytest.mark.parametrize("above", [-1e30, 1e30])
@pytest.mark.parametrize("top_k", [0, 2, 1000])
def test_min_p_beside_many_bins_ends(scr, above, top_k):
    x, min_p = min_p_rows(int(above > 0), above)
    u = torch.full((len(x),), LAST)
    got = check(scr, x, u, min_p=min_p, top_k=top_k)
    assert 0.2 < got.double().mean() < 0.8  # kept or not, both often


def test_min_p_beside_the_end_of_a_bin_of_many(scr):
    """More tokens in the bin than are sorted."""
    x, min_p = min_p_rows(5, 1e30)
    x, min_p = x[::29], min_p[::29]
    x = torch.cat([x[:, 1:].expand(-1, 1500), x[:, :1], x[:, 1:].expand(-1, 700)], 1).contiguous()
    u = torch.rand(len(x), generator=torch.Generator().manual_seed(6))
    check(scr, x, u, min_p=min_p)
    check(scr, x, u, min_p=min_p, top_p=0.999)


def test_min_p_far_below_the_largest(scr):
    """Many light tokens that only their sum makes weigh: min_p decides their number."""
    V, n = 1 << 16, 40
    g = torch.Generator().manual_seed(7)
    x = -(torch.rand(n, V, generator=g) * 4 + 11)  # weights 2^-16 to 2^-22
    x[:, 100] = 0.0
    u = 1 - torch.rand(n, generator=g) * 2.0 ** -2
    check(scr, x, u, min_p=torch.exp(-(torch.rand(n, generator=g) * 4 + 11)))
    check(scr, x[:2], u[:2], min_p=1e-12)


# ------------------------------------------------------- the farthest bins
@pytest.mark.parametrize("rows,V", [(40, 1100), (40, 20000), (4, 70000)])
@pytest.mark.parametrize("settings", [dict(), dict(top_p=0.8), dict(min_p=0.2)])
def test_top_k_that_ends_among_the_lightest(scr, rows, V, settings):
    """The last of top_k are tokens of weight 2^-63.88, behind which many of 2^-63.92
    lie: the largest and the smallest that are still told apart from none."""
    g = torch.Generator().manual_seed(V)
    x = torch.full((rows, V), -float("inf"))
    for r in range(rows):
        y = torch.cat([torch.rand(600, generator=g) * 2, 63.88 + 0.015 * torch.rand(10, generator=g),
                       63.905 + 0.025 * torch.rand(400, generator=g)])
        y[0] = 0
        x[r, torch.randperm(V, generator=g)[:len(y)]] = -y * float(np.log(2.0))
    u = torch.rand(rows, generator=g)
    for k in (601, 605, 609):
        check(scr, x, u, top_k=k, **settings)


# ------------------------------------------------------ bins that are cut
@pytest.mark.parametrize("rows,V", [(60, 2400), (60, 30000), (3, 80000)])
def test_cut_that_ends_beside_other_logits(scr, rows, V):
    """2147 tokens of one bin, which is cut by the logits' bits: into parts of 8192
    neighbouring numbers, then one of these, whose first 100 numbers are missing, into
    parts of 8. The last of these reaches past it, to numbers that stand there."""
    top = np.float32(100.0).view(np.uint32)
    g = np.random.default_rng(V)
    x = np.full((rows, V), -np.inf, dtype=np.float32)
    begin = 40 * 8192  # of the part, in binary32 numbers below the largest
    for r in range(rows):
        below = np.concatenate([
            [0, 2 ** 22 + 7], g.integers(begin + 101, begin + 8188, 1224), [begin + 100],
            np.repeat(begin + 8188 + np.arange(4), 30), np.repeat(begin + 8192 + np.arange(4), 200)])
        x[r, g.permutation(V)[:len(below)]] = (top - below.astype(np.uint32)).view(np.float32)
    x = torch.from_numpy(x)
    # all weights are within 4 % of one another; about the 1285th of 2147 is drawn
    assert float(x[x > -np.inf].min()) > 64
    u = torch.from_numpy(((1230 + 115 * g.random(rows)) / 2147).astype(np.float32))
    check(scr, x, u, temperature=1000.0)
    check(scr, x, torch.full((rows,), LAST), temperature=1000.0, top_k=1290)
    check(scr, x, torch.full((rows,), LAST), temperature=1000.0, top_p=0.6)


# ----------------------------------------------------- the largest roundings
@pytest.mark.parametrize("rows", [1, 3])
def test_weight_furthest_above_its_bins_own(scr, rows):
    """A logit whose distance, in the two binary32 numbers that hold it, has nearly the
    largest second number that it may have: its weight is 2^(-533 / 16) (1 + 1.04
    2^-18). Alone it weighs nothing; a million of them are 2^-13.3."""
    V, top, low, T = 1 << 20, 2.999998092651367, -30.16681671142578, 1.4363859649122808
    x = torch.full((rows, V), low, device=DEV)
    x[:, 77] = top
    w = float(np.exp((np.float64(np.float32(low)) - np.float64(np.float32(top))) / T))
    u = 1 - torch.arange(1, rows + 1) * 2.0 ** -15
    got = scr.sample(x, u.to(DEV), temperature=T).tolist()
    for a, v in zip(got, u.double().tolist()):
        at = (v * (1 + (V - 1) * w) - 1) / w  # so many of them come before
        assert at > 1000
        # sums are right to 2^-42 (2^-42 / w < 1) and a weight to 2^-32
        assert abs(a - at) <= 3
