"""Argument checks of layer norm, gated scan and sampling, which run on the host
before anything is enqueued (no GPU needed), and the tests' 64-bit gradient
formulas against differences of their forward formulas."""
import ctypes

import numpy as np
import pytest

from . import more_reference as M

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x100000  # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from scan_canonical_reduce_gb300 import model
    return model


def at(k):
    return FAKE * (k + 1)


def fill(cls, values, given):
    values.update({k: v for k, v in given.items() if k in values})
    return cls(*(values[n] for n, _ in cls._fields_))


def norm_args(m, **k):
    return fill(m._NormArgs, dict(batch=2, len=5, dim=16, dt=3, eps=1e-5, x=at(0),
                                  x_batch_stride=80, x_time_stride=16, weight=at(1), bias=at(2)), k)


def norm(m, **k):
    y = dict(y=at(3), ybs=80, yts=16, stats=at(4))
    y.update({n: v for n, v in k.items() if n in y})
    return m.lib().cr_layer_norm(ctypes.byref(norm_args(m, **k)), *y.values(), None)


BAD_NORM = [dict(batch=-1), dict(len=-1), dict(dim=-1), dict(dt=2), dict(dt=0), dict(eps=-1.0),
            dict(eps=float("nan")), dict(x=None), dict(x_batch_stride=-1), dict(x_time_stride=-1),
            dict(x=at(0) + 1), dict(weight=at(1) + 2), dict(bias=at(2) + 1)]


@pytest.mark.parametrize("bad", BAD_NORM + [
    dict(y=None), dict(y=at(0)), dict(ybs=15), dict(yts=15), dict(ybs=-1), dict(y=at(3) + 1),
    dict(stats=at(4) + 2), dict(stats=at(0))])
def test_norm_refuses(m, bad):
    assert norm(m, **bad) == INVALID
    assert m.lib().cr_layer_norm(None, at(3), 80, 16, None, None) == INVALID


def test_norm_unsupported_and_empty(m):
    assert norm(m, batch=1 << 40, len=1 << 10) == UNSUPPORTED
    for k in ("batch", "len", "dim"):
        assert norm(m, **{k: 0}) == OK


def norm_back(m, ws=at(20), size=1 << 24, **k):
    g = fill(m._NormGrads, dict(dy=at(5), dy_batch_stride=80, dy_time_stride=16, stats=at(6),
                                dx=at(7), dx_batch_stride=80, dx_time_stride=16, dweight=at(8),
                                dbias=at(9)), k)
    return m.lib().cr_layer_norm_backward(ctypes.byref(norm_args(m, **k)), ctypes.byref(g), ws,
                                          size, None)


@pytest.mark.parametrize("bad", BAD_NORM + [
    dict(dy=None), dict(dx=None), dict(dy_time_stride=-1), dict(dx_batch_stride=15),
    dict(dx_time_stride=15), dict(dx=at(5)), dict(dx=at(0)), dict(dweight=at(1)),
    dict(dbias=at(2)), dict(dy=at(5) + 1), dict(dx=at(7) + 1), dict(stats=at(6) + 2),
    dict(dweight=at(8) + 1), dict(dbias=at(9) + 2)])
def test_norm_backward_refuses(m, bad):
    assert norm_back(m, **bad) == INVALID
    assert m.lib().cr_layer_norm_backward(ctypes.byref(norm_args(m)), None, at(20), 1 << 24,
                                          None) == INVALID


def test_norm_backward_workspace(m):
    L = m.lib()
    for dim in (1, 16, 2048, 5000, 40000):
        need = L.cr_layer_norm_backward_workspace_bytes(2, 5, dim)
        assert need >= 256 and need % 256 == 0
        k = dict(dim=dim, x_batch_stride=5 * dim, x_time_stride=dim, dx_batch_stride=5 * dim,
                 dx_time_stride=dim)
        for ws, size in ((None, need), (at(20) + 4, need), (at(20), need - 1)):
            assert norm_back(m, ws, size, **k) == WORKSPACE
    assert L.cr_layer_norm_backward_workspace_bytes(-1, 5, 16) == 0
    assert L.cr_layer_norm_backward_workspace_bytes(1 << 40, 1 << 20, 16) == 0
    assert norm_back(m, dim=0) == OK


def gate_args(m, **k):
    a = dict(batch=2, len=5, dim=16, dt=3, index_bytes=8, state=at(3), lengths=at(4))
    for i, n in enumerate(("x", "gate", "z")):
        a.update({n: at(i), n + "_batch_stride": 80, n + "_time_stride": 16})
    return fill(m._GateArgs, a, k)


def gate(m, **k):
    y = dict(y=at(5), ybs=80, yts=16, final=at(6), kept=at(7))
    y.update({n: v for n, v in k.items() if n in y})
    return m.lib().cr_gated_scan(ctypes.byref(gate_args(m, **k)), *y.values(), None)


BAD_GATE = [dict(batch=-1), dict(len=-1), dict(dim=-1), dict(dt=2), dict(x=None), dict(gate=None),
            dict(x=at(0) + 1), dict(gate=at(1) + 1), dict(z=at(2) + 1)] + [
    {n + s: -1} for n in ("x", "gate", "z") for s in ("_batch_stride", "_time_stride")]


@pytest.mark.parametrize("bad", BAD_GATE + [
    dict(index_bytes=2), dict(lengths=at(4) + 4), dict(state=at(3) + 2), dict(y=None),
    dict(y=at(0)), dict(y=at(1)), dict(y=at(2)), dict(y=at(3)), dict(kept=at(3)), dict(ybs=15),
    dict(yts=15), dict(ybs=-1), dict(y=at(5) + 1), dict(final=at(6) + 1), dict(kept=at(7) + 2),
    dict(final=at(4))])
def test_gated_scan_refuses(m, bad):
    assert gate(m, **bad) == INVALID
    assert m.lib().cr_gated_scan(None, at(5), 80, 16, None, None, None) == INVALID


def test_gated_scan_unsupported_and_empty(m):
    assert gate(m, batch=1 << 40) == UNSUPPORTED
    assert gate(m, batch=0) == OK and gate(m, dim=0) == OK and gate(m, len=0, final=None) == OK
    L = m.lib()
    assert L.cr_gated_scan_checkpoints(0) == 0 and L.cr_gated_scan_checkpoints(1) == 1


def gate_back(m, **k):
    g = fill(m._GateGrads, dict(dy=at(8), dy_batch_stride=80, dy_time_stride=16, dfinal=at(9),
                                checkpoints=at(10), dx=at(11), dgate=at(12), dz=at(13),
                                dstate=at(14)), k)
    return m.lib().cr_gated_scan_backward(ctypes.byref(gate_args(m, **k)), ctypes.byref(g), None)


@pytest.mark.parametrize("bad", BAD_GATE + [
    dict(dy=None), dict(checkpoints=None), dict(dx=None), dict(dgate=None), dict(dz=None),
    dict(dy_time_stride=-1), dict(dx=at(0)), dict(dgate=at(8)), dict(dz=at(2)),
    dict(dstate=at(9)), dict(dx=at(10)), dict(dy=at(8) + 1), dict(dx=at(11) + 1),
    dict(dstate=at(14) + 2), dict(dfinal=at(9) + 1), dict(checkpoints=at(10) + 1)])
def test_gated_scan_backward_refuses(m, bad):
    assert gate_back(m, **bad) == INVALID


def gate_step(m, **k):
    y = dict(pool=at(3), rows=2, slots=None, y=at(5), ybs=16)
    y.update({n: v for n, v in k.items() if n in y})
    return m.lib().cr_gated_scan_step(ctypes.byref(gate_args(m, **{"len": 1, **k})), *y.values(),
                                      None)


@pytest.mark.parametrize("bad", [b for b in BAD_GATE if "len" not in b] + [
    dict(len=2), dict(len=0), dict(rows=-1), dict(rows=1), dict(slots=at(4), index_bytes=2),
    dict(slots=at(4) + 4), dict(y=None), dict(pool=None), dict(y=at(0)), dict(y=at(3)),
    dict(pool=at(1)), dict(ybs=8), dict(y=at(5) + 1), dict(pool=at(3) + 2)])
def test_gated_scan_step_refuses(m, bad):
    assert gate_step(m, **bad) == INVALID


def sample(m, tokens=at(9), **k):
    a = fill(m._SampleArgs, dict(rows=3, vocab=100, dt=1, index_bytes=4, logits=at(0),
                                 row_stride=100, u=at(1), temperature=1.0, top_p=1.0, min_p=0.0,
                                 top_k=0, temperatures=at(2), top_ps=at(3), min_ps=at(4),
                                 top_ks=at(5)), k)
    return m.lib().cr_sample(ctypes.byref(a), tokens, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(vocab=-1), dict(row_stride=-1), dict(dt=2), dict(dt=7),
    dict(index_bytes=3), dict(logits=None), dict(u=None), dict(tokens=None),
    dict(logits=at(0) + 2), dict(u=at(1) + 2), dict(tokens=at(9) + 4), dict(temperatures=at(2) + 1),
    dict(top_ps=at(3) + 2), dict(min_ps=at(4) + 3), dict(top_ks=at(5) + 2), dict(tokens=at(0)),
    dict(tokens=at(1)), dict(tokens=at(2)), dict(tokens=at(5))])
def test_sample_refuses(m, bad):
    assert sample(m, **bad) == INVALID
    assert m.lib().cr_sample(None, at(9), None) == INVALID


def test_sample_unsupported_and_empty(m):
    assert sample(m, vocab=(1 << 20) + 1) == UNSUPPORTED
    assert sample(m, rows=1 << 40) == UNSUPPORTED
    assert sample(m, rows=0) == OK


def test_binding_refuses_host_tensors(m):
    import torch
    x = torch.zeros(2, 3, 4)
    w = torch.ones(4)
    for call in (lambda: m.layer_norm(x, w), lambda: m.layer_norm_backward(x, x, w),
                 lambda: m.gated_scan(x, x), lambda: m.gated_scan_step(x[0], x[0], x[0]),
                 lambda: m.sample(x[0], w[:3])):
        with pytest.raises(ValueError):
            call()


def numeric(loss, args, name, rng):
    v = rng.standard_normal(args[name].shape)
    e = 1e-5
    up, down = ({**args, name: args[name] + s * e * v} for s in (1, -1))
    return (loss(up) - loss(down)) / (2 * e), v


def test_reference_gradients():
    """Central differences with e = 1e-5: e^2 of the third derivative plus
    2^-53 / e of the values, both below 1e-8 of sums of a few hundred terms."""
    rng = np.random.default_rng(0)
    f = rng.standard_normal
    a = dict(x=f((7, 9)), w=f(9), b=f(9), eps=1e-5)
    dy = f((7, 9))
    g = M.norm(**a, dy=dy)

    def norm_loss(q):
        return (M.norm(**q)["y"][0] * dy).sum()
    for k in ("x", "w", "b"):
        want, v = numeric(norm_loss, a, k, rng)
        got = g[{"x": "x", "w": "weight", "b": "bias"}[k]] if k != "x" else M.norm(**a, dy=dy)["x"]
        assert abs((got[0] * v).sum() - want) < 1e-6, k
    a = dict(x=f((2, 6, 3)), gate=f((2, 6, 3)), z=f((2, 6, 3)), state=f((2, 3)), lengths=[6, 3])
    dyg, df = f((2, 6, 3)), f((2, 3))
    g = M.gated(**a, dy=dyg, dfinal=df)

    def gate_loss(q):
        r = M.gated(**q)
        return (r["y"][0] * dyg).sum() + (r["final"][0] * df).sum()
    for k in ("x", "gate", "z", "state"):
        want, v = numeric(gate_loss, a, k, rng)
        assert abs((g["d" + k][0] * v).sum() - want) < 1e-6, k


def test_reference_sampling():
    """By hand: weights 1, 1/2, 1/4, 1/4 in the order of falling logits."""
    x = np.log(np.array([[0.25, 1.0, 0.25, 0.5]]))
    each = lambda **k: M.sample(x, np.array([k.get("u", 0.0)]), *(  # noqa: E731
        np.array([k.get(n, d)]) for n, d in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0),
                                             ("min_p", 0.0))))[0]
    assert [each(u=u) for u in (0.0, 0.49, 0.51, 0.76, 0.9)] == [1, 1, 3, 0, 2]
    assert [each(u=u, top_k=2) for u in (0.6, 0.7)] == [1, 3]
    assert each(u=0.999, top_p=0.5) == 1 and each(u=0.999, top_p=0.51) == 3
    assert each(u=0.999, min_p=0.4) == 3 and each(u=0.999, temperature=0.0) == 1
