"""The model operators' argument checks, which run on the host before anything
is enqueued (no GPU needed), and the tests' 64-bit gradient formulas against
differences of their forward formulas."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

from . import model_reference as R

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x100000  # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from scan_canonical_reduce_gb300 import model
    return model


WITHOUT_BINDING = """
import os
exists = os.path.exists
os.path.exists = lambda p: not str(p).endswith("cr_model_binding.so") and exists(p)
import scan_canonical_reduce_gb300 as cr
assert cr.lib().cr_version() > 0
assert cr.lib().cr_reduce_workspace_bytes(1000, 16, cr.CR_F64) > 0
import torch
for call in (lambda: cr.embedding(torch.zeros(3).long(), torch.zeros(4, 4)),
             lambda: cr.causal_conv(torch.zeros(2, 3, 4), torch.zeros(4, 4))):
    try:
        call()
    except ImportError as e:
        assert "cr_model_binding.so" in str(e)
    else:
        raise AssertionError("no ImportError")
print("fine")
"""


def test_reductions_and_scans_need_no_binding(m):
    """Without the model operators' native module everything else works, and
    they say what is missing."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", WITHOUT_BINDING], cwd=root, capture_output=True,
                       text=True)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr


def test_binding_is_built_anew_for_another_pytorch(m, tmp_path, monkeypatch):
    import importlib.util
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "_cr_build_for_test", os.path.join(root, "scan_canonical_reduce_gb300", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    assert os.path.exists(b.BINDING)
    jobs = []

    def run(command, **kw):
        jobs.append(command)
        raise RuntimeError("not compiled here")

    monkeypatch.setattr(b.subprocess, "run", run)
    b.build()  # up to date: nothing to do
    assert not jobs
    other = tmp_path / "torch"
    other.mkdir()
    (other / "version.py").write_text("__version__ = '99.0'")
    find = b.importlib.util.find_spec

    class Other:
        submodule_search_locations = [str(other)]

    monkeypatch.setattr(b.importlib.util, "find_spec",
                        lambda n: Other if n == "torch" else find(n))
    with pytest.raises(RuntimeError):
        b.build()
    assert len(jobs) == 1 and b.BINDING_SRC in jobs[0]


def at(k):
    return FAKE * (k + 1)


def embed(m, **k):
    a = dict(tokens=at(0), index=8, n=4, table=at(1), vocab=10, dim=16, row=16, dt=3, out=at(2),
             out_stride=16)
    a.update(k)
    return m.lib().cr_embedding(a["tokens"], a["index"], a["n"], a["table"], a["vocab"], a["dim"],
                                a["row"], 1.0, a["dt"], a["out"], a["out_stride"], None)


@pytest.mark.parametrize("bad", [
    dict(dt=2), dict(dt=0), dict(index=2), dict(n=-1), dict(vocab=-1), dict(dim=-1),
    dict(row=15), dict(out_stride=15), dict(tokens=None), dict(table=None), dict(out=None),
    dict(out=at(1)), dict(tokens=at(0) + 4), dict(table=at(1) + 1), dict(out=at(2) + 1)])
def test_embedding_refuses(m, bad):
    assert embed(m, **bad) == INVALID


def test_embedding_empty(m):
    assert embed(m, n=0) == OK and embed(m, dim=0) == OK


def embed_grad(m, **k):
    a = dict(tokens=at(0), index=8, n=4, grad=at(1), stride=16, vocab=10, dim=16, dt=3, dw=at(2),
             dw_stride=16, ws=at(3), bytes=1 << 20)
    a.update(k)
    return m.lib().cr_embedding_backward(a["tokens"], a["index"], a["n"], a["grad"], a["stride"],
                                         a["vocab"], a["dim"], 1.0, a["dt"], 0, a["dw"],
                                         a["dw_stride"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(dt=2), dict(index=1), dict(n=-1), dict(n=1 << 31), dict(vocab=-1), dict(vocab=1 << 31),
    dict(dim=-1), dict(stride=15), dict(dw_stride=15), dict(tokens=None), dict(grad=None),
    dict(dw=None), dict(dw=at(1)), dict(grad=at(1) + 1), dict(dw=at(2) + 2)])
def test_embedding_backward_refuses(m, bad):
    assert embed_grad(m, **bad) == INVALID


def test_embedding_backward_workspace(m):
    need = m.lib().cr_embedding_backward_workspace_bytes(4, 10, 16)
    assert need >= 256 and need % 256 == 0
    for bad in (dict(ws=None), dict(ws=at(3) + 8), dict(bytes=need - 1)):
        assert embed_grad(m, **bad) == WORKSPACE
    assert m.lib().cr_embedding_backward_workspace_bytes(-1, 10, 16) == 0
    assert m.lib().cr_embedding_backward_workspace_bytes(1 << 31, 10, 16) == 0
    assert embed_grad(m, vocab=0) == OK and embed_grad(m, dim=0) == OK


def conv_args(m, **k):
    a = dict(batch=2, len=5, dim=16, width=4, activation=1, dt=3, index_bytes=4, x=at(0),
             x_batch_stride=80, x_time_stride=16, weight=at(1), bias=at(2), state=at(3),
             lengths=at(4))
    a.update({n: v for n, v in k.items() if n in a})
    return m._ConvArgs(*(a[n] for n, _ in m._ConvArgs._fields_))


def conv(m, **k):
    y = dict(y=at(5), ybs=80, yts=16, final=at(6))
    y.update({n: v for n, v in k.items() if n in y})
    return m.lib().cr_causal_conv(ctypes.byref(conv_args(m, **k)), y["y"], y["ybs"], y["yts"],
                                  y["final"], None)


BAD_CONV = [dict(batch=-1), dict(len=-1), dict(dim=-1), dict(width=0), dict(activation=2),
            dict(activation=-1), dict(dt=2), dict(dt=9), dict(index_bytes=3), dict(x=None),
            dict(x_batch_stride=-1), dict(x_time_stride=-1), dict(weight=None), dict(x=at(0) + 1),
            dict(weight=at(1) + 2), dict(bias=at(2) + 1), dict(state=at(3) + 1),
            dict(lengths=at(4) + 2)]


@pytest.mark.parametrize("bad", BAD_CONV + [
    dict(y=None), dict(y=at(0)), dict(yts=15), dict(ybs=15), dict(yts=-1), dict(y=at(5) + 1),
    dict(final=at(6) + 1)])
def test_conv_refuses(m, bad):
    assert conv(m, **bad) == INVALID
    assert m.lib().cr_causal_conv(None, at(5), 80, 16, None, None) == INVALID


def test_conv_unsupported_and_empty(m):
    assert conv(m, width=1) == UNSUPPORTED and conv(m, width=5) == UNSUPPORTED
    assert conv(m, batch=1 << 40, len=1 << 20) == UNSUPPORTED
    assert conv(m, batch=0) == OK and conv(m, dim=0) == OK and conv(m, len=0, final=None) == OK


def conv_back(m, ws=at(9), size=1 << 24, **k):
    g = dict(dy=at(5), dy_batch_stride=80, dy_time_stride=16, dfinal=None, dx=at(6),
             dx_batch_stride=80, dx_time_stride=16, dweight=at(7), dbias=at(8), dstate=None)
    g.update({n: v for n, v in k.items() if n in g})
    c = m._ConvGrads(*(g[n] for n, _ in m._ConvGrads._fields_))
    return m.lib().cr_causal_conv_backward(ctypes.byref(conv_args(m, **k)), ctypes.byref(c), ws,
                                           size, None)


@pytest.mark.parametrize("bad", BAD_CONV + [
    dict(dy=None), dict(dy_time_stride=-1), dict(dweight=None), dict(dx=at(5)), dict(dx=at(0)),
    dict(dx_time_stride=8), dict(dx_batch_stride=8), dict(dweight=at(7) + 1), dict(dx=at(6) + 1)])
def test_conv_backward_refuses(m, bad):
    assert conv_back(m, **bad) == INVALID


def test_conv_backward_workspace(m):
    need = m.lib().cr_causal_conv_backward_workspace_bytes(2, 5, 16, 4)
    assert need >= 256 and need % 256 == 0
    assert m.lib().cr_causal_conv_backward_workspace_bytes(2, -5, 16, 4) == 0
    for ws, size in ((None, need), (at(9) + 4, need), (at(9), need - 1)):
        assert conv_back(m, ws, size) == WORKSPACE


def conv_step(m, **k):
    a = dict(x=at(0), xs=16, state=at(1), rows=4, slots=None, index=4, weight=at(2), bias=None,
             act=1, batch=3, dim=16, width=4, dt=3, y=at(3), ys=16)
    a.update(k)
    return m.lib().cr_causal_conv_step(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(dt=2), dict(batch=-1), dict(dim=-1), dict(rows=-1), dict(xs=-1), dict(width=0),
    dict(act=7), dict(rows=2), dict(slots=at(4), index=5), dict(slots=at(4) + 2), dict(x=None),
    dict(y=None), dict(weight=None), dict(state=None), dict(y=at(0)), dict(y=at(1)), dict(ys=8),
    dict(x=at(0) + 1), dict(state=at(1) + 1), dict(weight=at(2) + 2)])
def test_conv_step_refuses(m, bad):
    assert conv_step(m, **bad) == INVALID


def test_conv_step_unsupported_and_empty(m):
    assert conv_step(m, width=5) == UNSUPPORTED
    assert conv_step(m, batch=0) == OK and conv_step(m, dim=0) == OK


def scan_args(m, **k):
    a = dict(batch=2, len=5, dim=16, dstate=16, groups=2, softplus=1, dt_type=3, index_bytes=8,
             reserved=0, A=at(5), D=at(6), dt_bias=at(7), state=at(8), lengths=at(9))
    for i, n in enumerate(("u", "dt", "z", "B", "C")):
        w = 16 if i < 3 else 32
        a.update({n: at(i), n + "_batch_stride": 5 * w, n + "_time_stride": w})
    a.update({n: v for n, v in k.items() if n in a})
    return m._ScanArgs(*(a[n] for n, _ in m._ScanArgs._fields_))


def scan(m, **k):
    y = dict(y=at(10), ybs=80, yts=16, final=None, kept=None, ws=at(11), size=1 << 20)
    y.update({n: v for n, v in k.items() if n in y})
    return m.lib().cr_selective_scan(ctypes.byref(scan_args(m, **k)), *y.values(), None)


BAD_SCAN = [dict(batch=-1), dict(len=-1), dict(dim=-1), dict(dstate=0), dict(groups=0),
            dict(groups=3), dict(softplus=2), dict(dt_type=2), dict(reserved=1), dict(u=None),
            dict(dt=None), dict(A=None), dict(B=None), dict(C=None), dict(u=at(0) + 1),
            dict(z=at(2) + 1), dict(A=at(5) + 1), dict(dt_bias=at(7) + 2)] + [
    {n + s: -1} for n in ("u", "dt", "z", "B", "C") for s in ("_batch_stride", "_time_stride")]


@pytest.mark.parametrize("bad", BAD_SCAN + [
    dict(index_bytes=2), dict(state=at(8) + 1), dict(lengths=at(9) + 4), dict(y=None),
    dict(y=at(0)), dict(y=at(1)), dict(y=at(2)), dict(yts=15), dict(ybs=15), dict(ybs=-1),
    dict(y=at(10) + 1), dict(final=at(12) + 1), dict(kept=at(13) + 2)])
def test_scan_refuses(m, bad):
    assert scan(m, **bad) == INVALID


def test_scan_unsupported_workspace_and_empty(m):
    assert scan(m, dstate=129) == UNSUPPORTED
    assert scan(m, batch=1 << 40) == UNSUPPORTED
    for bad in (dict(ws=None), dict(ws=at(11) + 4), dict(size=8)):
        assert scan(m, **bad) == WORKSPACE
    assert scan(m, batch=0) == OK and scan(m, dim=0) == OK
    L = m.lib()
    assert L.cr_selective_scan_checkpoints(0) == 0 and L.cr_selective_scan_checkpoints(1) == 1
    assert L.cr_selective_scan_workspace_bytes(2, 5, 16, 16) >= 256
    assert L.cr_selective_scan_workspace_bytes(-2, 5, 16, 16) == 0


def scan_back(m, ws=at(30), size=1 << 26, **k):
    g = {n: at(12 + i) for i, (n, t) in enumerate(m._ScanGrads._fields_)}
    g.update(dy_batch_stride=80, dy_time_stride=16, dfinal=None, dstate=None)
    g.update({n: v for n, v in k.items() if n in g})
    c = m._ScanGrads(*(g[n] for n, _ in m._ScanGrads._fields_))
    return m.lib().cr_selective_scan_backward(ctypes.byref(scan_args(m, **k)), ctypes.byref(c),
                                              ws, size, None)


@pytest.mark.parametrize("bad", BAD_SCAN + [
    dict(dy=None), dict(dy_time_stride=-1), dict(checkpoints=None), dict(du=None), dict(ddt=None),
    dict(dz=None), dict(dB=None), dict(dC=None), dict(dA=None), dict(du=at(0)), dict(dC=at(4)),
    dict(dy=at(12) + 1), dict(dA=at(22) + 2)])
def test_scan_backward_refuses(m, bad):
    assert scan_back(m, **bad) == INVALID


def test_scan_backward_workspace(m):
    need = m.lib().cr_selective_scan_backward_workspace_bytes(2, 5, 16, 16, 2)
    assert need >= 256 and need % 256 == 0
    assert m.lib().cr_selective_scan_backward_workspace_bytes(2, 5, 16, 16, 3) == 0
    for ws, size in ((None, need), (at(30) + 4, need), (at(30), need - 1)):
        assert scan_back(m, ws, size) == WORKSPACE
    assert scan_back(m, dstate=129) == UNSUPPORTED


def test_scan_backward_refuses_before_it_starts(m):
    """What cannot be done is refused with nothing enqueued: more sums of B and C
    than a grid has blocks, and one gradient of two that is missing."""
    size = 1 << 62
    assert scan_back(m, size=size, batch=1 << 10, len=1 << 27, groups=1) == UNSUPPORTED
    assert scan_back(m, dim=0, dC=None) == INVALID
    assert scan_back(m, dim=0, dB=at(13) + 1) == INVALID
    assert scan_back(m, dim=0, dC=at(3)) == INVALID
    assert scan_back(m, dim=0, len=0, dC=None) == OK


def scan_step(m, **k):
    y = dict(state=at(8), rows=2, slots=None, y=at(10), ybs=16)
    y.update({n: v for n, v in k.items() if n in y})
    return m.lib().cr_selective_scan_step(ctypes.byref(scan_args(m, **{"len": 1, **k})),
                                          *y.values(), None)


@pytest.mark.parametrize("bad", [b for b in BAD_SCAN if "len" not in b] + [
    dict(len=2), dict(len=0), dict(rows=-1), dict(rows=1), dict(slots=at(9), index_bytes=2),
    dict(slots=at(9) + 4), dict(y=None), dict(y=at(0)), dict(ybs=8), dict(y=at(10) + 1)])
def test_scan_step_refuses(m, bad):
    assert scan_step(m, **bad) == INVALID


def test_binding_refuses_host_tensors(m):
    import torch
    x = torch.zeros(2, 3, 4)
    w = torch.zeros(4, 4)
    with pytest.raises(ValueError):
        m.causal_conv(x, w)
    with pytest.raises(ValueError):
        m.embedding(torch.zeros(3, dtype=torch.int64), w)
    with pytest.raises(ValueError):
        m.embedding_backward(torch.zeros(3, dtype=torch.int64), w[:3], 10)
    with pytest.raises(ValueError):
        m.selective_scan(x, x, w, x, x)


def numeric(loss, args, name, rng):
    v = rng.standard_normal(args[name].shape)
    e = 1e-5
    up, down = ({**args, name: args[name] + s * e * v} for s in (1, -1))
    return (loss(up) - loss(down)) / (2 * e), v


def test_reference_gradients(m):
    """Central differences with e = 1e-5: e^2 of the third derivative plus
    2^-53 / e of the values, both below 1e-8 of sums of a few hundred terms."""
    rng = np.random.default_rng(0)
    f = rng.standard_normal
    Bn, T, D, N, G = 2, 5, 4, 3, 2
    a = dict(u=f((Bn, T, D)), dt=f((Bn, T, D)), A=-np.exp(f((D, N))), B=f((Bn, T, G, N)),
             C=f((Bn, T, G, N)), D=f(D), z=f((Bn, T, D)), dt_bias=f(D), softplus=True,
             state=f((Bn, D, N)), lengths=[5, 3])
    dy, df = f((Bn, T, D)), f((Bn, D, N))
    g = R.scan(**a, dy=dy, dfinal=df)["grads"]

    def loss(q):
        r = R.scan(**q)
        return (r["y"][0] * dy).sum() + (r["final"][0] * df).sum()
    for k in ("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "state"):
        want, v = numeric(loss, a, k, rng)
        assert abs((g[k][0] * v).sum() - want) < 1e-6, k
    a = dict(x=f((2, 6, 3)), w=f((3, 4)), bias=f(3), silu=True, state=f((2, 3, 3)), lengths=[6, 2])
    dyc, dfc = f((2, 6, 3)), f((2, 3, 3))
    g = R.conv(**a, dy=dyc, dfinal=dfc)["grads"]

    def conv_loss(q):
        r = R.conv(**q)
        return (r["y"][0] * dyc).sum() + (r["final"][0] * dfc).sum()
    for k, n in (("x", "x"), ("w", "weight"), ("bias", "bias"), ("state", "state")):
        want, v = numeric(conv_loss, a, k, rng)
        assert abs((g[n][0] * v).sum() - want) < 1e-6, k


def scan_back_dstate(m, dstate_out, **k):
    """scan_back with the gradient of the state, whose name the argument block
    gives to the number of states."""
    g = {n: at(12 + i) for i, (n, t) in enumerate(m._ScanGrads._fields_)}
    g.update(dy_batch_stride=80, dy_time_stride=16)
    g.update({n: v for n, v in k.items() if n in g}, dstate=dstate_out)
    c = m._ScanGrads(*(g[n] for n, _ in m._ScanGrads._fields_))
    return m.lib().cr_selective_scan_backward(ctypes.byref(scan_args(m, **k)), ctypes.byref(c),
                                              at(30), 1 << 26, None)


SCAN_BACK_READ = dict(u=at(0), dt=at(1), z=at(2), B=at(3), C=at(4), A=at(5), D=at(6),
                      dt_bias=at(7), state=at(8), lengths=at(9), dy=at(40), dfinal=at(41),
                      checkpoints=at(42))
# what a call reads, by its name in the calls above, and what it writes
READ_AND_WRITTEN = [
    (embed, dict(tokens=at(0), table=at(1)), ("out",)),
    (embed_grad, dict(tokens=at(0), grad=at(1)), ("dw",)),
    (conv, dict(x=at(0), weight=at(1), bias=at(2), state=at(3), lengths=at(4)), ("y", "final")),
    (conv_back, dict(x=at(0), weight=at(1), bias=at(2), state=at(3), lengths=at(4), dy=at(5),
                     dfinal=at(40)), ("dx", "dweight", "dbias", "dstate")),
    (conv_step, dict(x=at(0), state=at(1), slots=at(41), weight=at(2), bias=at(42)), ("y",)),
    (conv_step, dict(x=at(0), slots=at(41), weight=at(2), bias=at(42)), ("state",)),
    (scan, dict(u=at(0), dt=at(1), z=at(2), B=at(3), C=at(4), A=at(5), D=at(6), dt_bias=at(7),
                lengths=at(9)), ("y", "final", "kept")),
    (scan, dict(state=at(8)), ("y", "kept")),  # the final state may take its place
    (scan_back, SCAN_BACK_READ, ("du", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias")),
    (scan_back_dstate, SCAN_BACK_READ, ("dstate_out",)),
    (scan_step, dict(u=at(0), dt=at(1), z=at(2), B=at(3), C=at(4), A=at(5), D=at(6),
                     dt_bias=at(7), slots=at(9), state=at(8)), ("y",)),
    (scan_step, dict(u=at(0), dt=at(1), z=at(2), B=at(3), C=at(4), A=at(5), D=at(6),
                     dt_bias=at(7), slots=at(9)), ("state",)),
]


@pytest.mark.parametrize("call,read,written", READ_AND_WRITTEN)
def test_outputs_that_are_inputs_are_refused(m, call, read, written):
    for name in written:
        for other, pointer in read.items():
            assert call(m, **{**read, name: pointer}) == INVALID, (name, other)
