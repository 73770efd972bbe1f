"""Gated scan with infinities: by the formulas, a state that is infinite stays so
(a > 0) until it meets the other infinity or NaN, and so does what a gradient
carries. What no infinity reaches has the bits that it has without them."""
import numpy as np
import pytest
import torch

from .model_reference import f64
from .more_reference import sigmoid

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def formulas(s, dfinal):
    """In binary64, with its rules for infinities and NaN."""
    x, gate, z, dy, state = (None if s[k] is None else f64(s[k])
                             for k in ("x", "gate", "z", "dy", "state"))
    B, T, D = x.shape
    n = np.full(B, T) if s["lengths"] is None else s["lengths"].numpy()
    out = {k: np.zeros_like(x) for k in ("y", "dx", "dgate", "dz")}
    out["final"], out["dstate"] = state.copy(), f64(dfinal).copy()
    with np.errstate(all="ignore"):
        a, r = sigmoid(gate), sigmoid(-gate)
        silu = 1.0 if z is None else z * sigmoid(z)
        for b in range(B):
            h = [state[b]]
            for t in range(n[b]):
                h.append(a[b, t] * h[-1] + r[b, t] * x[b, t])
                out["y"][b, t] = h[-1] if z is None else h[-1] * silu[b, t]
            out["final"][b] = h[-1]
            back = out["dstate"][b]
            for t in range(n[b] - 1, -1, -1):
                if z is not None:
                    w = sigmoid(z[b, t])
                    out["dz"][b, t] = dy[b, t] * h[t + 1] * (w * (1 + z[b, t] * (1 - w)))
                G = back + dy[b, t] * (1.0 if z is None else silu[b, t])
                out["dx"][b, t] = r[b, t] * G
                out["dgate"][b, t] = (h[t] - x[b, t]) * a[b, t] * r[b, t] * G
                back = a[b, t] * G
            out["dstate"][b] = back
    return out


def run(scr, s, dfinal):
    d = {k: None if s[k] is None else s[k].to(DEV) for k in ("x", "gate", "z", "state", "lengths")}
    y, final, kept = scr.gated_scan(**d, return_state=True, return_checkpoints=True)
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(scr.gated_scan(**d)))
    g = scr.gated_scan_backward(s["dy"].to(DEV), **d, dfinal=dfinal.to(DEV), checkpoints=kept)
    return {"y": y, "final": final, **{"d" + k: v for k, v in g.items()}}


def make(B, T, D, dtype, seed, z=True, lengths=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *q: torch.randn(*q, generator=g)  # noqa: E731
    s = {k: r(B, T, D).to(dtype) for k in ("x", "gate", "dy")}
    s["z"] = r(B, T, D).to(dtype) if z else None
    s["state"] = r(B, D)
    s["lengths"] = None if lengths is None else torch.tensor(lengths)
    return s, r(B, D), g


def check(scr, s, dfinal, put):
    """put: (name, index, value) of what is not finite."""
    plain = run(scr, s, dfinal)
    bad, bad_final = {k: v if v is None else v.clone() for k, v in s.items()}, dfinal.clone()
    for name, at, value in put:
        (bad_final if name == "dfinal" else bad[name])[at] = value
    got, want = run(scr, bad, bad_final), formulas(bad, bad_final)
    for k, v in got.items():
        v, w = f64(v), want[k]
        odd = ~np.isfinite(w)
        assert np.array_equal(v[odd], w[odd], equal_nan=True), k
        same = ~odd & (f64(plain[k]) == v)
        changed = ~odd & ~same  # a gradient of an infinite x is not of x
        assert not changed.any(), (k, np.argwhere(changed)[:5])
    return got


def somewhere(g, B, T, D, count, names):
    put = []
    for i in range(count):
        b, t, d = (int(torch.randint(0, n, (1,), generator=g)) for n in (B, T, D))
        name = names[i % len(names)]
        value = (INF, -INF, INF, NAN)[int(torch.randint(0, 4, (1,), generator=g))]
        put.append((name, (b, d) if name in ("state", "dfinal") else (b, t, d), value))
    return put


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(2, 1, 8), (2, 16, 40), (3, 47, 33), (2, 300, 64), (1, 700, 70),
                                   (1, 1100, 32)])
@pytest.mark.parametrize("z", [True, False])
def test_inputs(scr, dtype, shape, z):
    B, T, D = shape
    s, dfinal, g = make(B, T, D, dtype, T + D, z)
    check(scr, s, dfinal, somewhere(g, B, T, D, 1 + D // 2, ["x", "x", "state"]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(2, 1, 8), (3, 47, 33), (2, 300, 64), (1, 1100, 32)])
@pytest.mark.parametrize("z", [True, False])
def test_gradients(scr, dtype, shape, z):
    B, T, D = shape
    s, dfinal, g = make(B, T, D, dtype, T + D, z)
    check(scr, s, dfinal, somewhere(g, B, T, D, 1 + D // 2, ["dy", "dfinal", "dy"]))
    check(scr, s, dfinal, somewhere(g, B, T, D, 1 + D, ["x", "dy", "state", "dfinal"]))


def test_at_the_end_of_a_sequence(scr):
    """The last step's infinity is the final state, wherever a run of steps ends."""
    lengths = [1, 2, 15, 16, 17, 127, 128, 129, 250, 0]
    s, dfinal, _ = make(len(lengths), 260, 24, torch.bfloat16, 3, lengths=lengths)
    put = [("x", (b, n - 1, b), (INF, -INF)[b % 2]) for b, n in enumerate(lengths) if n]
    put += [("state", (9, 3), INF), ("dfinal", (9, 4), -INF), ("dfinal", (3, 7), INF)]
    got = check(scr, s, dfinal, put)
    assert got["final"].isinf().sum() == len(lengths)


def test_steps(scr):
    s, _, _ = make(4, 3, 33, torch.float32, 5)
    state = s["state"].to(DEV)
    state[1, 2], state[2, 3], state[3, 4] = INF, -INF, NAN
    d = {k: s[k].to(DEV) for k in ("x", "gate", "z")}
    d["x"][0, 1, 7] = -INF
    d["x"][2, 2, 3] = INF  # and the state's is the other one
    for t in range(3):
        scr.gated_scan_step(d["x"][:, t], d["gate"][:, t], state, d["z"][:, t])
    assert state[1, 2] == INF and state[0, 7] == -INF
    assert state[2, 3].isnan() and state[3, 4].isnan()
    assert state.isfinite().sum() == state.numel() - 4


def test_strided_rows_with_nan_beside_them(scr):
    """Rows that start anywhere: what stands beside the last channel is not its own."""
    s, dfinal, g = make(2, 150, 31, torch.bfloat16, 6)
    want = run(scr, s, dfinal)
    wide = {}
    for k in ("x", "gate", "z", "dy"):
        big = torch.full((2, 150, 35), NAN, dtype=torch.bfloat16, device=DEV)
        big[..., 2:33] = s[k].to(DEV)
        wide[k] = big[..., 2:33]
    d = dict(gate=wide["gate"], z=wide["z"], state=s["state"].to(DEV))
    y, final, kept = scr.gated_scan(wide["x"], **d, return_state=True, return_checkpoints=True)
    got = scr.gated_scan_backward(wide["dy"], wide["x"], **d, dfinal=dfinal.to(DEV),
                                  checkpoints=kept)
    assert torch.equal(y, want["y"]) and torch.equal(final, want["final"])
    assert all(torch.equal(v, want["d" + k]) for k, v in got.items())


@pytest.mark.parametrize("T", [40, 1100])
def test_final_state_over_the_initial_one(scr, T):
    """A sequence that is gone through again begins from the state that it was given."""
    import ctypes
    from scan_canonical_reduce_gb300 import model as m
    s, _, _ = make(2, T, 40, torch.bfloat16, 7)
    s["x"][0, T // 2, 3] = INF
    s["state"][1, 5] = -INF
    x, gate, z, state = (s[k].to(DEV) for k in ("x", "gate", "z", "state"))
    y, final = scr.gated_scan(x, gate, z, state=state, return_state=True)
    y2 = torch.empty_like(y)
    a = m._GateArgs(2, T, 40, 3, 8, *(v for k in (x, gate, z) for v in (k.data_ptr(), T * 40, 40)),
                    state.data_ptr(), None)
    assert scr.lib().cr_gated_scan(ctypes.byref(a), y2.data_ptr(), T * 40, 40, state.data_ptr(),
                                   None, torch.cuda.current_stream(DEV).cuda_stream) == 0
    assert torch.equal(y, y2) and torch.equal(final, state)
    assert final[0, 3] == INF and final[1, 5] == -INF and final.isinf().sum() == 2


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("z", [True, False])
def test_gates_that_are_nan(scr, dtype, z):
    """What is infinite becomes NaN there, on its way on and on its way back."""
    s, dfinal, _ = make(3, 300, 20, dtype, 8, z)
    put = [("dy", (0, 250, 3), INF), ("gate", (0, 240, 3), NAN),
           ("dy", (0, 100, 4), -INF), ("gate", (0, 100, 4), NAN),
           ("dfinal", (1, 5), INF), ("gate", (1, 299, 5), NAN),
           ("x", (1, 20, 6), INF), ("gate", (1, 21, 6), NAN),
           ("x", (2, 20, 7), INF), ("dy", (2, 200, 7), INF), ("gate", (2, 120, 7), NAN),
           ("state", (2, 8), INF), ("gate", (2, 0, 8), NAN)]
    check(scr, s, dfinal, put)
