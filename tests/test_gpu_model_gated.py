"""Gated scan: forward, gradient and single tokens against a plain 64-bit
evaluation (tests/more_reference.py derives the bounds)."""
import numpy as np
import pytest
import torch

from . import more_reference as M
from .model_reference import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAN = float("nan")


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def make(B, T, D, dtype, seed, z=True, state=True, lengths=None, memory=3.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = {"x": r(B, T, D).to(dtype), "gate": (r(B, T, D) + memory * r(D)).to(dtype),
         "z": r(B, T, D).to(dtype) if z else None, "state": r(B, D) if state else None,
         "lengths": None if lengths is None else torch.tensor(lengths, dtype=torch.int32)}
    dy, dfinal = r(B, T, D).to(dtype), r(B, D)
    if lengths is not None:
        for b, n in enumerate(lengths):
            for v in (s["x"], s["gate"], s["z"], dy):
                if v is not None:
                    v[b, max(n, 0):] = NAN
    return s, dy, dfinal


def dev(s):
    return {k: v if v is None else v.to(DEV) for k, v in s.items()}


def reference(s, dy=None, dfinal=None):
    n = None if s["lengths"] is None else s["lengths"].tolist()
    return M.gated(f64(s["x"]), f64(s["gate"]), f64(s["z"]), f64(s["state"]), n, f64(dy),
                   f64(dfinal))


def check(scr, s, dy, dfinal):
    d = dev(s)
    ref = reference(s, dy, dfinal)
    y, final, kept = scr.gated_scan(**d, return_state=True, return_checkpoints=True)
    M.near(y, *ref["y"], "y")
    M.near(final, *ref["final"], "final")
    g = scr.gated_scan_backward(dy.to(DEV), **d, dfinal=dfinal.to(DEV), checkpoints=kept)
    names = {"x", "gate"} | {k for k in ("z", "state") if s[k] is not None}
    assert set(g) == names
    for k in names:
        M.near(g[k], *ref["d" + k], "d" + k)
    again = scr.gated_scan_backward(dy.to(DEV), **d, dfinal=dfinal.to(DEV))
    assert all(torch.equal(g[k], again[k]) for k in g)
    return y, final, g


SHAPES = [(1, 1, 1), (1, 1, 8), (2, 3, 5), (2, 65, 33), (1, 200, 512), (3, 129, 1030),
          (1, 1100, 64), (2, 257, 130), (1, 2500, 40), (5, 16, 2048), (1, 17, 7)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(scr, dtype, shape):
    check(scr, *make(*shape, dtype, 1))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("z,state", [(False, False), (False, True), (True, False)])
def test_without_z_or_state(scr, dtype, z, state):
    check(scr, *make(2, 150, 70, dtype, 2, z, state))


LENGTHS = [[70, 0, 1, 2, 33, 69], [5, 5, 0, 300, -4, 64], [16, 17, 15, 48, 49, 32]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("z", [True, False])
def test_lengths(scr, dtype, lengths, z):
    y, final, g = check(scr, *make(6, 70, 36, dtype, 3, z, lengths=lengths))
    for b, n in enumerate(lengths):
        for v in (y, g["x"], g["gate"]) + ((g["z"],) if z else ()):
            assert not v[b, max(n, 0):].any()


def test_long_lengths(scr):
    """Sequences that end in every part of what is worked on at once."""
    lengths = [3000, 0, 1, 1023, 1024, 1025, 2047, 513, 129]
    check(scr, *make(9, 3000, 40, torch.bfloat16, 4, lengths=lengths))


def test_long_memory(scr):
    """A gate that forgets 2^-12 of a step: rounding a to binary32 would lose one
    part in 8000 of the rate, and the sum of many steps with it."""
    T, D = 20000, 4
    x = torch.ones(1, T, D)
    gate = torch.full((1, T, D), 8.3)
    s = {"x": x, "gate": gate, "z": None, "state": None, "lengths": None}
    check(scr, s, torch.full((1, T, D), 1e-3), torch.ones(1, D))


def test_forgetting_what_was_large(scr):
    """Nothing of a huge state is left after a step that forgets it."""
    D = 64
    g = torch.Generator().manual_seed(5)
    gate = 2 * torch.randn(1, 300, D, generator=g)
    gate[:, 5] = -90.0
    gate[:, 6, ::2] = -float("inf")
    gate[:, 40] = 90.0
    gate[:, 41, ::2] = float("inf")
    s = {"x": torch.randn(1, 300, D, generator=g), "gate": gate, "z": None,
         "state": torch.full((1, D), 1e30), "lengths": None}
    d = dev(s)
    y, final = scr.gated_scan(**d, return_state=True)
    ref = reference(s)
    M.near(y, *ref["y"], "y")
    M.near(final, *ref["final"], "final")
    assert torch.equal(y[:, 5:7, ::2], d["x"][:, 5:7, ::2])  # r is 1: nothing of it at all


def test_decay_past_binary32(scr):
    """Steps whose decays' product leaves binary32's range take the state with it."""
    D, T = 32, 2600
    for gate, state in ((-3.0, 1e30), (-40.0, 1e38), (0.0, 1e38), (-0.01, 1e25), (4.0, 1e38)):
        s = {"x": torch.zeros(1, T, D), "gate": torch.full((1, T, D), gate), "z": None,
             "state": torch.full((1, D), state), "lengths": None}
        y = scr.gated_scan(**dev(s))
        want, bound = reference(s)["y"]
        # a decay below 2^-126 is zero: what it would have left is below that of the state
        M.near(y, want, bound + 2.0 ** -126 * state, "y")


def test_nan_and_infinity_stay_in_their_channel_and_after_their_step(scr):
    s, dy, dfinal = make(2, 400, 70, torch.float32, 6)
    d = dev(s)
    y0, f0 = scr.gated_scan(**d, return_state=True)
    for t, value in ((0, NAN), (37, float("inf")), (399, NAN)):
        bad = {k: v if v is None else v.clone() for k, v in d.items()}
        bad["x"][1, t, 33] = value
        y, f = scr.gated_scan(**bad, return_state=True)
        mask = torch.ones_like(y0, dtype=torch.bool)
        mask[1, t:, 33] = False
        assert torch.equal(y[mask], y0[mask])
        assert not y[1, t, 33].isfinite()
        keep = torch.ones_like(f0, dtype=torch.bool)
        keep[1, 33] = False
        assert torch.equal(f[keep], f0[keep])


def test_gradient_matches_differences(scr):
    s, dy, dfinal = make(2, 20, 6, torch.float32, 7)
    got = scr.gated_scan_backward(dy.to(DEV), **dev(s), dfinal=dfinal.to(DEV))
    gen = torch.Generator().manual_seed(8)
    for name in got:
        v = torch.randn(s[name].shape, generator=gen, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            m = {k: f64(t) for k, t in s.items()}
            m[name] = m[name] + sign * 1e-4 * v.numpy()
            ref = M.gated(m["x"], m["gate"], m["z"], m["state"], None)
            ends.append((ref["y"][0] * f64(dy)).sum() + (ref["final"][0] * f64(dfinal)).sum())
        want = (ends[0] - ends[1]) / 2e-4
        have = (f64(got[name]) * v.numpy()).sum()
        size = (np.abs(f64(got[name])) * np.abs(v.numpy())).sum()
        assert abs(have - want) <= 1e-5 * size, name


def test_strides_and_alignment(scr):
    """The same bits from strided, misaligned, transposed and repeated inputs."""
    B, T, D = 3, 90, 72
    s, dy, dfinal = make(B, T, D, torch.bfloat16, 9)
    d, dyd, df = dev(s), dy.to(DEV), dfinal.to(DEV)
    want = scr.gated_scan(**d)
    gw = scr.gated_scan_backward(dyd, **d, dfinal=df)

    def placed(v, offset, pad):
        big = torch.full((B * (T + 1) * (D + pad) + offset,), NAN, dtype=v.dtype, device=DEV)
        return big[offset:].as_strided((B, T, D), ((T + 1) * (D + pad), D + pad, 1)).copy_(v)

    for offset, pad in ((0, 8), (1, 0), (3, 5), (2, 2), (2, 0)):
        q = {k: placed(d[k], offset, pad) for k in ("x", "gate", "z")}
        out = placed(torch.zeros_like(want), offset, pad)
        assert scr.gated_scan(**{**d, **q}, out=out) is out and torch.equal(out, want)
        got = scr.gated_scan_backward(placed(dyd, offset, pad), **{**d, **q}, dfinal=df)
        assert all(torch.equal(got[k], gw[k]) for k in gw)
    q = {k: d[k].transpose(1, 2).contiguous().transpose(1, 2) for k in ("x", "gate", "z")}
    assert torch.equal(scr.gated_scan(**{**d, **q}), want)
    one = {k: d[k][:1].expand(B, T, D) for k in ("x", "gate", "z")}
    assert torch.equal(scr.gated_scan(**one), scr.gated_scan(**{k: v.contiguous()
                                                               for k, v in one.items()}))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [1, 40, 333, 2048])
@pytest.mark.parametrize("z", [True, False])
def test_step(scr, dtype, D, z):
    s, _, _ = make(5, 1, D, dtype, 10, z)
    ref = reference(s)
    d = {k: v if v is None else v.to(DEV) for k, v in s.items()}
    state = d["state"].clone()
    one = [None if d[k] is None else d[k][:, 0] for k in ("x", "gate", "z")]
    y = scr.gated_scan_step(one[0], one[1], state, one[2])
    M.near(y, ref["y"][0][:, 0], ref["y"][1][:, 0], "y")
    M.near(state, *ref["final"], "state")
    # rows of a pool, one of them padding
    pool = torch.full((9, D), 7.0, device=DEV)
    slots = torch.tensor([8, 0, -1, 9, 3], device=DEV)
    live = [0, 1, 4]
    for b in live:
        pool[slots[b]] = d["state"][b]
    y2 = scr.gated_scan_step(one[0], one[1], pool, one[2], slots=slots)
    assert torch.equal(y2[live], y[live]) and not y2[2].any() and not y2[3].any()
    for b in live:
        assert torch.equal(pool[slots[b]], state[b])
    rest = [i for i in range(9) if i not in (8, 0, 3)]
    assert (pool[rest] == 7.0).all()


def test_single_tokens_follow_a_prompt(scr):
    """A prompt cut into calls, and token by token."""
    s, _, _ = make(3, 61, 130, torch.float32, 11)
    d = dev(s)
    ref = reference(s)
    h, parts = d["state"], []
    for t0, t1 in ((0, 20), (20, 21), (21, 40)):
        y, h = scr.gated_scan(*(d[k][:, t0:t1] for k in ("x", "gate", "z")), state=h,
                              return_state=True)
        parts.append(y)
    state = h.clone()
    for t in range(40, 61):
        parts.append(scr.gated_scan_step(d["x"][:, t], d["gate"][:, t], state, d["z"][:, t])[:, None])
    M.near(torch.cat(parts, 1), *ref["y"], "y")
    M.near(state, *ref["final"], "final")


def test_autograd(scr):
    s, dy, dfinal = make(2, 50, 36, torch.float32, 12)
    d, dyd, df = dev(s), dy.to(DEV), dfinal.to(DEV)
    want = scr.gated_scan_backward(dyd, **d, dfinal=df)
    leaves = {k: v.clone().requires_grad_(True) for k, v in d.items() if v is not None}
    y, final = scr.gated_scan(**leaves, return_state=True)
    torch.autograd.backward([y, final], [dyd, df])
    assert all(torch.equal(leaves[k].grad, want[k]) for k in want)
    y, final, kept = scr.gated_scan(**leaves, return_state=True, return_checkpoints=True)
    assert not kept.requires_grad and final.requires_grad
    (g,) = torch.autograd.grad(final, leaves["x"], df)  # the state alone is used
    assert torch.equal(g, scr.gated_scan_backward(torch.zeros_like(dyd), **d, dfinal=df)["x"])
    with pytest.raises(RuntimeError):
        scr.gated_scan(**leaves, out=torch.empty_like(d["x"]))
    y = scr.gated_scan(**leaves)
    (g,) = torch.autograd.grad(y, leaves["gate"], dyd, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    # a state that a step has overwritten is noticed
    y = scr.gated_scan(leaves["x"], leaves["gate"], state=d["state"])
    scr.gated_scan_step(d["x"][:, 0], d["gate"][:, 0], d["state"])
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_refusals(scr):
    s, dy, _ = make(2, 5, 16, torch.float32, 13)
    d = dev(s)
    for bad, error in ((dict(x=d["x"].double()), TypeError), (dict(gate=d["gate"].half()), TypeError),
                       (dict(gate=d["gate"][:1]), ValueError), (dict(z=d["z"][:, :2]), ValueError),
                       (dict(state=d["state"].half()), TypeError), (dict(state=d["x"]), ValueError),
                       (dict(lengths=torch.ones(2, device=DEV)), TypeError),
                       (dict(lengths=torch.ones(3, dtype=torch.int32, device=DEV)), ValueError),
                       (dict(x=d["x"].cpu()), ValueError), (dict(gate=d["gate"].cpu()), ValueError),
                       (dict(out=d["x"]), scr.CrError), (dict(out=d["x"][:1]), ValueError),
                       (dict(x=d["x"][0]), ValueError)):
        with pytest.raises(error):
            scr.gated_scan(**{**d, **bad})
    kept = scr.gated_scan(**d, return_checkpoints=True)[1]
    dyd = dy.to(DEV)
    for bad, error in ((dict(dy=dyd[:1]), ValueError), (dict(checkpoints=kept[:1]), ValueError),
                       (dict(checkpoints=kept.half()), TypeError), (dict(dfinal=dyd), ValueError)):
        with pytest.raises(error):
            scr.gated_scan_backward(**{"dy": dyd, "checkpoints": kept, **d, **bad})
    one = dict(x=d["x"][:, 0], gate=d["gate"][:, 0], state=d["state"])
    for bad, error in ((dict(state=d["state"][:1]), ValueError), (dict(state=d["x"]), ValueError),
                       (dict(state=torch.zeros(16, 2, device=DEV).t()), ValueError),
                       (dict(x=d["x"]), ValueError), (dict(out=one["x"]), scr.CrError),
                       (dict(slots=torch.zeros(2, device=DEV)), TypeError)):
        with pytest.raises(error):
            scr.gated_scan_step(**{**one, **bad})


def test_nothing_to_do(scr):
    for B, T, D in ((0, 5, 8), (2, 0, 8), (2, 5, 0)):
        s, dy, dfinal = make(B, T, D, torch.float32, 14)
        d = dev(s)
        y, final, kept = scr.gated_scan(**d, return_state=True, return_checkpoints=True)
        assert y.shape == (B, T, D) and final.shape == (B, D)
        g = scr.gated_scan_backward(dy.to(DEV), **d, dfinal=dfinal.to(DEV), checkpoints=kept)
        if T == 0:
            assert torch.equal(final, d["state"]) and torch.equal(g["state"], dfinal.to(DEV))
