"""Gated scan: what is left of a state, and of a gradient, is right to a few
roundings of itself, however much of it is forgotten within the steps that are
worked on at once."""
import numpy as np
import pytest
import torch

from .model_reference import f64
from .more_reference import U, sigmoid

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def relative(gate):
    """Bounds of the error of products of a along the steps, relative. A factor a = 1 -
    r is off by r / a of r's error (8 + |gate| roundings: its exponent's, the
    instructions') and a rounding of each product; a run's map, and two maps joined,
    round three times for each."""
    a, r = sigmoid(gate), sigmoid(-gate)
    return np.cumsum(U * (5 + (8 + np.abs(gate)) * r / a), axis=1)


@pytest.mark.parametrize("T", [1, 3, 9, 16, 25, 100, 128, 150, 700])
@pytest.mark.parametrize("left", [2.0 ** -3, 2.0 ** -6, 2.0 ** -8, 2.0 ** -40])
def test_what_is_left(scr, T, left):
    """x is zero, so that the state is a product: of it `left` remains after 16 steps
    (gates differ by a few)."""
    g = torch.Generator().manual_seed(T)
    B, D = 2, 64
    a = left ** (1 / 16)
    gate = float(np.log(a / (1 - a))) + 0.7 * torch.randn(B, T, D, generator=g)
    state = 100 * torch.randn(B, D, generator=g)
    zero = torch.zeros(B, T, D, device=DEV)
    y, final, kept = scr.gated_scan(zero, gate.to(DEV), state=state.to(DEV), return_state=True,
                                    return_checkpoints=True)
    e = relative(f64(gate))
    want = f64(state)[:, None] * np.cumprod(sigmoid(f64(gate)), axis=1)
    tiny = 2.0 ** -120  # (below 2^-126 the instructions give zero)
    for got, k in ((f64(y), slice(None)), (f64(final)[:, None], slice(-1, None)),
                   (f64(kept)[:, 1:], slice(15, T - 1, 16))):
        off = np.abs(got - want[:, k])
        assert (off <= e[:, k] * np.abs(want[:, k]) + tiny).all()
    # the way back: a gradient of the final state alone
    back = scr.gated_scan_backward(zero, zero, gate.to(DEV), state=state.to(DEV),
                                   dfinal=state.to(DEV), checkpoints=kept)["state"]
    assert (np.abs(f64(back) - want[:, -1]) <= e[:, -1] * np.abs(want[:, -1]) + tiny).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("z", [True, False])
def test_gradients_at_gates_that_hold(scr, dtype, z):
    """r = exp(-gate) as long as binary32 has it, and zero for a gate of infinity,
    where the gradients of x and gate are zero whatever comes back."""
    B, T, D = 2, 40, 32
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    gate = (70 + 16 * torch.rand(B, T, D, generator=g)).to(dtype)
    x, dy, zz = (r(B, T, D).to(dtype) for _ in range(3))
    state = r(B, D)
    gate[:, 7], x[:, 7] = float("inf"), 3e4
    d = dict(x=x, gate=gate, z=zz if z else None, state=state)
    d = {k: v if v is None else v.to(DEV) for k, v in d.items()}
    got = scr.gated_scan_backward(dy.to(DEV) * 2.0 ** 20, **d, dfinal=torch.zeros(B, D, device=DEV))
    s = f64(zz) * sigmoid(f64(zz)) if z else 1.0
    G = np.cumsum((f64(dy) * 2.0 ** 20 * s)[:, ::-1], axis=1)[:, ::-1]  # a is 1 here
    size = np.cumsum(np.abs(f64(dy) * 2.0 ** 20 * s)[:, ::-1], axis=1)[:, ::-1]
    with np.errstate(over="ignore"):
        rr = 1 / (1 + np.exp(f64(gate)))
    step = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    e = (100 + 3 * 86) * U  # r's, and the sums of 40 terms and silu's
    for name, want, many in (("x", rr * G, rr * size),
                             ("gate", rr * G * (f64(state)[:, None] - f64(x)),
                              rr * size * (np.abs(f64(state)[:, None]) + np.abs(f64(x))))):
        # h is the state to 2^-100; results below 2^-126 are zero
        off = np.abs(f64(got[name]) - want)
        assert (off <= step * np.abs(want) + e * many + 2.0 ** -126).all(), name
        assert not got[name][:, 7].any()
