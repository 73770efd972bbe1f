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
