"""Gated scan: sequences whose time is shared by every number of blocks of a
cluster, against a plain 64-bit evaluation (tests/more_reference.py derives the
bounds)."""
import pytest
import torch

from . import more_reference as M
from .model_reference import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TILE = 128  # steps of a block and turn


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def make(B, T, D, dtype, seed, lengths=None):
    g = torch.Generator().manual_seed(seed)
    s = {k: torch.randn(B, T, D, generator=g).to(dtype) for k in ("x", "gate", "z", "dy")}
    s["gate"] = (s["gate"].float() + 3 * torch.randn(D, generator=g)).to(dtype)
    s["state"], s["dfinal"] = (torch.randn(B, D, generator=g) for _ in range(2))
    s["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    for b, n in enumerate(lengths or ()):
        for k in ("x", "gate", "z", "dy"):
            s[k][b, n:] = float("nan")
    return s


def check(scr, s):
    n = None if s["lengths"] is None else s["lengths"].tolist()
    ref = M.gated(f64(s["x"]), f64(s["gate"]), f64(s["z"]), f64(s["state"]), n, f64(s["dy"]),
                  f64(s["dfinal"]))
    d = {k: v if v is None else v.to(DEV) for k, v in s.items()}
    dy, dfinal = d.pop("dy"), d.pop("dfinal")
    y, final, kept = scr.gated_scan(**d, return_state=True, return_checkpoints=True)
    M.near(y, *ref["y"], "y")
    M.near(final, *ref["final"], "final")
    g = scr.gated_scan_backward(dy, **d, dfinal=dfinal, checkpoints=kept)
    for k in ("x", "gate", "z", "state"):
        M.near(g[k], *ref["d" + k], "d" + k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 6, 7, 8, 11])
@pytest.mark.parametrize("D", [32, 33])
def test_blocks_by_length(scr, dtype, blocks, D):
    """One sequence of that many tiles, the last of them not whole."""
    check(scr, make(1, TILE * blocks - 28, D, dtype, blocks))


@pytest.mark.parametrize("sequences", [152, 101, 76, 60, 50, 43, 38])
def test_blocks_by_sequences(scr, sequences):
    """As many blocks a sequence as leave places for all (2 to 8), of sequences that
    leave some of them without a step, or all."""
    T = 2 * 8 * TILE + 5
    lengths = [(T, 0, 1, TILE, TILE + 1, 300, T - 6, 5 * TILE)[b % 8] if b < 16 else 3 + b % 40
               for b in range(sequences)]
    check(scr, make(sequences, T, 8, torch.bfloat16, sequences, lengths))


def test_many_launches(scr):
    """Clusters that begin while others end: the same bits every time."""
    s = {k: v if v is None else v.to(DEV)
         for k, v in make(4, 8 * TILE, 512, torch.bfloat16, 1, [1, 8 * TILE, 0, 17]).items()}
    dy, dfinal = s.pop("dy"), s.pop("dfinal")
    y, kept = scr.gated_scan(**s, return_checkpoints=True)
    g = scr.gated_scan_backward(dy, **s, dfinal=dfinal, checkpoints=kept)
    for _ in range(100):
        assert torch.equal(scr.gated_scan(**s), y)
        again = scr.gated_scan_backward(dy, **s, dfinal=dfinal, checkpoints=kept)
        assert all(torch.equal(again[k], g[k]) for k in g)
