"""Layer norm's gradient, sampling and the gated scan at the sizes where their
kernels take another shape: columns in threads, rows in a turn, blocks of a row,
slices that shared memory holds or not, the largest vocabulary, many sequences."""
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


# ------------------------------------------------------------- layer norm
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [128, 129, 136, 256, 257, 264, 512, 1024, 1025, 1032, 2048, 2056,
                               2050, 4096, 4104, 4100, 8192, 8191])
@pytest.mark.parametrize("rows", [1, 3, 13])
def test_norm_gradient_shapes(scr, dtype, D, rows):
    """Rows that fill no turn, columns around each number of threads."""
    g = torch.Generator().manual_seed(D)
    x, dy = (torch.randn(rows, D, generator=g).to(dtype) for _ in range(2))
    w = 1 + 0.3 * torch.randn(D, generator=g)
    ref = M.norm(f64(x), f64(w), np.zeros(D), float(np.float32(1e-5)), f64(dy))
    got = scr.layer_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), torch.zeros(D, device=DEV))
    for k in ("x", "weight", "bias"):
        M.near(got[k], *ref[k], "d" + k)


@pytest.mark.parametrize("D", [96, 1000, 2048, 4000, 8000])
def test_norm_gradient_of_a_row_among_others(scr, D):
    """A row's gradient has the same bits wherever it stands and however many
    rows a block takes."""
    g = torch.Generator().manual_seed(D)
    x, dy = (torch.randn(5000, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    w = torch.randn(D, generator=g).to(DEV)
    whole = scr.layer_norm_backward(dy, x, w)["x"]
    for a, b in ((0, 1), (1, 4), (4987, 5000), (17, 1300)):
        assert torch.equal(scr.layer_norm_backward(dy[a:b], x[a:b], w)["x"], whole[a:b])


# --------------------------------------------------------------- sampling
def tokens(x, u, **s):
    full = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    full.update(s)
    return M.sample(f64(x), f64(u), *(np.full(len(x), full[k], dtype=np.float64) for k in full))


def check(scr, x, u, **s):
    d = x.to(DEV)
    got = scr.sample(d, u.to(DEV), **s)
    assert got.cpu().tolist() == tokens(x, u, **s).tolist()
    pad = torch.full((x.shape[0], x.shape[1] + 3), float("nan"), dtype=x.dtype, device=DEV)
    pad[:, 1:-2] = d  # off 16 bytes
    assert torch.equal(scr.sample(pad[:, 1:-2], u.to(DEV), **s), got)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,V", [(1, 4095), (30, 8193), (70, 4100), (140, 16390), (150, 9000),
                                    (160, 4099), (310, 1025), (520, 3001), (3, 131075)])
def test_blocks_of_a_row(scr, dtype, rows, V):
    g = torch.Generator().manual_seed(V)
    x, u = (3 * torch.randn(rows, V, generator=g)).to(dtype), torch.rand(rows, generator=g)
    check(scr, x, u)
    check(scr, x, u, temperature=0.8, top_k=50, top_p=0.9)
    check(scr, x, u, top_p=0.8, min_p=0.01)


def test_slices_beyond_shared_memory(scr):
    """So many rows that each has one block, which reads its row again."""
    g = torch.Generator().manual_seed(20)
    x, u = 2 * torch.randn(310, 40003, generator=g), torch.rand(310, generator=g)
    check(scr, x, u)
    check(scr, x, u, temperature=1.3, top_p=0.95)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_largest_vocabulary(scr, dtype):
    V = 1 << 20
    g = torch.Generator().manual_seed(21)
    x, u = (2 * torch.randn(2, V, generator=g)).to(dtype), torch.rand(2, generator=g)
    check(scr, x, u)
    check(scr, x, u, top_k=200000, top_p=0.99)


def test_largest_vocabulary_of_equal_weights(scr):
    """All alike: the token is that of the index u V, by whole numbers."""
    V = 1 << 20
    u = torch.tensor([0.0, 0.25, 0.5 - 2.0 ** -24, 0.7123, 1 - 2.0 ** -24])
    x = torch.full((5, V), -2.5, device=DEV)
    want = [int(v * V) for v in u.double().tolist()]
    assert scr.sample(x, u.to(DEV)).tolist() == want
    assert scr.sample(x, u.to(DEV), top_k=V // 2).tolist() == [v // 2 for v in want]
    # one on top, all others in one bin, each with nearly the smallest weight in it: the
    # largest sums that a bin has (w is exact to 2^-32, so u V / (1 + (V - 1) w) to 2^-11)
    y = -2.5 - 0.0624 * float(np.log(2.0))
    x[:] = y
    x[:, 7] = -2.5
    w = float(np.exp(np.float64(np.float32(y)) + 2.5))
    got = scr.sample(x, u.to(DEV)).tolist()
    for a, v in zip(got, u.double().tolist()):
        at = v * (1 + (V - 1) * w)  # the first whose running sum is beyond it
        k = 0 if at < 1 else 1 + int((at - 1) / w)
        assert a == (7 if k == 0 else k - 1 if k <= 7 else k)


def test_temperature_without_end(scr):
    """At an infinite temperature all candidates weigh the same."""
    x = torch.tensor([[1.0, -float("inf"), 5.0, 2.0, float("nan")]] * 3, device=DEV)
    u = torch.tensor([0.1, 0.5, 0.9], device=DEV)
    for t in (float("inf"), torch.full((3,), float("inf"), device=DEV)):
        assert scr.sample(x, u, temperature=t).tolist() == [2, 3, 0]


# ------------------------------------------------------------- gated scan
@pytest.mark.parametrize("batch,T,D", [(700, 5, 40), (1, 1, 20000), (3, 129, 65), (2, 1025, 130),
                                       (1, 3000, 33), (37, 300, 200)])
def test_gated_scan_groups(scr, batch, T, D):
    """Many sequences, many channels, and tiles shared by one to eight blocks."""
    g = torch.Generator().manual_seed(T)
    x, gate, z, dy = (torch.randn(batch, T, D, generator=g) for _ in range(4))
    state = torch.randn(batch, D, generator=g)
    lengths = torch.randint(0, T + 1, (batch,), generator=g)
    lengths[0] = T
    ref = M.gated(f64(x), f64(gate), f64(z), f64(state), lengths.numpy(), f64(dy))
    d = dict(x=x.to(DEV), gate=gate.to(DEV), z=z.to(DEV), state=state.to(DEV),
             lengths=lengths.to(DEV))
    M.near(scr.gated_scan(**d), *ref["y"], "y")
    got = scr.gated_scan_backward(dy.to(DEV), **d)
    for k in ("x", "gate", "z", "state"):
        M.near(got[k], *ref["d" + k], "d" + k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [1, 2, 63, 64, 65, 127, 129, 200])
def test_gated_scan_rows_that_start_anywhere(scr, dtype, D):
    """The same bits from rows at any offset and distance, odd and even, whatever
    stands beside them, and from the first and the last elements of a buffer."""
    g = torch.Generator().manual_seed(D)
    B, T = 3, 37
    s = {k: torch.randn(B, T, D, generator=g).to(dtype).to(DEV) for k in ("x", "gate", "z", "dy")}
    lengths = torch.tensor([T, 0, 20], device=DEV)

    def run(v, out=None):
        y, kept = scr.gated_scan(v["x"], v["gate"], v["z"], lengths=lengths,
                                 return_checkpoints=True)
        if out is not None:
            assert scr.gated_scan(v["x"], v["gate"], v["z"], lengths=lengths, out=out) is out
            assert torch.equal(out, y)
        return [y, *scr.gated_scan_backward(v["dy"], v["x"], v["gate"], v["z"], lengths=lengths,
                                            checkpoints=kept).values()]
    want = run(s)

    def placed(v, offset, pad):
        n = B * T * (D + pad) - pad
        big = torch.full((n + offset,), float("nan"), dtype=dtype, device=DEV)
        t = big[offset:].as_strided((B, T, D), (T * (D + pad), D + pad, 1))
        return t.copy_(v)
    cases = (((0, 1, 2, 3), 0), ((1, 1, 1, 1), 1), ((3, 0, 5, 2), 2), ((8, 8, 8, 8), 5))
    for offsets, pad in cases:
        v = {k: placed(s[k], o, pad) for k, o in zip(s, offsets)}
        out = placed(torch.zeros_like(s["x"]), offsets[0], pad)
        for a, b in zip(run(v, out), want):
            assert torch.equal(a, b)
