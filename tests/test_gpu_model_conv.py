"""Short causal convolution: forward, gradient and single tokens against a
plain 64-bit evaluation (tests/model_reference.py says how the tolerances
follow from the number of roundings)."""
import numpy as np
import pytest
import torch

from . import model_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAN = float("nan")


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def make(B, T, D, K, dtype, seed, bias=True, state=True, lengths=None):
    g = torch.Generator().manual_seed(seed)
    s = {"x": torch.randn(B, T, D, generator=g).to(dtype),
         "weight": torch.randn(D, K, generator=g) * 0.5,
         "bias": torch.randn(D, generator=g) * 0.2 if bias else None,
         "state": torch.randn(B, K - 1, D, generator=g).to(dtype) if state else None,
         "lengths": None if lengths is None else torch.tensor(lengths, dtype=torch.int32)}
    dy = torch.randn(B, T, D, generator=g).to(dtype)
    dfinal = torch.randn(B, K - 1, D, generator=g).to(dtype)
    if lengths is not None:
        for b, n in enumerate(lengths):
            s["x"][b, max(n, 0):] = NAN
            dy[b, max(n, 0):] = NAN
    return s, dy, dfinal


def dev(s):
    return {k: v if v is None else v.to(DEV) for k, v in s.items()}


def reference(s, act, dy=None, dfinal=None):
    n = None if s["lengths"] is None else s["lengths"].tolist()
    return R.conv(R.f64(s["x"]), R.f64(s["weight"]), R.f64(s["bias"]), act == "silu",
                  R.f64(s["state"]), n, R.f64(dy), R.f64(dfinal))


# roundings: K products and sums, the sigmoid's few operations (each 2 to 4 units)
FORWARD = 16

SHAPES = [(1, 1, 1, 2), (1, 1, 8, 4), (2, 3, 5, 4), (2, 65, 33, 3), (1, 200, 512, 4),
          (3, 129, 1030, 2), (2, 0, 16, 4)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(scr, dtype, act, shape):
    s, _, _ = make(*shape, dtype, 1)
    y, final = scr.causal_conv(**dev(s), activation=act, return_state=True)
    ref = reference(s, act)
    R.close(y, *ref["y"], FORWARD, "y")
    assert np.array_equal(R.f64(final), ref["final"][0])
    s["bias"] = s["state"] = None
    y = scr.causal_conv(**dev(s), activation=act)
    R.close(y, *reference(s, act)["y"], FORWARD, "y without bias and state")


LENGTHS = [[70, 0, 1, 2, 33, 69], [5, 5, 0, 300, -4, 64]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("K", [2, 3, 4])
def test_lengths(scr, dtype, lengths, K):
    s, dy, dfinal = make(6, 70, 36, K, dtype, 2, lengths=lengths)
    y, final = scr.causal_conv(**dev(s), activation="silu", return_state=True)
    ref = reference(s, "silu", dy, dfinal)
    R.close(y, *ref["y"], FORWARD, "y")
    assert np.array_equal(R.f64(final), ref["final"][0])
    g = scr.causal_conv_backward(dy.to(DEV), **dev(s), activation="silu", dfinal=dfinal.to(DEV))
    check_grads(g, ref["grads"], 6 * 70)


def check_grads(g, ref, rows):
    for name, v in g.items():
        # the sums over positions add up to `rows` roundings to those of a term
        R.close(v, *ref[name], FORWARD + 8 + (rows if name in ("weight", "bias") else 0), name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(scr, dtype, act, shape):
    s, dy, dfinal = make(*shape, dtype, 3)
    g = scr.causal_conv_backward(dy.to(DEV), **dev(s), activation=act, dfinal=dfinal.to(DEV))
    assert set(g) == {"x", "weight", "bias", "state"}
    check_grads(g, reference(s, act, dy, dfinal)["grads"], shape[0] * shape[1])
    s["bias"] = s["state"] = None
    g = scr.causal_conv_backward(dy.to(DEV), **dev(s), activation=act)
    assert set(g) == {"x", "weight"}
    check_grads(g, reference(s, act, dy)["grads"], shape[0] * shape[1])


def test_gradient_matches_differences(scr):
    """The gradient's product with a direction against central differences of
    the 64-bit formula: their error is eps^2 / 6 of the third derivative, which
    eps = 1e-4 takes far below the gradient's own binary32 rounding."""
    s, dy, _ = make(2, 20, 6, 4, torch.float32, 4)
    g = scr.causal_conv_backward(dy.to(DEV), **dev(s), activation="silu")
    gen = torch.Generator().manual_seed(5)
    for name in g:
        v = torch.randn(s[name].shape, generator=gen, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            m = {k: R.f64(t) for k, t in s.items()}
            m[name] = m[name] + sign * 1e-4 * v.numpy()
            ref = R.conv(m["x"], m["weight"], m["bias"], True, m["state"], None)
            ends.append((ref["y"][0] * R.f64(dy)).sum())
        want = (ends[0] - ends[1]) / 2e-4
        got = (R.f64(g[name]) * v.numpy()).sum()
        size = (np.abs(R.f64(g[name])) * np.abs(v.numpy())).sum()
        assert abs(got - want) <= 1e-5 * size, name


def test_strides_and_alignment(scr):
    """The same bits from strided, misaligned, transposed and repeated inputs."""
    s, dy, _ = make(3, 40, 24, 4, torch.bfloat16, 6)
    d = dev(s)
    want = scr.causal_conv(**d, activation="silu")
    gwant = scr.causal_conv_backward(dy.to(DEV), **d, activation="silu")
    wide = torch.full((3, 40, 61), NAN, dtype=torch.bfloat16, device=DEV)
    for view in (wide[:, :, 5:29], wide[:, :, 8:32]):
        wide.fill_(NAN)
        view.copy_(d["x"])
        got = scr.causal_conv(**{**d, "x": view}, activation="silu")
        assert torch.equal(got, want)
        g = scr.causal_conv_backward(dy.to(DEV), **{**d, "x": view}, activation="silu")
        assert all(torch.equal(g[k], gwant[k]) for k in g)
    t = d["x"].permute(2, 0, 1).contiguous().permute(1, 2, 0)
    assert torch.equal(scr.causal_conv(**{**d, "x": t}, activation="silu"), want)
    t = d["x"].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(scr.causal_conv(**{**d, "x": t}, activation="silu"), want)
    out = torch.full((3, 40, 27), NAN, dtype=torch.bfloat16, device=DEV)
    scr.causal_conv(**d, activation="silu", out=out[:, :, 2:26])
    assert torch.equal(out[:, :, 2:26], want)
    assert out[:, :, :2].isnan().all() and out[:, :, 26:].isnan().all()
    one = d["x"][:1].expand(3, 40, 24)
    got = scr.causal_conv(**{**d, "x": one, "state": None})
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("act", [None, "silu"])
def test_unaligned_rows_give_the_same_bits(scr, dtype, K, act):
    s, dy, dfinal = make(2, 90, 136, K, dtype, 13, lengths=[90, 41])
    d = dev(s)

    def off(v):  # the same values, rows that start an element later
        wide = torch.zeros(*v.shape[:-1], v.shape[-1] + 8, dtype=v.dtype, device=DEV)
        wide[..., 1:1 + v.shape[-1]] = v
        return wide[..., 1:1 + v.shape[-1]]

    def results(d, dy):
        y = scr.causal_conv(**d, activation=act)
        return y, scr.causal_conv_backward(dy, **d, activation=act, dfinal=dfinal.to(DEV))

    y, g = results(d, dy.to(DEV))
    y2, g2 = results({**d, "x": off(d["x"])}, off(dy.to(DEV)))
    assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g)


@pytest.mark.parametrize("dtype", TYPES)
def test_parts_give_the_whole(scr, dtype):
    """A sequence cut anywhere, and single tokens, give the bits of one call."""
    s, _, _ = make(2, 90, 20, 4, dtype, 7)
    d = dev(s)
    want, final = scr.causal_conv(**d, activation="silu", return_state=True)
    state, got = d["state"], []
    for a, b in ((0, 1), (1, 3), (3, 70), (70, 90)):
        y, state = scr.causal_conv(d["x"][:, a:b], d["weight"], d["bias"], "silu", state,
                                   return_state=True)
        got.append(y)
    assert torch.equal(torch.cat(got, 1), want) and torch.equal(state, final)
    state = d["state"].clone()
    for t in range(90):
        y = scr.causal_conv_step(d["x"][:, t], state, d["weight"], d["bias"], "silu")
        assert torch.equal(y, want[:, t])
    assert torch.equal(state, final)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,D,K", [(1, 1, 2), (5, 1030, 3), (64, 513, 4)])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_step_slots(scr, dtype, B, D, K, index):
    s, _, _ = make(B, 1, D, K, dtype, 8)
    rows = B + 4
    g = torch.Generator().manual_seed(9)
    pool = torch.randn(rows, K - 1, D, generator=g).to(dtype)
    slots = torch.randperm(rows, generator=g)[:B]
    if B > 2:
        slots[0], slots[2] = -1, rows
    state = pool.to(DEV)
    y = scr.causal_conv_step(s["x"][:, 0].to(DEV), state, s["weight"].to(DEV),
                             s["bias"].to(DEV), "silu", slots=slots.to(index).to(DEV))
    real = [b for b in range(B) if 0 <= slots[b] < rows]
    s["state"] = torch.stack([pool[slots[b]] if b in real else torch.zeros(K - 1, D).to(dtype)
                              for b in range(B)])
    ref = reference(s, "silu")
    if real:
        R.close(y[real], ref["y"][0][real, 0], ref["y"][1][real, 0], FORWARD, "y")
    assert not y[[b for b in range(B) if b not in real]].any()
    want = pool.clone()
    for b in real:
        want[slots[b]] = torch.cat([pool[slots[b]], s["x"][b]])[1:]
    assert torch.equal(state.cpu(), want)


def test_gradients_past_32_bits(scr):
    """Results that begin more than 2^31 elements into their tensors, against a
    call on the last sequence alone."""
    batch, T, D, K = 66, 16384, 2048, 4
    g = torch.Generator(device=DEV).manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    x, dy, w, bias = r(1, T, D), r(1, T, D), r(D, K).float(), r(D).float()

    def whole(v):
        out = torch.zeros(batch, T, D, dtype=v.dtype, device=DEV)
        out[-1:] = v
        return out

    y = scr.causal_conv(whole(x), w, bias, "silu")
    assert y.numel() > 1 << 31
    assert torch.equal(y[-1:], scr.causal_conv(x, w, bias, "silu"))
    del y
    got = scr.causal_conv_backward(whole(dy), whole(x), w, bias, "silu")["x"]
    assert torch.equal(got[-1:], scr.causal_conv_backward(dy, x, w, bias, "silu")["x"])


def test_repeated_calls_give_the_same_bits(scr):
    s, dy, _ = make(2, 300, 260, 4, torch.bfloat16, 10)
    first = scr.causal_conv_backward(dy.to(DEV), **dev(s), activation="silu")
    for _ in range(3):
        again = scr.causal_conv_backward(dy.to(DEV), **dev(s), activation="silu")
        assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_what_no_position_uses(scr, act, K):
    """The state of an empty sequence may hold anything (a slot that no stream
    has): it reaches no gradient. And a position that holds NaN or infinity
    reaches none past its sequence's length."""
    s, dy, dfinal = make(4, 40, 36, K, torch.float32, 11, lengths=[40, 0, 7, 0])
    kinds = dict(activation=act, dfinal=dfinal.to(DEV))
    want = scr.causal_conv_backward(dy.to(DEV), **dev(s), **kinds)
    s["state"][1] = NAN
    s["state"][3, :, ::2], s["state"][3, :, 1::2] = float("inf"), float("-inf")
    g = scr.causal_conv_backward(dy.to(DEV), **dev(s), **kinds)
    for k in g:
        assert torch.equal(g[k], want[k]), k
    y, final = scr.causal_conv(**dev(s), activation=act, return_state=True)
    assert not y[1].any() and not y[3].any() and final[1].isnan().all()
    for bad in (NAN, float("inf"), float("-inf")):
        s["x"][2, 6] = bad
        g = scr.causal_conv_backward(dy.to(DEV), **dev(s), **kinds)
        assert not g["x"][2, 7:].any()
        assert torch.equal(g["x"][0], want["x"][0])
