"""Selective state space scan: forward, gradient and single tokens against a
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
SEQ = ("u", "dt", "z", "B", "C")


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def make(batch, T, D, N, groups, dtype, seed, lengths=None, plain=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = {"u": r(batch, T, D).to(dtype), "dt": (r(batch, T, D) * 0.7 - 1).to(dtype),
         "A": -torch.exp(r(D, N)), "B": r(batch, T, groups, N).to(dtype),
         "C": r(batch, T, groups, N).to(dtype), "D": r(D), "z": r(batch, T, D).to(dtype),
         "dt_bias": r(D) * 0.5 - 1, "state": r(batch, D, N),
         "lengths": None if lengths is None else torch.tensor(lengths)}
    dy, dfinal = r(batch, T, D).to(dtype), r(batch, D, N)
    if plain:
        for k in ("D", "z", "dt_bias", "state"):
            s[k] = None
    if lengths is not None:
        for b, n in enumerate(lengths):
            for k in SEQ:
                if s[k] is not None:
                    s[k][b, max(n, 0):] = NAN
            dy[b, max(n, 0):] = NAN
    return s, dy, dfinal


def dev(s):
    return {k: v if v is None else v.to(DEV) for k, v in s.items()}


def reference(s, softplus=True, dy=None, dfinal=None):
    n = None if s["lengths"] is None else s["lengths"].tolist()
    return R.scan(*(R.f64(s[k]) for k in ("u", "dt", "A", "B", "C", "D", "z", "dt_bias")),
                  softplus, R.f64(s["state"]), n, R.f64(dy), R.f64(dfinal))


def steps(T, N, sums=0):
    """Roundings of a result: up to 8 a time step, the sum over the states, the
    softplus, the gate, and where a result is summed over rows, those."""
    return 8 * T + N + 32 + sums


SHAPES = [(1, 1, 1, 1, 1), (1, 1, 40, 16, 1), (2, 3, 5, 2, 1), (2, 17, 33, 16, 1),
          (1, 70, 260, 16, 1), (2, 37, 66, 13, 2), (1, 33, 40, 8, 4), (1, 40, 24, 32, 1),
          (1, 35, 10, 64, 2), (1, 20, 6, 128, 1), (2, 50, 130, 4, 1), (1, 21, 300, 3, 1),
          (2, 0, 16, 16, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(scr, dtype, shape):
    T, N = shape[1], shape[3]
    s, _, _ = make(*shape, dtype, 1)
    y, final, kept = scr.selective_scan(**dev(s), return_state=True, return_checkpoints=True)
    ref = reference(s)
    R.close(y, *ref["y"], steps(T, N), "y")
    R.close(final, *ref["final"], steps(T, N), "state")
    if T:
        assert torch.equal(kept[:, 0].cpu(), s["state"])
    s, _, _ = make(*shape, dtype, 2, plain=True)
    y, final = scr.selective_scan(**dev(s), return_state=True)
    ref = reference(s)
    R.close(y, *ref["y"], steps(T, N), "plain y")
    R.close(final, *ref["final"], steps(T, N), "plain state")


def check_grads(g, ref, batch, T, D, N, groups):
    for name, v in g.items():
        sums = {"A": batch * T, "D": batch * T, "dt_bias": batch * T, "B": D // groups,
                "C": D // groups}.get(name, 0)
        R.close(v, *ref[name], steps(2 * T, N, sums), name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(scr, dtype, shape):
    s, dy, dfinal = make(*shape, dtype, 3)
    g = scr.selective_scan_backward(dy.to(DEV), **dev(s), dfinal=dfinal.to(DEV))
    assert set(g) == set(s) - {"lengths"}
    check_grads(g, reference(s, True, dy, dfinal)["grads"], *shape)
    s, dy, _ = make(*shape, dtype, 4, plain=True)
    g = scr.selective_scan_backward(dy.to(DEV), **dev(s))
    assert set(g) == {"u", "dt", "A", "B", "C"}
    check_grads(g, reference(s, True, dy)["grads"], *shape)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_without_softplus(scr, dtype):
    s, dy, _ = make(2, 20, 40, 16, 1, dtype, 5)
    s["dt"] = (s["dt"].abs() * 0.1).to(dtype)
    s["dt_bias"] = s["dt_bias"].abs() * 0.1
    ref = reference(s, False, dy)
    R.close(scr.selective_scan(**dev(s), softplus=False), *ref["y"], steps(20, 16), "y")
    g = scr.selective_scan_backward(dy.to(DEV), **dev(s), softplus=False)
    check_grads(g, ref["grads"], 2, 20, 40, 16, 1)


LENGTHS = [[70, 0, 1, 2, 33, 69], [16, 15, 17, 300, -4, 64]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("N,groups", [(16, 1), (5, 2)])
def test_lengths(scr, dtype, lengths, N, groups):
    """What lies past a length is not read (NaN here), gives zeros, and leaves
    the state; an empty sequence returns its state and its gradient as they came."""
    s, dy, dfinal = make(6, 70, 38, N, groups, dtype, 6, lengths=lengths)
    y, final = scr.selective_scan(**dev(s), return_state=True)
    ref = reference(s, True, dy, dfinal)
    R.close(y, *ref["y"], steps(70, N), "y")
    R.close(final, *ref["final"], steps(70, N), "state")
    g = scr.selective_scan_backward(dy.to(DEV), **dev(s), dfinal=dfinal.to(DEV))
    check_grads(g, ref["grads"], 6, 70, 38, N, groups)
    for b, n in enumerate(lengths):
        n = max(0, min(n, 70))
        assert not y[b, n:].any()
        assert not any(g[k][b, n:].any() for k in SEQ)
        if n == 0:
            assert torch.equal(final[b].cpu(), s["state"][b])
            assert torch.equal(g["state"][b].cpu(), dfinal[b])


def test_gradient_matches_differences(scr):
    """The gradient's product with a direction against central differences of
    the 64-bit formula: their error is eps^2 / 6 of the third derivative, which
    eps = 1e-4 takes far below the gradient's own binary32 rounding."""
    s, dy, dfinal = make(2, 9, 6, 5, 2, torch.float32, 7)
    g = scr.selective_scan_backward(dy.to(DEV), **dev(s), dfinal=dfinal.to(DEV))
    gen = torch.Generator().manual_seed(8)
    for name in g:
        v = torch.randn(s[name].shape, generator=gen, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            m = {k: R.f64(t) for k, t in s.items()}
            m[name] = m[name] + sign * 1e-4 * v.numpy()
            ref = R.scan(*(m[k] for k in ("u", "dt", "A", "B", "C", "D", "z", "dt_bias")), True,
                         m["state"], None)
            ends.append((ref["y"][0] * R.f64(dy)).sum() + (ref["final"][0] * R.f64(dfinal)).sum())
        want = (ends[0] - ends[1]) / 2e-4
        got = (R.f64(g[name]) * v.numpy()).sum()
        size = (np.abs(R.f64(g[name])) * np.abs(v.numpy())).sum()
        assert abs(got - want) <= 1e-5 * size, name


def test_extreme_steps(scr):
    """Steps so small that the softplus is its exponential, and so large that
    the decay underflows to zero."""
    s, dy, _ = make(1, 30, 16, 16, 1, torch.float32, 9)
    s["dt"][0, :, :4] = -30.0
    s["dt"][0, :, 4:8] = 60.0
    s["dt"][0, ::3, 8:12] = 200.0
    s["z"][0, :, 2] = -200.0
    s["z"][0, :, 3] = 200.0
    ref = reference(s, True, dy)
    R.close(scr.selective_scan(**dev(s)), *ref["y"], steps(30, 16), "y")
    check_grads(scr.selective_scan_backward(dy.to(DEV), **dev(s)), ref["grads"], 1, 30, 16, 16, 1)


def test_strides_and_alignment(scr):
    """The same bits from strided, misaligned and transposed inputs, and from
    B and C without a group axis."""
    s, dy, _ = make(3, 40, 24, 16, 1, torch.bfloat16, 10)
    d = dev(s)
    want = scr.selective_scan(**d)
    gwant = scr.selective_scan_backward(dy.to(DEV), **d)
    def same(**changed):
        m = {**d, **changed}
        assert torch.equal(scr.selective_scan(**m), want)
        g = scr.selective_scan_backward(dy.to(DEV), **m)
        assert all(torch.equal(g[k].view_as(gwant[k]), gwant[k]) for k in g)
    for at in (5, 8):
        wide = torch.full((3, 40, 24 * 3 + 16), NAN, dtype=torch.bfloat16, device=DEV)
        views = {}
        for i, k in enumerate(("u", "dt", "z")):
            views[k] = wide[:, :, at + 24 * i:at + 24 * (i + 1)]
            views[k].copy_(d[k])
        same(**views)
    same(u=d["u"].permute(2, 0, 1).contiguous().permute(1, 2, 0))
    same(z=d["z"].transpose(0, 1).contiguous().transpose(0, 1))
    both = torch.cat([d["B"], d["C"]], 3)
    same(B=both[..., :16], C=both[..., 16:])
    same(B=both[..., :16].squeeze(2), C=both[..., 16:].squeeze(2))
    odd = torch.zeros(3, 40, 1, 19, dtype=torch.bfloat16, device=DEV)
    odd[..., 3:] = d["B"]
    same(B=odd[..., 3:])
    same(A=d["A"].t().contiguous().t())
    out = torch.full((3, 40, 27), NAN, dtype=torch.bfloat16, device=DEV)
    scr.selective_scan(**d, out=out[:, :, 2:26])
    assert torch.equal(out[:, :, 2:26], want)
    assert out[:, :, :2].isnan().all() and out[:, :, 26:].isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [4, 8, 16, 32, 64, 128])
def test_unaligned_rows_give_the_same_bits(scr, dtype, N):
    """Whole accesses and elementwise ones, for every number of lanes a channel:
    forward, gradients and single tokens."""
    s, dy, dfinal = make(2, 37, 72, N, 1, dtype, 26)
    d = {**dev(s), "dy": dy.to(DEV)}

    def off(v):  # the same values, rows that start an element later
        wide = torch.zeros(*v.shape[:-1], v.shape[-1] + 8, dtype=v.dtype, device=DEV)
        wide[..., 1:1 + v.shape[-1]] = v
        return wide[..., 1:1 + v.shape[-1]]

    def results(d):
        dy, rest = d["dy"], {k: v for k, v in d.items() if k != "dy"}
        y, final = scr.selective_scan(**rest, return_state=True)
        g = scr.selective_scan_backward(dy, **rest, dfinal=dfinal.to(DEV))
        state = rest["state"].clone()
        one = scr.selective_scan_step(rest["u"][:, 0], rest["dt"][:, 0], rest["A"],
                                      rest["B"][:, 0], rest["C"][:, 0], state, rest["D"],
                                      rest["z"][:, 0], rest["dt_bias"])
        return {"y": y, "final": final, "one": one, "after": state,
                **{"d" + k: v for k, v in g.items()}}

    want = results(d)
    B, C = off(d["B"].squeeze(2)), off(d["C"].squeeze(2))
    got = results({**d, **{k: off(d[k]) for k in ("u", "dt", "z", "dy")}, "B": B, "C": C})
    for k in want:
        assert torch.equal(got[k].view(want[k].shape), want[k]), k


@pytest.mark.parametrize("N", [1, 4, 8, 16, 32, 64, 128])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("T", [1, 16])
def test_sums_over_channels_are_of_rounded_products(scr, N, off, T):
    """One step of two channels, whichever two, alone or the last of a whole tile:
    dB and dC are the rounded sums of two rounded products, to the bit. (Joined
    into one rounding they would depend on how the compiler has arranged a variant
    of the kernel.)"""
    D, last = 64, T - 1
    g = torch.Generator().manual_seed(27)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    u, dy = torch.zeros(D - 1, T, D), torch.zeros(D - 1, T, D)
    for j in range(1, D):
        for v in (u, dy):
            v[j - 1, last, 0], v[j - 1, last, j] = r(1), r(1)
    B, C = r(D - 1, T, N), r(D - 1, T, N)
    wide = torch.zeros(D - 1, T, D + 4, device=DEV)
    wide[..., off:off + D] = u.to(DEV)
    got = scr.selective_scan_backward(dy.to(DEV), wide[..., off:off + D],
                                      torch.ones(D - 1, T, D, device=DEV), -r(D, N).abs().to(DEV),
                                      B.to(DEV), C.to(DEV), softplus=False)
    u, dy, B, C = u.numpy(), dy.numpy(), B.numpy(), C.numpy()
    for j in range(1, D):
        two = [(dy[j - 1, last, d], u[j - 1, last, d]) for d in (0, j)]
        b, c = B[j - 1, last], C[j - 1, last]
        dB = [(c * y) * x for y, x in two]
        dC = [y * (x * b) for y, x in two]
        assert np.array_equal(got["B"][j - 1, last].cpu().numpy(), dB[0] + dB[1]), j
        assert np.array_equal(got["C"][j - 1, last].cpu().numpy(), dC[0] + dC[1]), j
    assert not got["B"][:, :last].any() and not got["C"][:, :last].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_single_tokens(scr, dtype):
    """Single tokens after a prompt: within the roundings of the formula of
    the whole sequence."""
    s, _, _ = make(2, 24, 36, 16, 1, dtype, 11)
    d = dev(s)
    ref = reference(s)
    cut = {k: (v[:, :20] if k in SEQ else v) for k, v in d.items()}
    y, state = scr.selective_scan(**cut, return_state=True)
    R.close(y, ref["y"][0][:, :20], ref["y"][1][:, :20], steps(20, 16), "prompt")
    for t in range(20, 24):
        y = scr.selective_scan_step(d["u"][:, t], d["dt"][:, t], d["A"], d["B"][:, t],
                                    d["C"][:, t], state, d["D"], d["z"][:, t], d["dt_bias"])
        R.close(y, ref["y"][0][:, t], ref["y"][1][:, t], steps(t + 1, 16), "token %d" % t)
    R.close(state, *ref["final"], steps(24, 16), "state")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,D,N,groups", [(1, 1, 1, 1), (5, 70, 16, 1), (64, 130, 13, 2),
                                              (3, 40, 64, 1), (3, 9, 128, 1)])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_step_slots(scr, dtype, batch, D, N, groups, index):
    s, _, _ = make(batch, 1, D, N, groups, dtype, 12)
    rows = batch + 4
    g = torch.Generator().manual_seed(13)
    pool = torch.randn(rows, D, N, generator=g)
    slots = torch.randperm(rows, generator=g)[:batch]
    if batch > 2:
        slots[0], slots[2] = -1, rows
    state = pool.to(DEV)
    one = {k: s[k][:, 0].to(DEV) for k in SEQ}
    y = scr.selective_scan_step(one["u"], one["dt"], s["A"].to(DEV), one["B"], one["C"], state,
                                s["D"].to(DEV), one["z"], s["dt_bias"].to(DEV),
                                slots=slots.to(index).to(DEV))
    real = [b for b in range(batch) if 0 <= slots[b] < rows]
    none = [b for b in range(batch) if b not in real]
    s["state"] = torch.stack([pool[slots[b]] if b in real else torch.zeros(D, N)
                              for b in range(batch)])
    ref = reference(s)
    if real:
        R.close(y[real], ref["y"][0][real, 0], ref["y"][1][real, 0], steps(1, N), "y")
        at = [int(slots[b]) for b in real]
        R.close(state[at], ref["final"][0][real], ref["final"][1][real], steps(1, N), "state")
    assert not y[none].any()
    left = [r for r in range(rows) if r not in [int(slots[b]) for b in real]]
    assert torch.equal(state[left].cpu(), pool[left])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,N,groups", [(36, 16, 1), (70, 13, 2), (9, 1, 1), (33, 8, 3), (10, 64, 2),
                                        (5, 128, 1)])
def test_steps_give_the_bits_of_a_prompt(scr, dtype, D, N, groups):
    """Sequences short enough not to be cut: one call, two calls and single tokens
    evaluate the same expression."""
    s, _, _ = make(2, 60, D, N, groups, dtype, 21)
    d = dev(s)
    want, last = scr.selective_scan(**d, return_state=True)
    cut = {k: (v[:, :23] if k in SEQ else v) for k, v in d.items()}
    y, state = scr.selective_scan(**cut, return_state=True)
    assert torch.equal(y, want[:, :23])
    rest = {**{k: (v[:, 23:] if k in SEQ else v) for k, v in d.items()}, "state": state}
    y, end = scr.selective_scan(**rest, return_state=True)
    assert torch.equal(y, want[:, 23:]) and torch.equal(end, last)
    for t in range(23, 60):
        y = scr.selective_scan_step(d["u"][:, t], d["dt"][:, t], d["A"], d["B"][:, t],
                                    d["C"][:, t], state, d["D"], d["z"][:, t], d["dt_bias"])
        assert torch.equal(y, want[:, t]), t
    assert torch.equal(state, last)


@pytest.mark.parametrize("batch", [1, 800])
def test_long_sequence_that_forgets(scr, batch):
    """Decays of at most e^-0.5 keep an error for 1 / (1 - e^-0.5) = 2.6 steps, so
    that thousands of steps leave no more than tens of roundings: 8 a step for
    2.6 steps, the sums over the states and the outputs', with room to 64. Cut into
    segments (one sequence) and whole (800 of them)."""
    T, D, N = 2500 if batch == 1 else 300, 8, 16
    s, dy, dfinal = make(1, T, D, N, 1, torch.float32, 22)
    s["dt"] = s["dt"].abs().clamp(max=0.5) + 0.5
    s["A"] = -1 - torch.rand(D, N, generator=torch.Generator().manual_seed(23))
    s["dt_bias"] = torch.zeros(D)
    ref = reference(s, False, dy, dfinal)
    many = {k: v if v is None or k in ("A", "D", "dt_bias") else
            v.expand(batch, *v.shape[1:]) for k, v in s.items()}
    y, final = scr.selective_scan(**dev(many), softplus=False, return_state=True)
    R.close(y[:1], *ref["y"], 64, "y")
    R.close(final[:1], *ref["final"], 64, "state")
    assert torch.equal(y[0].expand_as(y), y) and torch.equal(final[0].expand_as(final), final)
    if batch == 1:
        g = scr.selective_scan_backward(dy.to(DEV), **dev(s), softplus=False,
                                        dfinal=dfinal.to(DEV))
        for k in ("u", "dt", "z", "B", "C", "state"):
            R.close(g[k], *ref["grads"][k], 2 * 64 + (D if k in ("B", "C") else 0), k)


def test_long_sequence(scr):
    """Thousands of steps, a few channels."""
    s, dy, _ = make(1, 2500, 8, 16, 1, torch.float32, 14)
    ref = reference(s, True, dy)
    R.close(scr.selective_scan(**dev(s)), *ref["y"], steps(2500, 16), "y")
    check_grads(scr.selective_scan_backward(dy.to(DEV), **dev(s)), ref["grads"], 1, 2500, 8, 16, 1)


@pytest.mark.parametrize("rate,state,first", [(1.2, 0.0, 4950), (-1.2, 1e30, 0), (1.0, 1e-30, 0)])
def test_segments_that_grow_or_decay_far(scr, rate, state, first):
    """A segment's whole growth or decay may lie outside binary32's range where
    the states themselves do not: 5000 steps in segments of 96, with inputs from
    step `first` on (none: the state alone, as far as it stays normal)."""
    T, D = 5000, 8
    f32 = dict(dtype=torch.float32, device=DEV)
    u = torch.zeros(1, T, D, **f32)
    if first:
        u[:, first:] = 1.0
    one = torch.ones(1, T, 1, **f32)
    y, final = scr.selective_scan(u, torch.ones(1, T, D, **f32), torch.full((D, 1), rate, **f32),
                                  one, one, softplus=False, return_state=True,
                                  state=torch.full((1, D, 1), state, **f32))
    a, h, want = float(np.exp(np.float64(np.float32(rate)))), float(np.float32(state)), []
    for t in range(T):
        h = a * h + float(u[0, t, 0])
        want.append(h)
    want = np.array(want)
    n = T if first else int(np.argmax((np.abs(want) < 2.0 ** -120) | (np.abs(want) > 2.0 ** 120)))
    assert n > 120
    got = R.f64(y)[0, :n]
    # a step's decay: 1.4e-7 of the instruction, 2^-23 |log2 a| of its argument;
    # one rounding of the product and one of the sum; a factor 2 of room
    step = 2 * (1.4e-7 + 2.0 ** -23 * (abs(rate) * 1.4427 + 1))
    off = np.abs(got - want[:n, None])
    assert (off <= step * np.arange(1, n + 1)[:, None] * np.abs(want[:n, None])).all()


def test_no_channels(scr):
    """Without channels the gradients of B and C, which then reach nothing, are
    zero, whatever their memory held."""
    import ctypes

    from scan_canonical_reduce_gb300 import model as m
    s, dy, dfinal = make(2, 37, 0, 16, 2, torch.bfloat16, 18)
    y, final = scr.selective_scan(**dev(s), return_state=True)
    assert y.shape == (2, 37, 0) and final.shape == (2, 0, 16)
    g = scr.selective_scan_backward(dy.to(DEV), **dev(s), dfinal=dfinal.to(DEV))
    assert g["B"].shape == g["C"].shape == (2, 37, 2, 16)
    assert all(not v.any() for v in g.values())
    B, C = s["B"].to(DEV), s["C"].to(DEV)
    dB, dC = torch.full_like(B, 3.0), torch.full_like(C, 3.0)
    sizes = dict(batch=2, len=37, dim=0, dstate=16, groups=2, softplus=1, dt_type=3,
                 B=B.data_ptr(), B_batch_stride=37 * 32, B_time_stride=32, C=C.data_ptr(),
                 C_batch_stride=37 * 32, C_time_stride=32)
    args = m._ScanArgs(**sizes)
    grads = m._ScanGrads(dB=dB.data_ptr(), dC=dC.data_ptr())
    n = scr.lib().cr_selective_scan_backward_workspace_bytes(2, 37, 0, 16, 2)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream(DEV).cuda_stream
    assert scr.lib().cr_selective_scan_backward(ctypes.byref(args), ctypes.byref(grads),
                                                ws.data_ptr(), n, stream) == 0
    assert not dB.any() and not dC.any()


def test_repeated_calls_give_the_same_bits(scr):
    s, dy, _ = make(2, 300, 260, 16, 1, torch.bfloat16, 15)
    d = dev(s)
    y, kept = scr.selective_scan(**d, return_checkpoints=True)
    first = scr.selective_scan_backward(dy.to(DEV), **d, checkpoints=kept)
    again = scr.selective_scan_backward(dy.to(DEV), **d)  # computes its own checkpoints
    assert all(torch.equal(first[k], again[k]) for k in first)
    for _ in range(3):
        assert torch.equal(scr.selective_scan(**d), y)
        again = scr.selective_scan_backward(dy.to(DEV), **d, checkpoints=kept)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_overflow_stays_in_its_sequence(scr):
    """A state that has overflowed: positions past the length still give zeros,
    and the other sequences what they give without it."""
    s, dy, _ = make(3, 40, 24, 16, 1, torch.float32, 16, lengths=[40, 21, 33])
    want = scr.selective_scan(**dev(s))
    gwant = scr.selective_scan_backward(dy.to(DEV), **dev(s))
    s["u"][1, 5] = float("inf")
    y, final = scr.selective_scan(**dev(s), return_state=True)
    g = scr.selective_scan_backward(dy.to(DEV), **dev(s))
    assert not torch.isfinite(final[1]).all()
    for b in (0, 2):
        assert torch.equal(y[b], want[b])
        assert all(torch.equal(g[k][b], gwant[k][b]) for k in SEQ + ("state",))
    assert not y[1, 21:].any()
    assert not any(g[k][1, 21:].any() for k in SEQ)


@pytest.mark.parametrize("T", [20, 33, 47])
@pytest.mark.parametrize("N", [4, 16, 64])
def test_overflow_in_the_last_step(scr, T, N):
    """A state that overflows in the last step is part of no decay's gradient:
    that of A is what it is without the overflow."""
    s, dy, dfinal = make(1, T, 24, N, 1, torch.float32, 19)
    want = scr.selective_scan_backward(dy.to(DEV), **dev(s), dfinal=dfinal.to(DEV))
    s["u"][0, T - 1] = 3e38
    s["B"][0, T - 1] = 3e38
    _, final = scr.selective_scan(**dev(s), return_state=True)
    assert final.isinf().all()
    g = scr.selective_scan_backward(dy.to(DEV), **dev(s), dfinal=dfinal.to(DEV))
    assert torch.equal(g["A"], want["A"])


@pytest.mark.parametrize("shape", [(1, 40, 40, 16, 1), (2, 33, 66, 16, 2), (1, 40, 33, 4, 1),
                                   (1, 20, 9, 64, 1)])
def test_channels_that_grow(scr, shape):
    """A channel with a growth of its own, at steps so small that its states stay
    as they are: lanes that have no channel do not take it further."""
    s, dy, dfinal = make(*shape, torch.float32, 20)
    s["A"] = s["A"].abs() + 9
    s["dt_bias"] -= 20
    g = scr.selective_scan_backward(dy.to(DEV), **dev(s), dfinal=dfinal.to(DEV))
    check_grads(g, reference(s, True, dy, dfinal)["grads"], *shape)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(2, 35, 130, 33, 1), (1, 50, 200, 64, 2), (2, 19, 70, 100, 1),
                                   (1, 33, 96, 128, 3)])
def test_backward_of_many_states(scr, dtype, shape):
    """More than 32 states and more channels than a block has."""
    s, dy, dfinal = make(*shape, dtype, 24, lengths=[shape[1], 18][:shape[0]])
    g = scr.selective_scan_backward(dy.to(DEV), **dev(s), dfinal=dfinal.to(DEV))
    check_grads(g, reference(s, True, dy, dfinal)["grads"], *shape)


def test_gradients_past_32_bits(scr):
    """Results that begin more than 2^31 elements into their tensors, against a
    call on the last sequences alone (enough of them not to be cut)."""
    batch, T, D, N = 66, 16384, 2048, 4
    g = torch.Generator(device=DEV).manual_seed(25)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    last = {k: r(12, T, D) for k in ("u", "dt", "z")}
    last.update({k: r(12, T, 1, N) for k in ("B", "C")})
    dy = r(12, T, D)

    def whole(v):
        out = torch.zeros(batch, *v.shape[1:], dtype=v.dtype, device=DEV)
        out[-12:] = v
        return out

    rest = {"A": -torch.exp(r(D, N).float()), "D": r(D).float(), "dt_bias": r(D).float() - 3}
    y, final = scr.selective_scan(**{k: whole(v) for k, v in last.items()}, **rest,
                                  return_state=True)
    assert y.numel() > 1 << 31
    want, want_final = scr.selective_scan(**last, **rest, return_state=True)
    assert torch.equal(y[-12:], want) and torch.equal(final[-12:], want_final)
    del y
    want = scr.selective_scan_backward(dy, **last, **rest)
    got = scr.selective_scan_backward(whole(dy), **{k: whole(v) for k, v in last.items()}, **rest)
    for k in SEQ:
        assert torch.equal(got[k][-12:], want[k]), k


# few states: the gradient shares a channel among one, two or four lanes,
# by how many channels there are
MANY = [(2, 19, 20000, 4, 1), (2, 17, 20010, 3, 3), (2, 33, 5002, 8, 1), (1, 20, 5001, 7, 1),
        (1, 20, 10000, 4, 1), (1, 34, 1032, 4, 1), (3, 18, 501, 6, 3)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", MANY)
def test_backward_of_few_states(scr, dtype, shape):
    batch, T = shape[:2]
    lengths = [T, T // 2, 0][:batch]
    s, dy, dfinal = make(*shape, dtype, 17, lengths=lengths)
    g = scr.selective_scan_backward(dy.to(DEV), **dev(s), dfinal=dfinal.to(DEV))
    check_grads(g, reference(s, True, dy, dfinal)["grads"], *shape)
    for b, n in enumerate(lengths):
        assert not any(g[k][b, n:].any() for k in SEQ)
