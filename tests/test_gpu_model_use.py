"""The model operators as programs use them: on other streams, in CUDA graphs,
from several threads, with buffers of exactly their size, with offsets past
32 bits, and together in a small language model."""
import ctypes
import os
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def inputs(seed, batch=3, T=150, D=200, N=16, K=4, V=500, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = {"tokens": torch.randint(0, V, (batch, T), generator=g), "table": r(V, D).to(dtype),
         "x": r(batch, T, D).to(dtype), "dt": (r(batch, T, D) - 2).to(dtype),
         "z": r(batch, T, D).to(dtype), "B": r(batch, T, N).to(dtype),
         "C": r(batch, T, N).to(dtype), "A": -torch.exp(r(D, N)), "D": r(D), "dt_bias": r(D),
         "weight": r(D, K), "bias": r(D), "conv": r(batch, K - 1, D).to(dtype),
         "scan": r(batch, D, N), "dy": r(batch, T, D).to(dtype)}
    return {k: v.to(DEV) for k, v in t.items()}


def calls(scr, t, stream=None):
    """Every operator once, on t; {name: result}."""
    s = dict(stream=stream)
    scan = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"])
    main = (t["x"], t["dt"], t["A"], t["B"], t["C"])
    out = {"embedding": scr.embedding(t["tokens"], t["table"], 2.0, **s),
           "embedding_backward": scr.embedding_backward(t["tokens"], t["dy"], t["table"].shape[0],
                                                        2.0, **s)}
    conv = dict(activation="silu", state=t["conv"], **s)
    out["conv"], out["conv_state"] = scr.causal_conv(t["x"], t["weight"], t["bias"],
                                                     return_state=True, **conv)
    for k, v in scr.causal_conv_backward(t["dy"], t["x"], t["weight"], t["bias"], **conv).items():
        out["conv_d" + k] = v
    out["scan"], out["scan_state"], kept = scr.selective_scan(
        *main, state=t["scan"], return_state=True, return_checkpoints=True, **scan, **s)
    for k, v in scr.selective_scan_backward(t["dy"], *main, state=t["scan"], checkpoints=kept,
                                            **scan, **s).items():
        out["scan_d" + k] = v
    out["conv_step"] = scr.causal_conv_step(t["x"][:, 0], t["conv"], t["weight"], t["bias"],
                                            "silu", **s)
    one = {k: t[k][:, 0] for k in ("x", "dt", "z", "B", "C")}
    out["scan_step"] = scr.selective_scan_step(one["x"], one["dt"], t["A"], one["B"], one["C"],
                                               t["scan"], t["D"], one["z"], t["dt_bias"], **s)
    out["conv_after"], out["scan_after"] = t["conv"], t["scan"]
    return out


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a) and set(a) == set(b)


def test_other_streams(scr):
    """On a stream that is still busy when the call returns, with the inputs
    dropped and their memory asked for again at once."""
    want = calls(scr, inputs(1))
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    t = inputs(1)
    s.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # some milliseconds
    got = calls(scr, t, s)
    shapes = [(v.shape, v.dtype) for k, v in t.items() if k not in ("conv", "scan")]
    got.pop("conv_after"), got.pop("scan_after")
    del t
    junk = [torch.full(shape, 77, dtype=dtype, device=DEV) for shape, dtype in shapes * 2]
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in got)
    del junk


def test_other_streams_copy_inputs(scr):
    """Inputs that the calls copy, as their layout is not one that they take: what
    the copy reads stays the caller's until the busy stream has come to it."""
    def turned(v):  # the same values, the last axis not contiguous
        return v.transpose(0, -1).contiguous().transpose(0, -1)

    def spread(v):  # every second element of a longer tensor
        return torch.stack([v, v], -1)[..., 0]

    def run(stream):
        t = inputs(21)
        u = {k: turned(t[k]) for k in ("table", "x", "dt", "z", "B", "C", "A", "weight", "conv",
                                       "scan", "dy")}
        u.update({k: spread(t[k]) for k in ("tokens", "D", "dt_bias", "bias")})
        lengths = spread(torch.tensor([150, 3, 77], device=DEV))
        rows = t["x"][0, :1].clone()
        pools = t["conv"].clone(), t["scan"].clone()
        slots = spread(torch.tensor([2, 0, 1], device=DEV))
        dfinal = turned(t["scan"]), turned(t["conv"])
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream(DEV))
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)
        k = dict(stream=stream)
        out = [scr.embedding(u["tokens"], u["table"], 2.0, **k),
               scr.embedding(u["tokens"], rows.expand(500, 200), **k),
               scr.embedding_backward(u["tokens"], u["dy"], 500, **k),
               scr.embedding_backward(u["tokens"], rows[:, None].expand(3, 150, 200), 500, **k)]
        conv = dict(activation="silu", state=u["conv"], lengths=lengths, **k)
        out += scr.causal_conv(u["x"], u["weight"], u["bias"], return_state=True, **conv)
        out += scr.causal_conv_backward(u["dy"], u["x"], u["weight"], u["bias"], dfinal=dfinal[1],
                                        **conv).values()
        scan = dict(D=u["D"], z=u["z"], dt_bias=u["dt_bias"], **k)
        main = (u["x"], u["dt"], u["A"], u["B"], u["C"])
        out += scr.selective_scan(*main, state=u["scan"], lengths=lengths, return_state=True,
                                  **scan)
        out += scr.selective_scan_backward(u["dy"], *main, state=u["scan"], lengths=lengths,
                                           dfinal=dfinal[0], **scan).values()
        one = {n: u[n][:, 0] for n in ("x", "dt", "z", "B", "C")}
        out.append(scr.causal_conv_step(one["x"], pools[0], u["weight"], u["bias"], "silu", slots,
                                        **k))
        out.append(scr.selective_scan_step(one["x"], one["dt"], u["A"], one["B"], one["C"],
                                           pools[1], u["D"], one["z"], u["dt_bias"], slots=slots,
                                           **k))
        held = list(u.values()) + [lengths, rows, slots, *dfinal]
        return out, [(v.shape, v.dtype) for v in held]

    want, _ = run(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    got, shapes = run(s)  # every input is dropped here, its memory asked for again at once
    junk = [torch.full(shape, 77, dtype=dtype, device=DEV) for shape, dtype in shapes * 3]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))
    del junk


def test_graph_replay(scr):
    """Captured once, replayed on new contents of the same buffers."""
    t = inputs(2)
    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(s):
        calls(scr, t)  # the workspace exists before the capture
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = calls(scr, t)
    for seed in (3, 4):
        new = inputs(seed)
        for k in t:
            t[k].copy_(new[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, calls(scr, new)), seed


# calls whose scratch memory a captured graph has to keep
def scratch_calls(scr, t):
    main = (t["x"], t["dt"], t["A"], t["B"], t["C"])
    y, kept = scr.selective_scan(*main, return_checkpoints=True)
    out = {"y": y, "dW": scr.embedding_backward(t["tokens"], t["dy"], 500)}
    out.update({"conv_" + k: v for k, v in scr.causal_conv_backward(
        t["dy"], t["x"], t["weight"], t["bias"], "silu").items()})
    out.update(scr.selective_scan_backward(t["dy"], *main, checkpoints=kept))
    return out


def captured(scr, t, s):
    s.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(s):
        scratch_calls(scr, t)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = scratch_calls(scr, t)
    return graph, got


def test_graph_replay_after_larger_calls(scr):
    """A graph's scratch memory is not given to tensors that are made after a
    larger call on its stream, nor do they lose what they hold to a replay."""
    t = inputs(22, T=400)  # a scan of seven segments
    want = scratch_calls(scr, t)
    s = torch.cuda.Stream(DEV)
    graph, got = captured(scr, t, s)
    with torch.cuda.stream(s):
        scratch_calls(scr, inputs(23, batch=8, T=900, D=520, V=5000))
        s.synchronize()
        held = [torch.full((1 << k,), 7, dtype=torch.uint8, device=DEV)
                for k in (12, 16, 18, 20, 22, 24) for _ in range(8)]
    torch.cuda.synchronize()
    for v in got.values():
        v.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, want)
    assert all(bool((h == 7).all()) for h in held)


def test_graphs_of_one_stream_replayed_on_two(scr):
    t = [inputs(24, T=400), inputs(25, T=420)]
    want = [scratch_calls(scr, x) for x in t]
    s = torch.cuda.Stream(DEV)
    graphs = [captured(scr, x, s) for x in t]
    streams = [torch.cuda.Stream(DEV) for _ in t]
    for _ in range(20):
        for _, got in graphs:
            for v in got.values():
                v.zero_()
        torch.cuda.synchronize()
        for (graph, _), on in zip(graphs, streams):
            with torch.cuda.stream(on):
                graph.replay()
        torch.cuda.synchronize()
        assert all(same(got, w) for (_, got), w in zip(graphs, want))


def test_threads_on_their_own_streams(scr):
    want = {seed: calls(scr, inputs(seed)) for seed in range(10, 14)}
    torch.cuda.synchronize()
    bad = []

    def work(seed):
        s = torch.cuda.Stream(DEV)
        with torch.cuda.stream(s):
            for _ in range(5):
                t = inputs(seed)
                got = calls(scr, t)
                s.synchronize()
                if not same(got, want[seed]):
                    bad.append(seed)

    threads = [threading.Thread(target=work, args=(seed,)) for seed in want]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad


def test_launches_are_counted_and_named(scr):
    t, many = inputs(5), inputs(5, T=900)  # the gradient of the lookup: few tokens, and many
    calls(scr, t)
    calls(scr, many)
    before = scr.launch_count()
    scr.profile_enable(True)
    scr.profile_collect()
    calls(scr, t)
    calls(scr, many)
    torch.cuda.synchronize()
    records = scr.profile_collect()
    scr.profile_enable(False)
    assert scr.launch_count() - before == len(records)
    names = {n for n, _ in records}
    assert "embedding_few_kernel" in names
    assert {"embedding_kernel", "token_sort_kernel", "embedding_rows_kernel", "causal_conv_kernel",
            "causal_conv_backward_kernel", "causal_conv_step_kernel", "selective_scan_kernel",
            "selective_scan_backward_kernel", "selective_scan_step_kernel"} <= names


def test_status_word_is_left_alone(scr):
    """The model operators share the binding's workspace with calls that keep a
    status word in it: what sync_status reports is those calls' own."""
    s = torch.cuda.Stream(DEV)
    with torch.cuda.stream(s):
        t = inputs(15)
        calls(scr, t)
        scr.sync_status(DEV, s)  # a workspace that no other call has used
        x = torch.rand(5000, dtype=torch.float64, device=DEV)
        scr.inclusive_scan(x, "iterated_pairwise", stream=s)
        calls(scr, t)
        scr.sync_status(DEV, s)
        scr.lib().cr_debug_skip_publish(2)
        try:
            scr.inclusive_scan(torch.rand(2048 * 16 + 5, dtype=torch.float64, device=DEV),
                               "iterated_pairwise", stream=s)
            s.synchronize()
        finally:
            scr.lib().cr_debug_skip_publish(-1)
        scr.embedding_backward(t["tokens"], t["dy"], 500)
        with pytest.raises(scr.CrError):  # that call's wait gave up, and still says so
            scr.sync_status(DEV, s)


class Guarded:
    """Device bytes between bands that must keep their pattern."""
    BAND = 1 << 14

    def __init__(self, values=None, nbytes=0):
        n = values.numel() * values.element_size() if values is not None else nbytes
        self.n = n
        self.buf = torch.full((2 * self.BAND + n,), 0xFF if values is not None else 0xA5,
                              dtype=torch.uint8, device=DEV)
        self.ptr = self.buf.data_ptr() + self.BAND
        if values is not None:
            self.buf[self.BAND:self.BAND + n] = values.contiguous().view(torch.uint8).flatten()
        self.fill = int(self.buf[0])

    def view(self, dtype, shape):
        return self.buf[self.BAND:self.BAND + self.n].view(dtype).view(shape)

    def intact(self):
        return bool((self.buf[:self.BAND] == self.fill).all()) and \
            bool((self.buf[self.BAND + self.n:] == self.fill).all())


@pytest.mark.parametrize("D", [200, 77])
def test_buffers_of_exact_size(scr, D):
    """Through the C ABI: inputs between NaN bands, outputs and workspaces of
    exactly their size between canaries, which stay as they were."""
    from scan_canonical_reduce_gb300 import model as m
    L = scr.lib()
    t = inputs(6, D=D)
    want = calls(scr, {k: v.clone() for k, v in t.items()})
    batch, T, N, K, V = 3, 150, 16, 4, 500
    stream = torch.cuda.current_stream(DEV).cuda_stream
    g = {k: Guarded(v) for k, v in t.items()}
    bands, outs = list(g.values()), {}

    def out(name, like):
        outs[name] = (Guarded(nbytes=like.numel() * like.element_size()), like)
        bands.append(outs[name][0])
        return outs[name][0].ptr

    def ws(n):
        bands.append(Guarded(nbytes=n))
        return bands[-1].ptr, n

    rows = batch * T
    assert L.cr_embedding(g["tokens"].ptr, 8, rows, g["table"].ptr, V, D, D, 2.0, 3,
                          out("embedding", want["embedding"]), D, stream) == 0
    assert L.cr_embedding_backward(
        g["tokens"].ptr, 8, rows, g["dy"].ptr, D, V, D, 2.0, 3, 0,
        out("embedding_backward", want["embedding_backward"]), D,
        *ws(L.cr_embedding_backward_workspace_bytes(rows, V, D)), stream) == 0
    ca = m._ConvArgs(batch, T, D, K, 1, 3, 4, g["x"].ptr, T * D, D, g["weight"].ptr,
                     g["bias"].ptr, g["conv"].ptr, None)
    assert L.cr_causal_conv(ctypes.byref(ca), out("conv", want["conv"]), T * D, D,
                            out("conv_state", want["conv_state"]), stream) == 0
    cg = m._ConvGrads(g["dy"].ptr, T * D, D, None, out("conv_dx", want["conv_dx"]), T * D, D,
                      out("conv_dweight", want["conv_dweight"]),
                      out("conv_dbias", want["conv_dbias"]),
                      out("conv_dstate", want["conv_dstate"]))
    assert L.cr_causal_conv_backward(
        ctypes.byref(ca), ctypes.byref(cg),
        *ws(L.cr_causal_conv_backward_workspace_bytes(batch, T, D, K)), stream) == 0
    sa = m._ScanArgs(batch, T, D, N, 1, 1, 3, 4, 0, g["x"].ptr, T * D, D, g["dt"].ptr, T * D, D,
                     g["z"].ptr, T * D, D, g["B"].ptr, T * N, N, g["C"].ptr, T * N, N, g["A"].ptr,
                     g["D"].ptr, g["dt_bias"].ptr, g["scan"].ptr, None)
    n_check = L.cr_selective_scan_checkpoints(T)
    kept = Guarded(nbytes=batch * n_check * D * N * 4)
    bands.append(kept)
    assert L.cr_selective_scan(
        ctypes.byref(sa), out("scan", want["scan"]), T * D, D,
        out("scan_state", want["scan_state"]), kept.ptr,
        *ws(L.cr_selective_scan_workspace_bytes(batch, T, D, N)), stream) == 0
    sg = m._ScanGrads(g["dy"].ptr, T * D, D, None, kept.ptr,
                      *(out("scan_d" + k, want["scan_d" + k])
                        for k in ("u", "dt", "z", "B", "C", "A", "D", "dt_bias", "state")))
    assert L.cr_selective_scan_backward(
        ctypes.byref(sa), ctypes.byref(sg),
        *ws(L.cr_selective_scan_backward_workspace_bytes(batch, T, D, N, 1)), stream) == 0
    # single tokens: the first of each sequence, states in place
    assert L.cr_causal_conv_step(g["x"].ptr, T * D, g["conv"].ptr, batch, None, 4,
                                 g["weight"].ptr, g["bias"].ptr, 1, batch, D, K, 3,
                                 out("conv_step", want["conv_step"]), D, stream) == 0
    sa.len, sa.state = 1, None
    assert L.cr_selective_scan_step(ctypes.byref(sa), g["scan"].ptr, batch, None,
                                    out("scan_step", want["scan_step"]), D, stream) == 0
    torch.cuda.synchronize()
    for name, (buf, like) in outs.items():
        assert torch.equal(buf.view(like.dtype, like.shape), like), name
    assert torch.equal(g["conv"].view(torch.bfloat16, want["conv_after"].shape),
                       want["conv_after"])
    assert torch.equal(g["scan"].view(torch.float32, want["scan_after"].shape),
                       want["scan_after"])
    assert all(b.intact() for b in bands)


@pytest.mark.parametrize("batch,T,D,N", [(1, 2500, 8, 16), (5, 301, 40, 13), (3, 64, 16, 4),
                                         (2, 40, 36, 16), (1, 900, 6, 128)])
def test_state_in_place(scr, batch, T, D, N):
    """The C call may write the final state over the initial one: whole, and cut
    into segments, with a last segment that has nothing to do."""
    from scan_canonical_reduce_gb300 import model as m
    L = scr.lib()
    t = inputs(26, batch=batch, T=T, D=D, N=N)
    lengths = torch.tensor([T, 7, 0, T // 2, T - 1][:batch], device=DEV)
    main = (t["x"], t["dt"], t["A"], t["B"], t["C"])
    extra = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], lengths=lengths)
    stream = torch.cuda.current_stream(DEV).cuda_stream
    size = L.cr_selective_scan_workspace_bytes(batch, T, D, N)
    for _ in range(5):
        y, final, kept = scr.selective_scan(*main, state=t["scan"], return_state=True,
                                            return_checkpoints=True, **extra)
        state, y2, kept2 = t["scan"].clone(), torch.empty_like(y), torch.empty_like(kept)
        kept2.copy_(kept)  # those past a length are not written and may hold anything
        ws = Guarded(nbytes=size)
        args = m._ScanArgs(batch, T, D, N, 1, 1, 3, 8, 0, *(
            v for k in ("x", "dt", "z") for v in (t[k].data_ptr(), T * D, D)), *(
            v for k in ("B", "C") for v in (t[k].data_ptr(), T * N, N)), t["A"].data_ptr(),
            t["D"].data_ptr(), t["dt_bias"].data_ptr(), state.data_ptr(), lengths.data_ptr())
        assert L.cr_selective_scan(ctypes.byref(args), y2.data_ptr(), T * D, D, state.data_ptr(),
                                   kept2.data_ptr(), ws.ptr, size, stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(final, state)
        assert torch.equal(kept.view(torch.int32), kept2.view(torch.int32))
        assert ws.intact()
        t["scan"] = torch.randn_like(t["scan"])


def test_offsets_past_32_bits(scr):
    """Rows that begin more than 2^31 elements into their tensors."""
    gap = (1 << 31) + 4096
    big = torch.zeros(gap + 40 * 64 * 4, dtype=torch.bfloat16, device=DEV)
    t = inputs(7, batch=2, T=40, D=64)
    far = {}
    for i, k in enumerate(("x", "dt", "z", "dy")):
        far[k] = big.as_strided((2, 40, 64), (gap, 64 * 4, 1), i * 64)
        far[k].copy_(t[k])
    want = calls(scr, {k: v.clone() for k, v in t.items()})
    got = calls(scr, {**{k: v.clone() for k, v in t.items()}, **far})
    assert same(got, want)
    del far, got
    # a table of more than 2^31 elements, and its last rows
    rows = big.numel() // 64
    table = big[:rows * 64].view(rows, 64)
    table[-3:] = t["table"][:3, :64]
    tok = torch.tensor([rows - 1, 0, rows - 3, rows, -1], device=DEV)
    got = scr.embedding(tok, table)
    assert torch.equal(got[0], table[-1]) and torch.equal(got[2], table[-3])
    assert not got[3:].any()


def test_empty_calls(scr):
    """No sequences, no steps, no channels: shapes and states without a kernel's help."""
    for batch, T, D in ((0, 5, 8), (2, 0, 8)):
        t = inputs(8, batch=max(batch, 1), T=max(T, 1), D=D)
        cut = {k: v[:batch, :T] for k, v in t.items() if k in ("x", "dt", "z", "B", "C", "dy")}
        conv, scan = t["conv"][:batch], t["scan"][:batch]
        y, last = scr.causal_conv(cut["x"], t["weight"], t["bias"], "silu", conv, return_state=True)
        assert y.shape == cut["x"].shape and torch.equal(last, conv)
        g = scr.causal_conv_backward(cut["dy"], cut["x"], t["weight"], t["bias"], "silu", conv)
        assert not g["weight"].any() and not g["bias"].any()
        main = (cut["x"], cut["dt"], t["A"], cut["B"], cut["C"])
        y, last = scr.selective_scan(*main, state=scan, return_state=True)
        assert y.shape == cut["x"].shape and torch.equal(last, scan)
        g = scr.selective_scan_backward(cut["dy"], *main, D=t["D"], state=scan)
        assert not g["A"].any() and not g["D"].any()
        assert g["B"].shape == cut["B"].shape


def test_binding_refusals(scr):
    t = inputs(9)
    with pytest.raises(TypeError):
        scr.causal_conv(t["x"].double(), t["weight"])
    with pytest.raises(TypeError):
        scr.causal_conv(t["x"], t["weight"].bfloat16())
    with pytest.raises(ValueError):
        scr.causal_conv(t["x"], t["weight"][:5])
    with pytest.raises(ValueError):
        scr.causal_conv(t["x"], t["weight"], activation="relu")
    with pytest.raises(ValueError):
        scr.causal_conv(t["x"], t["weight"], state=t["conv"][:, :1])
    with pytest.raises(TypeError):
        scr.causal_conv(t["x"], t["weight"], lengths=torch.ones(3, device=DEV))
    with pytest.raises(ValueError):
        scr.causal_conv(t["x"], t["weight"], lengths=torch.ones(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        scr.causal_conv(t["x"], t["weight"], out=torch.empty(1, device=DEV, dtype=t["x"].dtype))
    with pytest.raises(scr.CrError):  # the C call's own: K = 1
        scr.causal_conv(t["x"], t["weight"][:, :1].contiguous())
    with pytest.raises(ValueError):
        scr.causal_conv_step(t["x"][:, 0], t["conv"][:2], t["weight"])
    with pytest.raises(ValueError):
        scr.causal_conv_step(t["x"][:, 0], t["conv"].transpose(1, 2).contiguous().transpose(1, 2),
                             t["weight"])
    main = (t["x"], t["dt"], t["A"], t["B"], t["C"])
    with pytest.raises(TypeError):
        scr.selective_scan(t["x"], t["dt"].float(), *main[2:])
    with pytest.raises(ValueError):
        scr.selective_scan(*main[:3], t["B"][:, :5], t["C"])
    with pytest.raises(ValueError):
        scr.selective_scan(*main[:3], t["B"].unsqueeze(2).expand(-1, -1, 3, -1),
                           t["C"].unsqueeze(2).expand(-1, -1, 3, -1))
    with pytest.raises(scr.CrError):  # more than 128 states
        wide = torch.zeros(3, 150, 129, dtype=t["x"].dtype, device=DEV)
        scr.selective_scan(t["x"], t["dt"], torch.zeros(200, 129, device=DEV), wide, wide)
    with pytest.raises(ValueError):
        scr.selective_scan_backward(t["dy"], *main, checkpoints=torch.zeros(1, device=DEV))
    with pytest.raises(ValueError):
        scr.embedding(t["tokens"], t["table"][0])
    with pytest.raises(TypeError):
        scr.embedding(t["tokens"].float(), t["table"])
    with pytest.raises(ValueError):
        scr.embedding_backward(t["tokens"], t["dy"], 500, accumulate=True)
    with pytest.raises(ValueError):
        scr.embedding_backward(t["tokens"][:, :3], t["dy"], 500)


def with_grad(t, names):
    return {k: v.clone().requires_grad_(k in names) for k, v in t.items()}


SCAN_ARGS = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")  # and their names in the gradients
SCAN_GRADS = ("u",) + SCAN_ARGS[1:]


@pytest.mark.parametrize("other", [False, True])
def test_autograd_gives_the_backward_calls(scr, other):
    """What autograd finds for a recorded call is, to the bit, what the backward
    call gives: with states and lengths, on the current stream and on another."""
    t = inputs(30)
    lengths = torch.tensor([150, 0, 77], device=DEV)
    dconv, dscan = torch.randn_like(t["conv"]), torch.randn_like(t["scan"])
    stream = torch.cuda.Stream(DEV) if other else None

    def joined(call):
        if not other:
            return call(None)
        stream.wait_stream(torch.cuda.current_stream(DEV))
        torch.cuda._sleep(2_000_000)
        out = call(stream)
        torch.cuda.current_stream(DEV).wait_stream(stream)
        return out

    p = with_grad(t, t.keys() - {"tokens", "dy"})
    y = joined(lambda s: scr.embedding(p["tokens"], p["table"], 2.0, stream=s))
    y.backward(t["dy"])
    want = scr.embedding_backward(t["tokens"], t["dy"], 500, 2.0).to(t["table"].dtype)
    assert torch.equal(p["table"].grad, want)

    y, last = joined(lambda s: scr.causal_conv(p["x"], p["weight"], p["bias"], "silu", p["conv"],
                                               lengths, return_state=True, stream=s))
    torch.autograd.backward([y, last], [t["dy"], dconv])
    want = scr.causal_conv_backward(t["dy"], t["x"], t["weight"], t["bias"], "silu", t["conv"],
                                    lengths, dconv)
    for k, name in (("x", "x"), ("weight", "weight"), ("bias", "bias"), ("conv", "state")):
        assert torch.equal(p[k].grad, want[name]), k
        p[k].grad = None

    y, last, kept = joined(lambda s: scr.selective_scan(
        *(p[k] for k in SCAN_ARGS), state=p["scan"], lengths=lengths, return_state=True,
        return_checkpoints=True, stream=s))
    assert not kept.requires_grad
    torch.autograd.backward([y, last], [t["dy"], dscan])
    want = scr.selective_scan_backward(t["dy"], *(t[k] for k in SCAN_ARGS), state=t["scan"],
                                       lengths=lengths, dfinal=dscan)
    for k, name in zip(SCAN_ARGS + ("scan",), SCAN_GRADS + ("state",)):
        assert torch.equal(p[k].grad, want[name]), k


def test_autograd_of_some_arguments_and_results(scr):
    t = inputs(31)
    main = [t[k] for k in SCAN_ARGS]
    # one argument that requires a gradient, the state alone used
    A = t["A"].clone().requires_grad_()
    y, last = scr.selective_scan(*main[:2], A, *main[3:], return_state=True)
    last.sum().backward()
    want = scr.selective_scan_backward(torch.zeros_like(t["dy"]), *main,
                                       dfinal=torch.ones_like(last))
    assert torch.equal(A.grad, want["A"]) and y.requires_grad
    y = scr.selective_scan(*main[:2], A, *main[3:])
    assert torch.equal(y.detach(), scr.selective_scan(*main))
    weight = t["weight"].clone().requires_grad_()
    _, last = scr.causal_conv(t["x"], weight, return_state=True)
    last.float().sum().backward()
    assert not weight.grad.any()
    # an expanded gradient, a view of the table, tokens of any shape
    base = torch.randn(2, 500, 200, device=DEV, requires_grad=True)
    scr.embedding(t["tokens"], base[1], 3.0).sum().backward()
    want = scr.embedding_backward(t["tokens"], torch.ones(3, 150, 200, device=DEV), 500, 3.0)
    assert torch.equal(base.grad[1], want) and not base.grad[0].any()
    # nothing is recorded where nothing asks for it, or where recording is off
    assert not scr.embedding(t["tokens"], t["table"]).requires_grad
    with torch.no_grad():
        assert not scr.embedding(t["tokens"], base[0]).requires_grad
        assert not scr.causal_conv(t["x"], weight).requires_grad


def test_autograd_notices_what_is_overwritten(scr):
    """A state that a recorded call has saved and a step then moves on, or a saved
    input that another call's out= replaces, is an error in the backward."""
    t = inputs(33)
    step = scr.selective_scan_step, scr.causal_conv_step
    A, weight = t["A"].clone().requires_grad_(), t["weight"].clone().requires_grad_()
    main = [t[k] for k in SCAN_ARGS]
    one = [v[:, 0] if v.dim() == 3 else v for v in main]
    for touch in (False, True):
        y = scr.selective_scan(*main[:2], A, *main[3:], state=t["scan"])
        x = scr.causal_conv(t["x"], weight, state=t["conv"])
        if touch:
            step[0](*one[:5], t["scan"], one[5], one[6], one[7])
            step[1](t["x"][:, 0], t["conv"], t["weight"])
            for out in (y, x):
                with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                    out.sum().backward()
        else:
            y.sum().backward(), x.sum().backward()
    x = scr.causal_conv(t["x"], weight)
    scr.causal_conv(t["z"], t["weight"], out=t["x"])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        x.sum().backward()
    with torch.inference_mode():  # states of inference: no counter, no complaint
        state = t["conv"].clone()
    scr.causal_conv_step(t["x"][:, 0], state, t["weight"])


def test_autograd_refusals(scr):
    import torch.autograd.forward_ad as forward_ad
    t = inputs(32)
    weight = t["weight"].clone().requires_grad_()
    with pytest.raises(RuntimeError):  # out= leaves no history
        scr.causal_conv(t["x"], weight, out=torch.empty_like(t["x"]))
    y = scr.causal_conv(t["x"], weight, activation="silu")
    with pytest.raises(RuntimeError):  # no gradient of a gradient
        (g,) = torch.autograd.grad(y.float().square().sum(), weight, create_graph=True)
        g.sum().backward()
    with forward_ad.dual_level():  # no tangents
        dual = forward_ad.make_dual(t["table"].float(), torch.ones(500, 200, device=DEV))
        with pytest.raises(RuntimeError):
            scr.embedding(t["tokens"], dual)


def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import recurrent_lm
    finally:
        sys.path.pop(0)
    return recurrent_lm


def test_example_learns_and_repeats(scr):
    """The example's model learns its sequence, and training it again from the
    same seed gives the same losses to the bit."""
    ex = example()
    first = ex.train(ex.RecurrentLM(vocab=13, dim=64, seed=3), 60)
    again = ex.train(ex.RecurrentLM(vocab=13, dim=64, seed=3), 60)
    assert torch.equal(first, again)
    assert first[-5:].mean() < 0.5 * first[:5].mean()


def test_example_steps_follow_the_prompt(scr):
    """Single tokens after a prompt give the logits of the whole sequence: the
    matrix products round differently for one row, binary32 otherwise."""
    ex = example()
    model = ex.RecurrentLM(vocab=13, dim=64, seed=4)
    t = ex.sequence(3, 40, 13, 5)
    with torch.no_grad():
        whole = model.logits(t)
    logits, state = model.prompt(t[:, :30])
    assert torch.allclose(logits, whole[:, :30], rtol=1e-4, atol=1e-4)
    for i in range(30, 40):
        assert torch.allclose(model.step(t[:, i], state), whole[:, i], rtol=1e-3, atol=1e-3), i
