"""Layer norm, gated scan and sampling as programs use them: on other streams, in
CUDA graphs, from several threads, with buffers of exactly their size, with
offsets past 32 bits, and together in a small language model."""
import ctypes
import os
import sys
import threading

import pytest
import torch

from .test_gpu_model_use import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def inputs(seed, batch=3, T=300, D=200, V=5000, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = {"x": r(batch, T, D).to(dtype), "gate": (r(batch, T, D) + 2).to(dtype),
         "z": r(batch, T, D).to(dtype), "dy": r(batch, T, D).to(dtype), "state": r(batch, D),
         "dfinal": r(batch, D), "weight": r(D), "bias": r(D), "pool": r(batch, D),
         "logits": 3 * r(batch, V), "u": torch.rand(batch, generator=g),
         "temperature": 0.5 + torch.rand(batch, generator=g),
         "top_k": torch.randint(0, 800, (batch,), generator=g),
         "top_p": 0.5 + 0.5 * torch.rand(batch, generator=g),
         "min_p": 0.1 * torch.rand(batch, generator=g)}
    return {k: v.to(DEV) for k, v in t.items()}


def calls(scr, t, stream=None):
    """Every operator once, on t; {name: result}."""
    s = dict(stream=stream)
    out = {}
    out["norm"], out["stats"] = scr.layer_norm(t["x"], t["weight"], t["bias"], return_stats=True,
                                               **s)
    for name, stats in (("norm_d", out["stats"]), ("norm_again_d", None)):
        for k, v in scr.layer_norm_backward(t["dy"], t["x"], t["weight"], t["bias"], stats=stats,
                                            **s).items():
            out[name + k] = v
    gate = dict(z=t["z"], state=t["state"], **s)
    out["gated"], out["final"], out["kept"] = scr.gated_scan(
        t["x"], t["gate"], return_state=True, return_checkpoints=True, **gate)
    for k, v in scr.gated_scan_backward(t["dy"], t["x"], t["gate"], dfinal=t["dfinal"],
                                        checkpoints=out["kept"], **gate).items():
        out["gated_d" + k] = v
    out["step"] = scr.gated_scan_step(t["x"][:, 0], t["gate"][:, 0], t["pool"], t["z"][:, 0], **s)
    for name, keys in (("sample", ()), ("sample_k", ("top_k",)),
                       ("sample_all", ("temperature", "top_k", "top_p", "min_p")),
                       ("sample_p", ("temperature", "top_p", "min_p"))):
        out[name] = scr.sample(t["logits"], t["u"], **{k: t[k] for k in keys}, **s)
    out["pool_after"] = t["pool"]
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
    shapes = [(v.shape, v.dtype) for k, v in t.items() if k != "pool"]
    got.pop("pool_after")
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
        t = inputs(2)
        u = {k: turned(t[k]) for k in ("x", "gate", "z", "dy", "state", "dfinal", "logits")}
        u.update({k: spread(t[k]) for k in ("weight", "bias", "u", "temperature", "top_k", "top_p",
                                            "min_p")})
        four = turned(t["x"].view(3, 15, 20, 200))
        lengths = spread(torch.tensor([300, 3, 77], device=DEV))
        slots = spread(torch.tensor([2, 0, 1], device=DEV))
        stats = spread(scr.layer_norm(t["x"], return_stats=True)[1])
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream(DEV))
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)
        k = dict(stream=stream)
        out = [scr.layer_norm(u["x"], u["weight"], u["bias"], **k), scr.layer_norm(four, **k)]
        out += scr.layer_norm_backward(u["dy"], u["x"], u["weight"], u["bias"], stats=stats,
                                       **k).values()
        gate = dict(z=u["z"], state=u["state"], lengths=lengths, **k)
        out += scr.gated_scan(u["x"], u["gate"], return_state=True, **gate)
        out += scr.gated_scan_backward(u["dy"], u["x"], u["gate"], dfinal=u["dfinal"],
                                       **gate).values()
        out.append(scr.gated_scan_step(u["x"][:, 0], u["gate"][:, 0], t["pool"], u["z"][:, 0],
                                       slots=slots, **k))
        out.append(scr.sample(u["logits"], u["u"], u["temperature"], u["top_k"], u["top_p"],
                              u["min_p"], **k))
        held = list(u.values()) + [four, lengths, slots, stats]
        return out, [(v.shape, v.dtype) for v in held]

    want, _ = run(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    got, shapes = run(s)  # every input is dropped here, its memory asked for again at once
    junk = [torch.full(shape, 77, dtype=dtype, device=DEV) for shape, dtype in shapes * 3]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))
    del junk


def captured(scr, t, s):
    s.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(s):
        calls(scr, t)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = calls(scr, t)
    return graph, got


def test_graph_replay(scr):
    """Captured once, replayed on new contents of the same buffers, and after
    larger calls on its stream have had scratch memory of their own."""
    t = inputs(3)
    s = torch.cuda.Stream(DEV)
    graph, got = captured(scr, t, s)
    with torch.cuda.stream(s):
        calls(scr, inputs(4, batch=9, T=700, D=520, V=20000))
        s.synchronize()
        held = [torch.full((1 << k,), 7, dtype=torch.uint8, device=DEV)
                for k in (12, 16, 18, 20, 22) for _ in range(8)]
    for seed in (5, 6):
        new = inputs(seed)
        for k in t:
            t[k].copy_(new[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, calls(scr, new)), seed
    assert all(bool((h == 7).all()) for h in held)


def test_graphs_of_one_stream_replayed_on_two(scr):
    t = [inputs(7), inputs(8, T=420)]
    want = [calls(scr, {k: v.clone() for k, v in x.items()}) for x in t]
    s = torch.cuda.Stream(DEV)
    pools = [x["pool"].clone() for x in t]
    graphs = [captured(scr, x, s) for x in t]
    streams = [torch.cuda.Stream(DEV) for _ in t]
    for _ in range(10):
        for x, p in zip(t, pools):
            x["pool"].copy_(p)
        torch.cuda.synchronize()
        for (graph, _), on in zip(graphs, streams):
            with torch.cuda.stream(on):
                graph.replay()
        torch.cuda.synchronize()
        assert all(same(got, w) for (_, got), w in zip(graphs, want))


def test_threads_on_their_own_streams(scr):
    """Also with sizes that take different amounts of shared memory."""
    sizes = {seed: dict(D=d, V=v) for seed, d, v in ((10, 200, 5000), (11, 2048, 70000),
                                                    (12, 4096, 30000), (13, 72, 200000))}
    want = {seed: calls(scr, inputs(seed, **k)) for seed, k in sizes.items()}
    torch.cuda.synchronize()
    bad = []

    def work(seed):
        s = torch.cuda.Stream(DEV)
        with torch.cuda.stream(s):
            for _ in range(4):
                got = calls(scr, inputs(seed, **sizes[seed]))
                s.synchronize()
                if not same(got, want[seed]):
                    bad.append(seed)

    threads = [threading.Thread(target=work, args=(seed,)) for seed in sizes]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad


def test_repeated_calls_give_the_same_bits(scr):
    for k in (dict(), dict(T=2100, D=2048, V=100003), dict(batch=1, T=3000, D=64, V=300000)):
        want = calls(scr, inputs(14, **k))
        for _ in range(3):
            assert same(calls(scr, inputs(14, **k)), want)


def test_launches_are_counted_and_named(scr):
    t, long = inputs(15), inputs(15, D=20000, T=3)
    calls(scr, t)
    before = scr.launch_count()
    scr.profile_enable(True)
    scr.profile_collect()
    calls(scr, t)
    calls(scr, long)
    torch.cuda.synchronize()
    records = scr.profile_collect()
    scr.profile_enable(False)
    assert scr.launch_count() - before == len(records)
    assert {"layer_norm_kernel", "layer_norm_backward_kernel", "layer_norm_sum_kernel",
            "gated_scan_kernel", "gated_scan_backward_kernel", "gated_scan_step_kernel",
            "sample_kernel"} <= {n for n, _ in records}


@pytest.mark.parametrize("D", [200, 77, 2048, 9001])
def test_buffers_of_exact_size(scr, D):
    """Through the C ABI: inputs between NaN bands, outputs and workspaces of
    exactly their size between canaries, which stay as they were."""
    from scan_canonical_reduce_gb300 import model as m
    L = scr.lib()
    batch, T, V = 3, 150, 5001
    t = inputs(16, batch=batch, T=T, D=D, V=V)
    want = calls(scr, {k: v.clone() for k, v in t.items()})
    stream = torch.cuda.current_stream(DEV).cuda_stream
    g = {k: Guarded(v) for k, v in t.items()}
    bands, outs = list(g.values()), {}

    def out(name):
        like = want[name]
        outs[name] = (Guarded(nbytes=like.numel() * like.element_size()), like)
        bands.append(outs[name][0])
        return outs[name][0].ptr

    na = m._NormArgs(batch, T, D, 3, 1e-5, g["x"].ptr, T * D, D, g["weight"].ptr, g["bias"].ptr)
    assert L.cr_layer_norm(ctypes.byref(na), out("norm"), T * D, D, out("stats"), stream) == 0
    size = L.cr_layer_norm_backward_workspace_bytes(batch, T, D)
    for name, stats in (("norm_d", outs["stats"][0].ptr), ("norm_again_d", None)):
        ng = m._NormGrads(g["dy"].ptr, T * D, D, stats, out(name + "x"), T * D, D,
                          out(name + "weight"), out(name + "bias"))
        ws = Guarded(nbytes=size)
        bands.append(ws)
        assert L.cr_layer_norm_backward(ctypes.byref(na), ctypes.byref(ng), ws.ptr, size,
                                        stream) == 0
    ga = m._GateArgs(batch, T, D, 3, 8, *(
        v for k in ("x", "gate", "z") for v in (g[k].ptr, T * D, D)), g["state"].ptr, None)
    assert L.cr_gated_scan(ctypes.byref(ga), out("gated"), T * D, D, out("final"), out("kept"),
                           stream) == 0
    gg = m._GateGrads(g["dy"].ptr, T * D, D, g["dfinal"].ptr, outs["kept"][0].ptr,
                      *(out("gated_d" + k) for k in ("x", "gate", "z", "state")))
    assert L.cr_gated_scan_backward(ctypes.byref(ga), ctypes.byref(gg), stream) == 0
    ga.len, ga.state = 1, None
    assert L.cr_gated_scan_step(ctypes.byref(ga), g["pool"].ptr, batch, None, out("step"), D,
                                stream) == 0
    sa = m._SampleArgs(batch, V, 1, 8, g["logits"].ptr, V, g["u"].ptr, 1.0, 1.0, 0.0, 0,
                       g["temperature"].ptr, g["top_p"].ptr, g["min_p"].ptr, g["top_k"].ptr)
    assert L.cr_sample(ctypes.byref(sa), out("sample_all"), stream) == 0
    torch.cuda.synchronize()
    for name, (buf, like) in outs.items():
        assert torch.equal(buf.view(like.dtype, like.shape), like), name
    assert torch.equal(g["pool"].view(torch.float32, t["pool"].shape), want["pool_after"])
    assert all(b.intact() for b in bands)


def test_final_state_over_the_initial_one(scr):
    """The C call may write the final state over the initial one, however many
    blocks share a sequence."""
    from scan_canonical_reduce_gb300 import model as m
    L = scr.lib()
    stream = torch.cuda.current_stream(DEV).cuda_stream
    for batch, T, D in ((1, 5000, 8), (5, 301, 40), (2, 1, 16), (3, 0, 16)):
        t = inputs(17, batch=batch, T=max(T, 1), D=D)
        cut = {k: t[k][:, :T].contiguous() for k in ("x", "gate", "z")}
        y, final = scr.gated_scan(*cut.values(), state=t["state"], return_state=True)
        y2, state = torch.empty_like(y), t["state"].clone()
        a = m._GateArgs(batch, T, D, 3, 8, *(
            v for k in cut.values() for v in (k.data_ptr(), T * D, D)), state.data_ptr(), None)
        assert L.cr_gated_scan(ctypes.byref(a), y2.data_ptr(), T * D, D, state.data_ptr(), None,
                               stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(final, state)


def test_offsets_past_32_bits(scr):
    """Rows that begin more than 2^31 elements into their tensors."""
    gap = (1 << 31) + 4096
    big = torch.zeros(gap + 40 * 64 * 4, dtype=torch.bfloat16, device=DEV)
    t = inputs(18, batch=2, T=40, D=64)
    far = {}
    for i, k in enumerate(("x", "gate", "z", "dy")):
        far[k] = big.as_strided((2, 40, 64), (gap, 64 * 4, 1), i * 64)
        far[k].copy_(t[k])
    want = calls(scr, {k: v.clone() for k, v in t.items()})
    assert same(calls(scr, {**{k: v.clone() for k, v in t.items()}, **far}), want)
    rows = big.as_strided((2, 500), (gap, 1), 0)
    near = torch.randn(2, 500, device=DEV).bfloat16()
    rows.copy_(near)
    assert torch.equal(scr.sample(rows, t["u"][:2]), scr.sample(near, t["u"][:2]))


def test_autograd_on_another_stream(scr):
    t = inputs(19, dtype=torch.float32)
    want = scr.gated_scan_backward(t["dy"], t["x"], t["gate"], t["z"])
    normed = scr.layer_norm_backward(t["dy"], t["x"], t["weight"], t["bias"])
    s = torch.cuda.Stream(DEV)
    leaves = {k: t[k].clone().requires_grad_(True) for k in ("x", "gate", "z", "weight", "bias")}
    s.wait_stream(torch.cuda.current_stream(DEV))
    y = scr.gated_scan(leaves["x"], leaves["gate"], leaves["z"], stream=s)
    n = scr.layer_norm(leaves["x"], leaves["weight"], leaves["bias"], stream=s)
    torch.cuda.current_stream(DEV).wait_stream(s)
    y.backward(t["dy"])
    assert torch.equal(leaves["gate"].grad, want["gate"])
    leaves["x"].grad = None
    n.backward(t["dy"])
    torch.cuda.synchronize()
    assert torch.equal(leaves["x"].grad, normed["x"])
    assert torch.equal(leaves["weight"].grad, normed["weight"])


def test_another_device_than_the_current_one_is_named(scr):
    """Tensors of one device, and streams of that device."""
    t = inputs(20)
    for call in (lambda: scr.layer_norm(t["x"], t["weight"].cpu()),
                 lambda: scr.gated_scan(t["x"], t["gate"].cpu()),
                 lambda: scr.sample(t["logits"], t["u"], top_p=t["top_p"].cpu())):
        with pytest.raises(ValueError):
            call()


def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import recurrent_lm
    finally:
        sys.path.pop(0)
    return recurrent_lm


def test_example_trains_and_repeats(scr):
    """A training run of the gated model: the same losses to the bit from the same
    seed, and gradients of every parameter."""
    ex = example()
    first = ex.train(ex.GatedLM(vocab=13, dim=64, seed=3), 8)
    again = ex.train(ex.GatedLM(vocab=13, dim=64, seed=3), 8)
    assert torch.equal(first, again) and first.isfinite().all()
    model = ex.GatedLM(vocab=13, dim=64, seed=4)
    model.logits(ex.sequence(2, 30, 13, 5)).square().sum().backward()
    assert all(v.grad is not None and v.grad.isfinite().all() and v.grad.any()
               for v in model.p.values())


def test_example_gradients_match_differences(scr):
    """The whole model's derivative along a direction of each parameter, against
    differences of a loss that is summed in binary64. The model's binary32 values
    are off by some 2^-20 of themselves, which 2 e = 4e-3 divides; the rest is e^2
    of the third derivative."""
    ex = example()
    torch.backends.cuda.matmul.allow_tf32 = False
    model = ex.GatedLM(vocab=11, dim=32, seed=6)
    t = ex.sequence(2, 12, 11, 7)
    pick = torch.randn(2, 12, 11, generator=torch.Generator().manual_seed(8)).to(DEV)

    def loss():
        return (model.logits(t).double() * pick).sum()
    loss().backward()
    gen = torch.Generator().manual_seed(9)
    for name, p in model.p.items():
        v = torch.randn(p.shape, generator=gen).to(DEV)
        v *= 1.0 / v.norm()
        with torch.no_grad():
            ends = []
            for sign in (1, -1):
                p += sign * 2e-3 * v
                ends.append(loss())
                p -= sign * 2e-3 * v
        want = float(ends[0] - ends[1]) / 4e-3
        got = float((p.grad * v).sum())
        size = float(p.grad.norm())
        assert abs(got - want) <= 2e-2 * size + 2e-2, (name, got, want)


def test_example_steps_follow_the_prompt(scr):
    """Single tokens after a prompt give the logits of the whole sequence: the
    matrix products round differently for one row, binary32 otherwise."""
    ex = example()
    model = ex.GatedLM(vocab=13, dim=64, seed=4)
    t = ex.sequence(3, 40, 13, 5)
    with torch.no_grad():
        whole = model.logits(t)
    logits, state = model.prompt(t[:, :30])
    assert torch.allclose(logits, whole[:, :30], rtol=1e-4, atol=1e-4)
    for i in range(30, 40):
        assert torch.allclose(model.step(t[:, i], state), whole[:, i], rtol=1e-3, atol=1e-3), i


def test_sampling_of_the_example(scr):
    """u picks the tokens: 0 the likeliest, the same ones again, none outside the
    vocabulary; a temperature of 0 is the greedy continuation."""
    ex = example()
    model = ex.GatedLM(vocab=13, dim=64, seed=4)
    t = ex.sequence(3, 20, 13, 5)
    u = torch.rand(6, 3, generator=torch.Generator().manual_seed(1)).to(DEV)
    got = ex.sampled(model, t, u, top_p=0.9)
    assert torch.equal(got, ex.sampled(model, t, u, top_p=0.9))
    assert ((got >= 0) & (got < 13)).all()
    greedy = ex.generate(model, t, 6)
    assert torch.equal(ex.sampled(model, t, u, temperature=0.0), greedy)
    assert torch.equal(ex.sampled(model, t, torch.zeros_like(u)), greedy)
