"""The operators of a recurrent language model's token path, as cases to measure:

  embedding       out[i] = scale * table[tokens[i]], and its gradient
                  dW[v] = scale * sum of grad[i] over the i with tokens[i] = v
  causal_conv     y[t] = act(bias + sum_k w[k] x[t - (K-1) + k]) per channel,
                  for prompts, for training and for single tokens
  selective_scan  h[t] = exp(delta[t] A) h[t-1] + delta[t] B[t] u[t],
                  y[t] = (sum_n C[t,n] h[t,n] + D u[t]) silu(z[t]),
                  delta[t] = softplus(dt[t] + dt_bias), per channel and state,
                  for prompts, for training and for single tokens

Tensors are token-major: (batch, time, channel). A token id outside [0, V) is
padding: it reads as a zero row and gets no gradient. Positions at or past a
sequence's length are never read and give zeros.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the lookup of one decoding step of a small batch: latency alone
        dict(name="embed_decode", kind="embed", n=5, V=65536, D=1024, dtype="bf16"),
        # the lookup of a long packed prompt
        dict(name="embed_prompt", kind="embed", n=32768 + 37, V=65536, D=4096, dtype="bf16"),
        # a small model's gradient: odd sizes, binary32, padding ids
        dict(name="embed_grad_odd", kind="embed_grad", n=1037, V=10007, D=333, dtype="f32"),
        # a large training batch: skewed tokens, the whole dense gradient
        dict(name="embed_grad_batch", kind="embed_grad", n=65536, V=65536, D=2048, dtype="bf16"),
        # one token of each running stream of a serving batch
        dict(name="conv_step", kind="conv_step", batch=64, D=4096, K=4, dtype="bf16"),
        # a padded batch of prompts of uneven lengths, some empty
        dict(name="conv_ragged", kind="conv", batch=9, T=517, D=1000, K=3, dtype="f16", ragged=True),
        # the convolution of a training step, both directions
        dict(name="conv_train", kind="conv_train", batch=4, T=4096, D=4096, K=4, dtype="bf16",
             ragged=False),
        # one token of one stream
        dict(name="scan_step_one", kind="scan_step", batch=1, D=2048, N=16, groups=1, dtype="bf16"),
        # one token of each running stream of a large serving batch
        dict(name="scan_step_batch", kind="scan_step", batch=200, D=4096, N=16, groups=1,
             dtype="bf16"),
        # a padded batch of prompts of uneven lengths, binary32, odd sizes, two groups
        dict(name="scan_ragged", kind="scan", batch=5, T=301, D=346, N=13, groups=2, dtype="f32",
             ragged=True),
        # one long prompt: few channels, many steps
        dict(name="scan_long", kind="scan", batch=1, T=32768, D=2048, N=16, groups=1, dtype="bf16",
             ragged=False),
        # the scan of a training step, both directions
        dict(name="scan_train", kind="scan_train", batch=4, T=2048, D=2048, N=16, groups=1,
             dtype="bf16", ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["embed", "embed_grad", "conv_step", "conv", "conv_train", "scan_step",
                       "scan", "scan_train"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind in ("embed", "embed_grad"):
        n = _log(rng, 1, 32768 if kind == "embed" else 65536)
        return dict(kind=kind, n=n, V=_log(rng, 1000, 65536), D=_log(rng, 64, 2048), dtype=dtype)
    if kind == "conv_step":
        return dict(kind=kind, batch=_log(rng, 1, 256), D=_log(rng, 64, 4096),
                    K=rng.randint(2, 4), dtype=dtype)
    if kind == "scan_step":
        groups = rng.choice([1, 1, 2])
        return dict(kind=kind, batch=_log(rng, 1, 200), D=groups * _log(rng, 64, 2048),
                    N=rng.choice([8, 13, 16, 16, 32]), groups=groups, dtype=dtype)
    T = _log(rng, 1, 4096)
    most = 2 ** 23 if kind == "scan_train" else 2 ** 24  # channel steps
    batch = _log(rng, 1, 8)
    ragged = rng.random() < 0.4
    D = max(32, min(4096, most // (batch * T)))
    if kind in ("conv", "conv_train"):
        return dict(kind=kind, batch=batch, T=T, D=_log(rng, 32, D) if D > 32 else 32,
                    K=rng.randint(2, 4), dtype=dtype, ragged=ragged)
    groups = rng.choice([1, 1, 2])
    D = max(32, D // groups)
    return dict(kind=kind, batch=batch, T=T, D=groups * (_log(rng, 32, D) if D > 32 else 32),
                N=rng.choice([8, 13, 16, 16]), groups=groups, dtype=dtype, ragged=ragged)


def work(case):
    kind, es = case["kind"], SIZE[case["dtype"]]
    if kind == "embed":
        e = case["n"] * case["D"]
        return {"bytes": 2 * e * es + 8 * case["n"], "flops": e}
    if kind == "embed_grad":
        e = case["n"] * case["D"]
        return {"bytes": e * es + 8 * case["n"] + 4 * case["V"] * case["D"], "flops": 2 * e}
    D = case["D"]
    if kind == "conv_step":
        e = case["batch"] * D
        K = case["K"]
        return {"bytes": e * es * (2 + 2 * (K - 1)) + 4 * D * (K + 1), "flops": e * (2 * K + 6)}
    if kind in ("conv", "conv_train"):
        e, K = case["batch"] * case["T"] * D, case["K"]
        # forward: x in, y out; backward: x and dy in, dx out
        more = kind == "conv_train"
        return {"bytes": e * es * (5 if more else 2) + 4 * D * (K + 1) * (3 if more else 1),
                "flops": e * (2 * K + 6) * (4 if more else 1)}
    N, G = case["N"], case["groups"]
    if kind == "scan_step":
        e = case["batch"] * D
        return {"bytes": e * es * 4 + e * N * 8 + case["batch"] * G * N * 2 * es + 4 * D * (N + 2),
                "flops": e * (7 * N + 20)}
    rows = case["batch"] * case["T"]
    e, small = rows * D, rows * G * N * 2 * es + 4 * D * (N + 2) + case["batch"] * D * N * 4
    if kind == "scan":  # u, dt, z in, y out
        return {"bytes": e * es * 4 + small, "flops": e * (7 * N + 20)}
    # and u, dt, z, dy in, du, ddt, dz out
    return {"bytes": e * es * 11 + 3 * small, "flops": e * (28 * N + 60)}


# ----------------------------------------------------------------- inputs
def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _tokens(g, n, V):
    """Ids whose k-th most frequent has a share of about 1 / (k ln V), spread over
    the table, with a few padding ids (-1)."""
    r = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(r * math.log(V)) - 1).long().clamp_(0, V - 1)
    ids = (rank * 40503 + 12345) % V
    pad = torch.rand(n, generator=g, device="cuda") < 0.01
    return torch.where(pad, torch.full_like(ids, -1), ids)


def _lengths(g, batch, T):
    """Uneven lengths: the whole range, with an empty sequence and a single token."""
    n = (torch.rand(batch, generator=g, device="cuda") * T).int() + 1
    n.clamp_(max=T)
    n[0] = T
    if batch > 2:
        n[1], n[2] = 0, 1
    return n


def prepare(case, seed):
    kind, dt = case["kind"], TYPES[case["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"kind": kind}
    if kind in ("embed", "embed_grad"):
        n, V, D = case["n"], case["V"], case["D"]
        s["tokens"] = _tokens(g, n, V)
        s["scale"] = math.sqrt(D)
        if kind == "embed":
            s["table"] = _normal(g, (V, D), dt, 0.02)
        else:
            s["vocab"] = V
            s["grad"] = _normal(g, (n, D), dt, 0.01)
        return s
    batch, D = case["batch"], case["D"]
    if kind.startswith("conv"):
        K = case["K"]
        s["weight"] = _normal(g, (D, K), torch.float32, 1 / math.sqrt(K))
        s["bias"] = _normal(g, (D,), torch.float32, 0.1)
        s["state"] = _normal(g, (batch, K - 1, D), dt)
        if kind == "conv_step":
            s["x"] = _normal(g, (batch, D), dt)
            return s
        T = case["T"]
        s["x"] = _normal(g, (batch, T, D), dt)
        s["dy"] = _normal(g, (batch, T, D), dt, 0.1) if kind == "conv_train" else None
        many = ("x", "dy")
    else:
        N, G = case["N"], case["groups"]
        # decays of a trained layer: -1 .. -N with a spread over the channels
        n = torch.arange(1, N + 1, device="cuda", dtype=torch.float32)
        s["A"] = -n * torch.exp(0.3 * torch.randn(D, N, generator=g, device="cuda"))
        s["D"] = 1 + _normal(g, (D,), torch.float32, 0.1)
        # steps between 1e-3 and 1e-1, the usual range of such a layer
        step = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["state"] = _normal(g, (batch, D, N), torch.float32, 0.3)
        lead = (batch,) if kind == "scan_step" else (batch, case["T"])
        s["u"] = _normal(g, lead + (D,), dt)
        s["dt"] = _normal(g, lead + (D,), dt, 0.5)
        s["z"] = _normal(g, lead + (D,), dt)
        s["B"] = _normal(g, lead + (G, N), dt)
        s["C"] = _normal(g, lead + (G, N), dt, 1 / math.sqrt(N))
        if kind == "scan_step":
            return s
        T = case["T"]
        s["dy"] = _normal(g, lead + (D,), dt, 0.1) if kind == "scan_train" else None
        many = ("u", "dt", "z", "B", "C", "dy")
    s["lengths"] = None
    if case["ragged"]:  # what lies past a length is whatever the buffer held
        s["lengths"] = _lengths(g, batch, T)
        past = torch.arange(T, device="cuda")[None, :] >= s["lengths"][:, None]
        for k in many:
            if s[k] is not None:
                s[k][past] = float("nan")
    return s


# ------------------------------------------------------------- plain forms
def _live(s, x):
    """Which (batch, time) positions lie inside their sequences."""
    if s["lengths"] is None:
        return torch.ones(x.shape[:2], dtype=torch.bool, device=x.device)
    return torch.arange(x.shape[1], device=x.device)[None, :] < s["lengths"][:, None]


def _f(x, live):
    """x in 32 bits, with zeros where a position is past its length."""
    return torch.where(live.view(live.shape + (1,) * (x.dim() - 2)), x.float(), 0.0)


def _plain_embed(s):
    t, w = s["tokens"], s["table"]
    rows = w[t.clamp(0, w.shape[0] - 1)].float() * s["scale"]
    return torch.where((t >= 0)[:, None], rows, 0.0).to(w.dtype)


def _plain_embed_grad(s):
    t, g = s["tokens"], s["grad"]
    rows = torch.where((t >= 0)[:, None], g.float() * s["scale"], 0.0)
    out = torch.zeros(s["vocab"], g.shape[1], device=g.device)
    return out.index_add_(0, t.clamp(min=0), rows)


def _plain_conv_step(s):
    x, state = s["x"], s["state"]
    window = torch.cat([state, x[:, None]], 1)
    pre = (window.float() * s["weight"].t()).sum(1) + s["bias"]
    state.copy_(window[:, 1:])
    return {"y": (pre * torch.sigmoid(pre)).to(x.dtype), "state": state}


def _conv_pre(s, x, live):
    K = s["weight"].shape[1]
    xs = torch.cat([s["state"].float(), _f(x, live)], 1)
    return xs, (xs.unfold(1, K, 1) * s["weight"]).sum(-1) + s["bias"]


def _conv_final(s, x):
    """The last K - 1 inputs of each sequence, the state's own where it is shorter."""
    k = s["state"].shape[1]
    xs = torch.cat([s["state"], x], 1)
    n = s["lengths"].long() if s["lengths"] is not None else torch.full(
        (x.shape[0],), x.shape[1], device=x.device)
    at = n[:, None] + torch.arange(k, device=x.device)
    return xs.gather(1, at[:, :, None].expand(-1, -1, x.shape[2]))


def _plain_conv(s):
    x = s["x"]
    live = _live(s, x)
    xs, pre = _conv_pre(s, x, live)
    y = torch.where(live[..., None], pre * torch.sigmoid(pre), 0.0)
    return {"y": y.to(x.dtype), "state": _conv_final(s, x)}


def _plain_conv_train(s):
    x, w = s["x"], s["weight"]
    K, T = w.shape[1], x.shape[1]
    live = _live(s, x)
    xs, pre = _conv_pre(s, x, live)
    sig = torch.sigmoid(pre)
    y = torch.where(live[..., None], pre * sig, 0.0)
    dpre = _f(s["dy"], live) * (sig * (1 + pre * (1 - sig)))
    pad = torch.nn.functional.pad(dpre, (0, 0, K - 1, K - 1))
    dxs = (pad.unfold(1, K, 1) * w.flip(1)).sum(-1)
    dw = (xs.unfold(1, K, 1) * dpre[..., None]).sum((0, 1))
    return {"y": y.to(x.dtype), "x": dxs[:, K - 1:].to(x.dtype), "state": dxs[:, :K - 1].to(x.dtype),
            "weight": dw, "bias": dpre.sum((0, 1))}


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _spread(x, D):
    """(..., groups, N) to (..., D, N): each group's values for all of its channels."""
    return x.repeat_interleave(D // x.shape[-2], -2)


def _plain_scan_step(s):
    u, st = s["u"], s["state"]
    D = u.shape[1]
    uf, zf = u.float(), s["z"].float()
    B, C = _spread(s["B"].float(), D), _spread(s["C"].float(), D)
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    st.copy_(torch.exp(delta[..., None] * s["A"]) * st + (delta * uf)[..., None] * B)
    y = ((st * C).sum(-1) + s["D"] * uf) * (zf * torch.sigmoid(zf))
    return {"y": y.to(u.dtype), "state": st}


def _linear_prefix(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dim 1, by doubling."""
    k = 1
    while k < b.shape[1]:
        b = torch.cat([b[:, :k], torch.addcmul(b[:, k:], a[:, k:], b[:, :-k])], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _scan_forward(s):
    u, A = s["u"], s["A"]
    D = u.shape[2]
    live = _live(s, u)
    uf, zf = _f(u, live), _f(s["z"], live)
    B, C = _spread(_f(s["B"], live), D), _spread(_f(s["C"], live), D)
    raw = _f(s["dt"], live) + s["dt_bias"]
    delta = torch.where(live[..., None], _softplus(raw), 0.0)
    a = torch.exp(delta[..., None] * A)
    b = (delta * uf)[..., None] * B
    b[:, 0] += a[:, 0] * s["state"]
    h = _linear_prefix(a, b)
    y = (h * C).sum(-1) + s["D"] * uf
    sig = torch.sigmoid(zf)
    return live, uf, zf, B, C, raw, delta, a, h, y, sig


def _plain_scan(s):
    live, uf, zf, B, C, raw, delta, a, h, y, sig = _scan_forward(s)
    return {"y": (y * zf * sig).to(s["u"].dtype), "state": h[:, -1].contiguous()}


def _plain_scan_train(s):
    u, A = s["u"], s["A"]
    dtype, D, G = u.dtype, u.shape[2], s["B"].shape[2]
    live, uf, zf, B, C, raw, delta, a, h, y, sig = _scan_forward(s)
    dy = _f(s["dy"], live)
    dz = dy * y * (sig * (1 + zf * (1 - sig)))
    out = (y * zf * sig).to(dtype)
    dy = dy * zf * sig
    prev = torch.cat([s["state"][:, None], h[:, :-1]], 1)
    shifted = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    dC = (dy[..., None] * h).unflatten(2, (G, D // G)).sum(3)
    del h
    g = _linear_prefix(shifted.flip(1), (dy[..., None] * C).flip(1)).flip(1)
    del shifted, C
    dB = (g * (delta * uf)[..., None]).unflatten(2, (G, D // G)).sum(3)
    dstate = a[:, 0] * g[:, 0]
    through = g * a * prev
    gB = (g * B).sum(-1)
    ddelta = (through * A).sum(-1) + gB * uf
    draw_ = ddelta * torch.sigmoid(raw)
    draw_ = torch.where(live[..., None], draw_, 0.0)
    return {"y": out, "u": (gB * delta + s["D"] * dy).to(dtype), "dt": draw_.to(dtype),
            "A": (through * delta[..., None]).sum((0, 1)), "B": dB.to(dtype), "C": dC.to(dtype),
            "D": (dy * uf).sum((0, 1)), "z": dz.to(dtype), "dt_bias": draw_.sum((0, 1)),
            "state": dstate}


# -------------------------------------------------------- the framework's
def _own(s):
    import scan_canonical_reduce_gb300 as cr
    kind = s["kind"]
    if kind == "embed":
        return cr.embedding(s["tokens"], s["table"], s["scale"])
    if kind == "embed_grad":
        return cr.embedding_backward(s["tokens"], s["grad"], s["vocab"], s["scale"])
    if kind == "conv_step":
        y = cr.causal_conv_step(s["x"], s["state"], s["weight"], s["bias"], activation="silu")
        return {"y": y, "state": s["state"]}
    if kind in ("conv", "conv_train"):
        args = dict(bias=s["bias"], activation="silu", state=s["state"], lengths=s["lengths"])
        if kind == "conv":
            y, final = cr.causal_conv(s["x"], s["weight"], return_state=True, **args)
            return {"y": y, "state": final}
        y = cr.causal_conv(s["x"], s["weight"], **args)
        return {"y": y, **cr.causal_conv_backward(s["dy"], s["x"], s["weight"], **args)}
    args = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    main = (s["u"], s["dt"], s["A"], s["B"], s["C"])
    if kind == "scan_step":
        return {"y": cr.selective_scan_step(*main, s["state"], **args), "state": s["state"]}
    args.update(state=s["state"], lengths=s["lengths"])
    if kind == "scan":
        y, final = cr.selective_scan(*main, return_state=True, **args)
        return {"y": y, "state": final}
    y, kept = cr.selective_scan(*main, return_checkpoints=True, **args)
    return {"y": y, **cr.selective_scan_backward(s["dy"], *main, checkpoints=kept, **args)}


PLAIN = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "conv_step": _plain_conv_step,
         "conv": _plain_conv, "conv_train": _plain_conv_train, "scan_step": _plain_scan_step,
         "scan": _plain_scan, "scan_train": _plain_scan_train}


def run(state):
    return _own(state) if own else PLAIN[state["kind"]](state)


# ---------------------------------------------- the definitions in 64 bits
def _exact_embed_grad(s):
    """Sorted rows, their running sums, and the differences at the borders of the tokens."""
    order = torch.argsort(s["tokens"], stable=True)
    t = s["tokens"][order]
    total = torch.cumsum(s["grad"][order].double(), 0)
    total = torch.cat([torch.zeros_like(total[:1]), total])
    v = torch.arange(s["vocab"], device=t.device)
    first, last = torch.searchsorted(t, v), torch.searchsorted(t, v, right=True)
    return (total[last] - total[first]) * s["scale"]


def _exact_conv(s, train):
    """Tap by tap over the sequence with the state in front of it."""
    w, x = s["weight"].double(), s["x"].double()
    K, T = w.shape[1], x.shape[1]
    n = s["lengths"].tolist() if s["lengths"] is not None else [T] * x.shape[0]
    y, dx, dstate = (torch.zeros_like(q) for q in (x, x, s["state"].double()))
    dw, db = torch.zeros_like(w), torch.zeros_like(w[:, 0])
    final = torch.zeros_like(dstate)
    for b in range(x.shape[0]):
        m = n[b]
        xs = torch.cat([s["state"][b].double(), x[b, :m]])
        final[b] = xs[m:]
        pre = s["bias"].double().expand(m, -1).clone()
        for k in range(K):
            pre += xs[k:k + m] * w[:, k]
        y[b, :m] = pre / (1 + torch.exp(-pre))
        if train:
            sig = 1 / (1 + torch.exp(-pre))
            dp = s["dy"][b, :m].double() * (sig + pre * sig * (1 - sig))
            dxs = torch.zeros_like(xs)
            for k in range(K):
                dxs[k:k + m] += dp * w[:, k]
                dw[:, k] += (dp * xs[k:k + m]).sum(0)
            db += dp.sum(0)
            dstate[b], dx[b, :m] = dxs[:K - 1], dxs[K - 1:]
    if train:
        return {"y": y, "x": dx, "state": dstate, "weight": dw, "bias": db}
    return {"y": y, "state": final}


def _exact_scan(s, train):
    """The recurrence, step after step, and for the gradients back again."""
    d = {k: v.double() if isinstance(v, torch.Tensor) and k != "lengths" else v for k, v in s.items()}
    batch, T, D = d["u"].shape
    G, N = d["B"].shape[2:]
    live = torch.ones(batch, T, dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        live = torch.arange(T, device="cuda") < s["lengths"][:, None]
    for k in ("u", "dt", "z", "dy"):
        if d.get(k) is not None:
            d[k] = torch.where(live[..., None], d[k], 0.0)
    for k in ("B", "C"):
        d[k] = torch.where(live[..., None, None], d[k], 0.0)
    raw = d["dt"] + d["dt_bias"]
    delta = torch.where(live[..., None], torch.logaddexp(raw, torch.zeros_like(raw)), 0.0)
    gate = d["z"] / (1 + torch.exp(-d["z"]))
    h = d["state"].clone()
    y = torch.empty_like(raw)
    kept = [h] if train else None
    wide = lambda v: v[:, :, None, :].expand(batch, G, D // G, N).reshape(batch, D, N)  # noqa: E731
    for t in range(T):
        e = delta[:, t, :, None]
        h = torch.exp(e * d["A"]) * h + e * d["u"][:, t, :, None] * wide(d["B"][:, t])
        y[:, t] = (h * wide(d["C"][:, t])).sum(-1)
        if train:
            kept.append(h)
    y += d["D"] * d["u"]
    if not train:
        return {"y": y * gate, "state": h}
    sig = 1 / (1 + torch.exp(-d["z"]))
    dyp = d["dy"] * gate
    out = {"y": y * gate, "z": d["dy"] * y * (sig + d["z"] * sig * (1 - sig)),
           "D": (dyp * d["u"]).sum((0, 1)), "u": d["D"] * dyp, "dt": torch.zeros_like(raw),
           "A": torch.zeros_like(d["A"]), "B": torch.zeros_like(d["B"]), "C": torch.zeros_like(d["C"])}
    back = torch.zeros_like(h)
    for t in range(T - 1, -1, -1):
        e, ut = delta[:, t], d["u"][:, t]
        a = torch.exp(e[..., None] * d["A"])
        b = wide(d["B"][:, t])
        back = back + dyp[:, t, :, None] * wide(d["C"][:, t])
        out["C"][:, t] = (dyp[:, t, :, None] * kept[t + 1]).view(batch, G, D // G, N).sum(2)
        out["B"][:, t] = (back * (e * ut)[..., None]).view(batch, G, D // G, N).sum(2)
        gb = (back * b).sum(-1)
        out["u"][:, t] += gb * e
        q = back * a * kept[t]
        out["A"] += (q * e[..., None]).sum(0)
        out["dt"][:, t] = ((q * d["A"]).sum(-1) + gb * ut) / (1 + torch.exp(-raw[:, t]))
        back = back * a
    out["dt"] = torch.where(live[..., None], out["dt"], 0.0)
    return {**out, "dt_bias": out["dt"].sum((0, 1)), "state": back}


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "embed":
        t, w = s["tokens"], s["table"].double()
        out = torch.zeros(t.shape[0], w.shape[1], dtype=torch.float64, device=t.device)
        out[t >= 0] = w[t[t >= 0]] * s["scale"]
        return out
    if kind == "embed_grad":
        return _exact_embed_grad(s)
    if kind == "conv_step":
        s.update(x=s["x"][:, None], lengths=None)
        r = _exact_conv(s, False)
        return {"y": r["y"][:, 0], "state": r["state"]}
    if kind in ("conv", "conv_train"):
        return _exact_conv(s, kind == "conv_train")
    if kind == "scan_step":
        s.update({k: s[k][:, None] for k in ("u", "dt", "z", "B", "C")}, lengths=None)
        r = _exact_scan(s, False)
        return {"y": r["y"][:, 0], "state": r["state"]}
    return _exact_scan(s, kind == "scan_train")
