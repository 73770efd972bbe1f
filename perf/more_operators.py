"""More operators of a recurrent language model, as cases to measure:

  layer_norm  y = (x - mean) rstd weight + bias over the last axis,
              rstd = 1 / sqrt(mean of (x - mean)^2 + eps), and its gradients with
              the sums over rows for weight and bias
  gated_scan  a[t] = sigmoid(gate[t]), h[t] = a[t] h[t-1] + (1 - a[t]) x[t],
              y[t] = h[t] silu(z[t]) per channel, for prompts, for training and
              for single tokens
  sample      the next token of each row of logits from a given uniform number:
              tokens in the order of falling logits (equal ones by index) have
              weights w = exp((logit - largest) / temperature); kept are the
              first of them: top_k at most, those before which less than top_p
              of the top_k's weight lies, and with w >= min_p, the first in any
              case; the token is the first whose running sum of kept weights
              exceeds u times their sum

Tensors are token-major: (batch, time, channel). Positions at or past a
sequence's length are never read and give zeros. A logit of -inf or NaN is no
candidate; a row without candidates gives -1. A temperature of zero takes the
first token; top_k 0, top_p 1 and min_p 0 set no limit.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm in front of a layer in one decoding step of one stream: latency alone
        dict(name="norm_one", kind="norm", rows=1, D=2048, dtype="bf16", affine=True),
        # the norm over a long packed prompt
        dict(name="norm_prompt", kind="norm", rows=32768 + 37, D=4096, dtype="bf16", affine=True),
        # a small model's training step: odd sizes, binary32
        dict(name="norm_train_odd", kind="norm_train", rows=1037, D=333, dtype="f32", affine=True),
        # the norm of a training step, both directions
        dict(name="norm_train", kind="norm_train", rows=16384, D=2048, dtype="bf16", affine=True),
        # one token of each running stream of a serving batch
        dict(name="gate_step", kind="gate_step", batch=64, D=4096, dtype="bf16", z=True),
        # a padded batch of prompts of uneven lengths, some empty
        dict(name="gate_ragged", kind="gate", batch=9, T=517, D=1000, dtype="f16", z=True,
             ragged=True),
        # one long prompt: few channels, many steps
        dict(name="gate_long", kind="gate", batch=1, T=32768, D=2048, dtype="bf16", z=True,
             ragged=False),
        # the recurrence of a training step, both directions
        dict(name="gate_train", kind="gate_train", batch=4, T=4096, D=4096, dtype="bf16", z=True,
             ragged=False),
        # the next token of one stream
        dict(name="sample_one", kind="sample", rows=1, V=65536, dtype="f32", k=50, p=0.95,
             min_p=0.0, mixed=False, masked=False),
        # a small vocabulary, part of it masked by a grammar, one row wholly
        dict(name="sample_odd", kind="sample", rows=37, V=10007, dtype="f16", k=0, p=0.9,
             min_p=0.0, mixed=False, masked=True),
        # a serving batch whose streams each have their own settings
        dict(name="sample_batch", kind="sample", rows=200, V=65536, dtype="f32", k=0, p=0.95,
             min_p=0.05, mixed=True, masked=False),
        # a large vocabulary, temperature alone: every token counts
        dict(name="sample_wide", kind="sample", rows=64, V=262144, dtype="bf16", k=0, p=1.0,
             min_p=0.0, mixed=False, masked=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm", "norm_train", "gate_step", "gate", "gate_train", "sample",
                       "sample"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind in ("norm", "norm_train"):
        D = _log(rng, 64, 16384)
        rows = _log(rng, 1, min(65536, 2 ** (26 if kind == "norm" else 25) // D))
        return dict(kind=kind, rows=rows, D=D, dtype=dtype, affine=rng.random() < 0.8)
    if kind == "gate_step":
        return dict(kind=kind, batch=_log(rng, 1, 256), D=_log(rng, 64, 8192), dtype=dtype,
                    z=rng.random() < 0.7)
    if kind in ("gate", "gate_train"):
        T, batch = _log(rng, 1, 8192), _log(rng, 1, 8)
        most = max(32, min(8192, 2 ** 24 // (batch * T)))
        return dict(kind=kind, batch=batch, T=T, D=_log(rng, 32, most) if most > 32 else 32,
                    dtype=dtype, z=rng.random() < 0.7, ragged=rng.random() < 0.4)
    V = _log(rng, 1000, 262144)
    return dict(kind=kind, rows=_log(rng, 1, min(512, 2 ** 23 // V)), V=V, dtype=dtype,
                k=rng.choice([0, 0, 1, 40, 1000]), p=rng.choice([1.0, 0.95, 0.8, 0.5]),
                min_p=rng.choice([0.0, 0.0, 0.02, 0.1]), mixed=rng.random() < 0.3,
                masked=rng.random() < 0.3)


def work(case):
    kind, es = case["kind"], SIZE[case["dtype"]]
    if kind in ("norm", "norm_train"):
        e, D = case["rows"] * case["D"], case["D"]
        vectors = 2 if case["affine"] else 0
        if kind == "norm":  # x in, y out
            return {"bytes": 2 * e * es + 4 * D * vectors, "flops": 8 * e}
        # and x and dy in, dx out
        return {"bytes": 5 * e * es + 4 * D * vectors * 2, "flops": 24 * e}
    if kind == "sample":
        e = case["rows"] * case["V"]
        return {"bytes": e * es + 28 * case["rows"], "flops": 8 * e}
    n, D = 4 if case["z"] else 3, case["D"]
    if kind == "gate_step":
        e = case["batch"] * D
        return {"bytes": e * (n * es + 8), "flops": 20 * e}
    e, state = case["batch"] * case["T"] * D, 4 * case["batch"] * D
    if kind == "gate":  # x, gate, z in, y out
        return {"bytes": n * e * es + 2 * state, "flops": 20 * e}
    # and x, gate, z, dy in, dx, dgate, dz out
    return {"bytes": (3 * n - 1) * e * es + 3 * state, "flops": 70 * e}


# ----------------------------------------------------------------- inputs
def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _lengths(g, batch, T):
    """Uneven lengths: the whole range, with an empty sequence and a single token."""
    n = (torch.rand(batch, generator=g, device="cuda") * T).int() + 1
    n.clamp_(max=T)
    n[0] = T
    if batch > 2:
        n[1], n[2] = 0, 1
    return n


def _norm_inputs(s, case, g, dt):
    rows, D = case["rows"], case["D"]
    # a residual stream: channels of uneven size, rows that are off zero
    size = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))
    off = torch.randn(rows, 1, generator=g, device="cuda")
    s["x"] = torch.randn(rows, D, generator=g, device="cuda").mul_(size).add_(off).to(dt)
    s["weight"] = s["bias"] = None
    if case["affine"]:
        s["weight"] = 1 + _normal(g, (D,), torch.float32, 0.1)
        s["bias"] = _normal(g, (D,), torch.float32, 0.1)
    if case["kind"] == "norm_train":
        s["dy"] = _normal(g, (rows, D), dt, 0.1)


def _gate_inputs(s, case, g, dt):
    batch, D = case["batch"], case["D"]
    lead = (batch,) if case["kind"] == "gate_step" else (batch, case["T"])
    # memories of 1 to 1000 steps over the channels, with the spread of a trained layer
    steps = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(1000.0))
    s["gate"] = torch.randn(lead + (D,), generator=g, device="cuda").add_(torch.log(steps)).to(dt)
    s["x"] = _normal(g, lead + (D,), dt)
    s["z"] = _normal(g, lead + (D,), dt) if case["z"] else None
    s["state"] = _normal(g, (batch, D), torch.float32, 0.3)
    if case["kind"] == "gate_step":
        return
    s["dy"] = _normal(g, lead + (D,), dt, 0.1) if case["kind"] == "gate_train" else None
    s["lengths"] = None
    if case["ragged"]:  # what lies past a length is whatever the buffer held
        s["lengths"] = _lengths(g, batch, case["T"])
        past = torch.arange(case["T"], device="cuda")[None, :] >= s["lengths"][:, None]
        for k in ("x", "gate", "z", "dy"):
            if s[k] is not None:
                s[k][past] = float("nan")


def _sample_inputs(s, case, g, dt):
    rows, V = case["rows"], case["V"]
    # a bell of unlikely tokens and a few that the context asks for
    x = torch.randn(rows, V, generator=g, device="cuda").mul_(2.0)
    few = torch.rand(rows, 8, generator=g, device="cuda")
    x.scatter_(1, torch.randint(0, V, (rows, 8), generator=g, device="cuda"), 6.0 + 6.0 * few)
    if case["masked"]:
        out = torch.rand(rows, V, generator=g, device="cuda") < 0.6
        x[out] = -math.inf
        x[:, ::7] = torch.finfo(dt).min  # the other way in which programs mask
        if rows > 2:
            x[1] = -math.inf
    s["logits"] = x.to(dt)
    s["u"] = torch.rand(rows, generator=g, device="cuda")
    if not case["mixed"]:
        s.update(temperature=0.8, top_k=case["k"], top_p=case["p"], min_p=case["min_p"])
        return
    r = lambda: torch.rand(rows, generator=g, device="cuda")  # noqa: E731
    s["temperature"] = torch.where(r() < 0.2, 0.0, 0.5 + r())
    s["top_k"] = torch.where(r() < 0.4, 0.0, 1 + 200 * r()).int()
    s["top_p"] = torch.where(r() < 0.3, 1.0, 0.5 + 0.5 * r())
    s["min_p"] = torch.where(r() < 0.5, 0.0, 0.2 * r())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s, kind = {"kind": case["kind"]}, case["kind"]
    fill = _norm_inputs if kind.startswith("norm") else _sample_inputs if kind == "sample" \
        else _gate_inputs
    fill(s, case, g, TYPES[case["dtype"]])
    return s


# ------------------------------------------------------------- plain forms
def _normed(s):
    x = s["x"].float()
    d = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS)
    return d * rstd, rstd


def _scaled(s, xhat):
    y = xhat if s["weight"] is None else xhat * s["weight"] + s["bias"]
    return y.to(s["x"].dtype)


def _plain_norm(s):
    return _scaled(s, _normed(s)[0])


def _plain_norm_train(s):
    xhat, rstd = _normed(s)
    dy, w = s["dy"].float(), s["weight"]
    g = dy if w is None else dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    out = {"y": _scaled(s, xhat), "x": dx.to(s["x"].dtype)}
    if w is not None:
        out["weight"], out["bias"] = (dy * xhat).sum(0), dy.sum(0)
    return out


def _live(s):
    """Which (batch, time) positions lie inside their sequences."""
    x = s["x"]
    if s["lengths"] is None:
        return torch.ones(x.shape[:2], dtype=torch.bool, device=x.device)[..., None]
    return (torch.arange(x.shape[1], device=x.device) < s["lengths"][:, None])[..., None]


def _linear_prefix(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dim 1, by doubling."""
    k = 1
    while k < b.shape[1]:
        b = torch.cat([b[:, :k], torch.addcmul(b[:, k:], a[:, k:], b[:, :-k])], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _plain_gate_step(s):
    gate, st = s["gate"].float(), s["state"]
    st.copy_(torch.sigmoid(gate) * st + torch.sigmoid(-gate) * s["x"].float())
    y = st
    if s["z"] is not None:
        z = s["z"].float()
        y = st * (z * torch.sigmoid(z))
    return {"y": y.to(s["x"].dtype), "state": st}


def _gate_forward(s):
    """Past a length the state is held: a = 1, 1 - a = 0."""
    live = _live(s)
    x = torch.where(live, s["x"].float(), 0.0)
    gate = torch.where(live, s["gate"].float(), math.inf)
    a, rest = torch.sigmoid(gate), torch.sigmoid(-gate)
    b = rest * x
    b[:, 0] += a[:, 0] * s["state"]
    h = _linear_prefix(a, b)
    z = None if s["z"] is None else torch.where(live, s["z"].float(), 0.0)
    y = torch.where(live, h, 0.0) if z is None else h * (z * torch.sigmoid(z))
    return live, x, a, rest, h, z, y.to(s["x"].dtype)


def _plain_gate(s):
    live, x, a, rest, h, z, y = _gate_forward(s)
    return {"y": y, "state": h[:, -1].contiguous()}


def _plain_gate_train(s):
    live, x, a, rest, h, z, y = _gate_forward(s)
    dtype = s["x"].dtype
    dy = torch.where(live, s["dy"].float(), 0.0)
    out = {"y": y}
    if z is not None:
        sig = torch.sigmoid(z)
        out["z"] = (dy * h * (sig * (1 + z * (1 - sig)))).to(dtype)
        dy = dy * (z * sig)
    shifted = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _linear_prefix(shifted.flip(1), dy.flip(1)).flip(1)
    prev = torch.cat([s["state"][:, None], h[:, :-1]], 1)
    out["state"] = a[:, 0] * g[:, 0]
    out["gate"] = ((prev - x) * g * (a * rest)).to(dtype)
    out["x"] = (g * rest).to(dtype)
    return out


def _column(v, like):
    """A setting, one for all rows or one a row, as a column in 64 bits."""
    v = torch.as_tensor(v, device=like.device, dtype=torch.float64)
    return v.expand(like.shape[0])[:, None]


def _plain_sample(s):
    x = s["logits"].double()
    x = torch.where(x.isnan(), -math.inf, x)
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    T, k, p, min_p = (_column(s[n], x) for n in ("temperature", "top_k", "top_p", "min_p"))
    rank = torch.arange(x.shape[1], device=x.device)
    real = x > -math.inf
    w = torch.where(real, torch.exp((x - x[:, :1]) / torch.where(T > 0, T, 1.0)), 0.0)
    w = torch.where((k <= 0) | (rank < k), w, 0.0)
    run = torch.cumsum(w, 1)
    keep = ((p >= 1) | (run - w < p * run[:, -1:])) & (w >= min_p) & ((T > 0) | (rank == 0))
    w = torch.where(keep | (rank == 0), w, 0.0)
    run = torch.cumsum(w, 1)
    beyond = (w > 0) & (run > s["u"].double()[:, None] * run[:, -1:])
    last = (w > 0).sum(1) - 1
    at = torch.where(beyond.any(1), beyond.int().argmax(1), last).clamp(min=0)
    return torch.where(real[:, 0], order.gather(1, at[:, None])[:, 0], -1)


# -------------------------------------------------------- the framework's
def _own(s):
    import scan_canonical_reduce_gb300 as cr
    kind = s["kind"]
    if kind == "norm":
        return cr.layer_norm(s["x"], s["weight"], s["bias"], EPS)
    if kind == "norm_train":
        y, stats = cr.layer_norm(s["x"], s["weight"], s["bias"], EPS, return_stats=True)
        return {"y": y, **cr.layer_norm_backward(s["dy"], s["x"], s["weight"], s["bias"], EPS,
                                                 stats=stats)}
    if kind == "sample":
        return cr.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                         top_p=s["top_p"], min_p=s["min_p"])
    if kind == "gate_step":
        return {"y": cr.gated_scan_step(s["x"], s["gate"], s["state"], s["z"]),
                "state": s["state"]}
    args = dict(z=s["z"], state=s["state"], lengths=s["lengths"])
    if kind == "gate":
        y, final = cr.gated_scan(s["x"], s["gate"], return_state=True, **args)
        return {"y": y, "state": final}
    y, kept = cr.gated_scan(s["x"], s["gate"], return_checkpoints=True, **args)
    return {"y": y, **cr.gated_scan_backward(s["dy"], s["x"], s["gate"], checkpoints=kept, **args)}


PLAIN = {"norm": _plain_norm, "norm_train": _plain_norm_train, "gate_step": _plain_gate_step,
         "gate": _plain_gate, "gate_train": _plain_gate_train, "sample": _plain_sample}


def run(state):
    return _own(state) if own else PLAIN[state["kind"]](state)


# ---------------------------------------------- the definitions in 64 bits
def _exact_norm(s, train):
    """By raw moments about the row's first element."""
    x = s["x"].double()
    D = x.shape[1]
    first = x[:, :1]
    d = x - first
    m = d.sum(1, keepdim=True) / D
    scale = ((d * d).sum(1, keepdim=True) / D - m * m + EPS) ** -0.5
    xhat = (d - m) * scale
    w = 1.0 if s["weight"] is None else s["weight"].double()
    y = xhat * w + (0.0 if s["bias"] is None else s["bias"].double())
    if not train:
        return y
    dy = s["dy"].double()
    out = {"y": y}
    if s["weight"] is not None:
        out["weight"] = torch.einsum("rd,rd->d", dy, xhat)
        out["bias"] = torch.einsum("rd->d", dy)
    q = dy * w
    dots = torch.einsum("rd,rd->r", q, xhat)[:, None]
    out["x"] = (D * q - q.sum(1, keepdim=True) - dots * xhat) * (scale / D)
    return out


def _exact_gate(s, train):
    """The recurrence, step after step, and for the gradients back again."""
    x, gate = s["x"].double(), s["gate"].double()
    batch, T, D = x.shape
    n = torch.full((batch,), T, device=x.device) if s["lengths"] is None else s["lengths"]
    z = None if s["z"] is None else s["z"].double()
    h = s["state"].double()
    y = torch.zeros_like(x)
    hs = torch.empty_like(x) if train else None
    rest = 1 / (1 + torch.exp(gate))
    for t in range(T):
        inside = (t < n)[:, None]
        new = h + rest[:, t] * (x[:, t] - h)
        h = torch.where(inside, new, h)
        y[:, t] = torch.where(inside, h, 0.0)
        if train:
            hs[:, t] = h
    if z is not None:
        sig = 1 / (1 + torch.exp(-z))
        y = torch.where(y == 0, 0.0, y * z * sig)
    if not train:
        return {"y": y, "state": h}
    out = {"y": y, "x": torch.zeros_like(x), "gate": torch.zeros_like(x)}
    dy = s["dy"].double()
    if z is not None:
        inside = (torch.arange(T, device=x.device) < n[:, None])[..., None]
        out["z"] = torch.where(inside, dy * hs * (sig + z * sig * (1 - sig)), 0.0)
        dy = dy * z * sig
    back = torch.zeros_like(h)
    for t in range(T - 1, -1, -1):
        inside = (t < n)[:, None]
        g = back + dy[:, t]
        before = hs[:, t - 1] if t else s["state"].double()
        r = rest[:, t]
        out["x"][:, t] = torch.where(inside, g * r, 0.0)
        out["gate"][:, t] = torch.where(inside, g * (before - x[:, t]) * (r * (1 - r)), 0.0)
        back = torch.where(inside, g - g * r, back)
    return {**out, "state": back}


def _exact_sample(s):
    """Row by row: what lies above each level of the logits, without the rest."""
    out = []
    rows, V = s["logits"].shape
    T, k, p, min_p = (_column(s[n], s["logits"])[:, 0].tolist()
                      for n in ("temperature", "top_k", "top_p", "min_p"))
    for r in range(rows):
        x = s["logits"][r].double()
        ids = (x > -math.inf).nonzero()[:, 0]
        if ids.numel() == 0:
            out.append(-1)
            continue
        ids = ids[torch.argsort(-x[ids], stable=True)]
        if k[r] > 0:
            ids = ids[:int(k[r])]
        if not T[r] > 0:
            out.append(int(ids[0]))
            continue
        prob = torch.softmax(x[ids] / T[r], 0)
        n = ids.numel()
        if p[r] < 1:
            n = int((torch.cumsum(prob, 0) < p[r]).sum()) + 1
        n = max(1, min(n, int((prob >= min_p[r] * prob[0]).sum())))
        run = torch.cumsum(prob[:n], 0)
        at = int((run <= s["u"][r].double() * run[-1]).sum())
        out.append(int(ids[min(at, n - 1)]))
    return torch.tensor(out, device="cuda")


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "sample":
        return _exact_sample(s)
    if kind.startswith("norm"):
        return _exact_norm(s, kind == "norm_train")
    if kind == "gate_step":
        s.update({k: s[k][:, None] for k in ("x", "gate")}, lengths=None,
                 z=None if s["z"] is None else s["z"][:, None])
        r = _exact_gate(s, False)
        return {"y": r["y"][:, 0], "state": r["state"]}
    return _exact_gate(s, kind == "gate_train")
