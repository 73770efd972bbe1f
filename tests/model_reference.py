"""Plain 64-bit evaluation of the model operators (test infrastructure): the
formulas step by step on the CPU, with a magnitude beside each result.

The magnitude of a result is the same formula with every term replaced by its
absolute value (decays as they are). A sum of terms evaluated in binary32 with
k roundings and steps in any order is within k * 2^-23 * magnitude of the
exact value, which is how the tests' tolerances are derived."""
import numpy as np
import torch

U32 = 2.0 ** -23  # a binary32 operation's relative error, with a factor 2 of room
# relative rounding of a stored result, and the spacing of its smallest values
STORE = {torch.float32: (2.0 ** -24, 2.0 ** -149), torch.bfloat16: (2.0 ** -8, 2.0 ** -133),
         torch.float16: (2.0 ** -11, 2.0 ** -24)}


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def close(got, want, magnitude, steps, what=""):
    """|got - want| <= store * |want| + steps * 2^-23 * magnitude, elementwise."""
    rel, tiny = STORE[got.dtype]
    g = f64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    assert np.isfinite(g).all(), what
    tol = rel * np.abs(want) + (1 + rel) * steps * U32 * magnitude + tiny
    bad = np.abs(g - want) > tol
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(g - want) / tol), g.shape)
        raise AssertionError("%s: %d of %d off, worst at %s: got %r want %r tol %r" % (
            what, bad.sum(), bad.size, i, g[i], want[i], tol[i]))


def sigmoid(v):
    return 0.5 * (1 + np.tanh(0.5 * v))


# ------------------------------------------------------------------ conv
def conv(x, w, bias, silu, state, lengths, dy=None, dfinal=None):
    """x (batch, T, D) etc. as float64 arrays. Returns {name: (value, magnitude)}."""
    Bn, T, D = x.shape
    K = w.shape[1]
    y, ym = np.zeros((Bn, T, D)), np.zeros((Bn, T, D))
    final = np.zeros((Bn, K - 1, D))
    g = {k: [np.zeros(s), np.zeros(s)] for k, s in (
        ("x", x.shape), ("weight", w.shape), ("bias", (D,)), ("state", final.shape))}
    b0 = np.zeros(D) if bias is None else bias
    for b in range(Bn):
        n = T if lengths is None else int(min(max(lengths[b], 0), T))
        xs = np.concatenate([np.zeros((K - 1, D)) if state is None else state[b], x[b, :n]])
        final[b] = xs[n:]
        dxs, dxm = np.zeros_like(xs), np.zeros_like(xs)
        if dfinal is not None:
            dxs[n:] += dfinal[b]
            dxm[n:] += np.abs(dfinal[b])
        for t in range(n):
            p = b0 + (w.T * xs[t:t + K]).sum(0)
            pm = np.abs(b0) + np.abs(w.T * xs[t:t + K]).sum(0)
            s = sigmoid(p)
            y[b, t] = p * s if silu else p
            # |silu'| <= 1.1, and the sigmoid's own error grows with |p|
            ym[b, t] = 1.1 * pm + np.abs(p * s) * (2 + np.abs(p)) if silu else pm
            if dy is None:
                continue
            d = dy[b, t] * (s * (1 + p * (1 - s)) if silu else 1.0)
            # |silu''| <= 1/2; the sigmoid's error as above, times the terms it is in
            dm = np.abs(dy[b, t]) * (0.5 * pm + (2 + np.abs(p)) * s * (1 + np.abs(p) * (2 - s))
                                     if silu else 1.0)
            dm = np.maximum(dm, np.abs(d))
            dxs[t:t + K] += d * w.T
            dxm[t:t + K] += dm * np.abs(w.T)
            g["weight"][0] += (d * xs[t:t + K]).T
            g["weight"][1] += (dm * np.abs(xs[t:t + K])).T
            g["bias"][0] += d
            g["bias"][1] += dm
        g["state"][0][b], g["x"][0][b, :n] = dxs[:K - 1], dxs[K - 1:]
        g["state"][1][b], g["x"][1][b, :n] = dxm[:K - 1], dxm[K - 1:]
    return {"y": (y, ym), "final": (final, np.abs(final)), "grads": g}


# ------------------------------------------------------------------ scan
def scan(u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths, dy=None, dfinal=None):
    """float64 arrays, B and C (batch, T, groups, N). {name: (value, magnitude)}."""
    Bn, T, Dm = u.shape
    G, N = B.shape[2:]
    grp = np.arange(Dm) // (Dm // G)
    names = {"u": u.shape, "dt": u.shape, "z": u.shape, "A": A.shape, "B": B.shape, "C": C.shape,
             "D": (Dm,), "dt_bias": (Dm,), "state": (Bn, Dm, N)}
    g = {k: [np.zeros(s), np.zeros(s)] for k, s in names.items()}
    y, ym = np.zeros(u.shape), np.zeros(u.shape)
    final, finalm = np.zeros((Bn, Dm, N)), np.zeros((Bn, Dm, N))
    Dd = np.zeros(Dm) if D is None else D
    bias = np.zeros(Dm) if dt_bias is None else dt_bias
    for b in range(Bn):
        n = T if lengths is None else int(min(max(lengths[b], 0), T))
        h = np.zeros((Dm, N)) if state is None else state[b].copy()
        hm = np.abs(h)
        hs, hms = [h], [hm]
        kept = []
        for t in range(n):
            raw = dt[b, t] + bias
            delta = np.logaddexp(raw, 0.0) if softplus else raw
            x = delta[:, None] * A
            a = np.exp(x)
            a[a < 2.0 ** -126] = 0.0  # by definition: such a decay is zero
            # the exponential's error grows with its argument
            am = a * (1 + np.abs(x))
            Bt, Ct = B[b, t][grp], C[b, t][grp]
            h = a * h + (delta * u[b, t])[:, None] * Bt
            hm = am * hm + np.abs((delta * u[b, t])[:, None] * Bt)
            hs.append(h)
            hms.append(hm)
            v = (Ct * h).sum(1) + Dd * u[b, t]
            vm = (np.abs(Ct) * hm).sum(1) + np.abs(Dd * u[b, t])
            zt = None if z is None else z[b, t]
            gate = 1.0 if z is None else zt * sigmoid(zt)
            gm = 1.0 if z is None else np.abs(gate) * (3 + np.abs(zt))
            y[b, t], ym[b, t] = v * gate, vm * gm
            kept.append((raw, delta, a, am, Bt, Ct, v, vm, gate, gm, zt))
        final[b], finalm[b] = h, hm
        if dy is None:
            continue
        back = np.zeros((Dm, N)) if dfinal is None else dfinal[b].copy()
        backm = np.abs(back)

        def add(name, at, v, m):
            g[name][0][at] += v
            g[name][1][at] += m

        for t in range(n - 1, -1, -1):
            raw, delta, a, am, Bt, Ct, v, vm, gate, gm, zt = kept[t]
            ut, d, da = u[b, t], dy[b, t], np.abs(delta)
            if z is not None:
                s = sigmoid(zt)
                add("z", (b, t), d * v * (s * (1 + zt * (1 - s))),
                    np.abs(d) * vm * s * (1 + np.abs(zt) * (2 - s)) * (3 + np.abs(zt)))
            p, pm = d * gate, np.abs(d) * gm
            gg, ggm = back + Ct * p[:, None], backm + np.abs(Ct) * pm[:, None]
            q, qm = gg * a * hs[t], ggm * am * hms[t]
            for k in range(G):
                m = grp == k
                add("C", (b, t, k), (p[:, None] * hs[t + 1])[m].sum(0),
                    (pm[:, None] * hms[t + 1])[m].sum(0))
                add("B", (b, t, k), (gg * (delta * ut)[:, None])[m].sum(0),
                    (ggm * np.abs(delta * ut)[:, None])[m].sum(0))
            gB, gBm = (gg * Bt).sum(1), (ggm * np.abs(Bt)).sum(1)
            add("u", (b, t), gB * delta + Dd * p, gBm * da + np.abs(Dd) * pm)
            add("A", slice(None), q * delta[:, None], qm * da[:, None])
            add("D", slice(None), p * ut, pm * np.abs(ut))
            dd = ((q * A).sum(1) + gB * ut) * (sigmoid(raw) if softplus else 1.0)
            ddm = (qm * np.abs(A)).sum(1) + gBm * np.abs(ut)
            if softplus:
                ddm = ddm * sigmoid(raw) * (3 + np.abs(raw))
            add("dt", (b, t), dd, ddm)
            add("dt_bias", slice(None), dd, ddm)
            back, backm = gg * a, ggm * am
        g["state"][0][b], g["state"][1][b] = back, backm
    return {"y": (y, ym), "final": (final, finalm), "grads": g}
