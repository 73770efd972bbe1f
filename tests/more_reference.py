"""Plain 64-bit evaluation of layer norm, gated scan and sampling (test
infrastructure), with an error bound beside each number.

A bound is what binary32 arithmetic may be off by: the roundings of each
operation, 2^-24 of its result, carried through the formulas. ``near`` adds the
rounding of the stored result."""
import numpy as np

from .model_reference import STORE, f64

U = 2.0 ** -24


def sigmoid(v):
    """With its digits where it is small, too."""
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-v))


def near(got, want, bound, what=""):
    """|got - want| <= store * (|want| + bound) + bound, elementwise."""
    rel, tiny = STORE[got.dtype]
    g = f64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    assert np.isfinite(g).all(), what
    tol = rel * (np.abs(want) + bound) + bound + tiny
    bad = np.abs(g - want) > tol
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(g - want) / tol), g.shape)
        raise AssertionError("%s: %d of %d off, worst at %s: got %r want %r tol %r" % (
            what, bad.sum(), bad.size, i, g[i], want[i], tol[i]))


def _sum_steps(n):
    """Roundings of a sum of n terms: 32 or n / 1024 of them in a row, and trees."""
    return 16 + min(n, 32 + n // 32)


def norm(x, w, b, eps, dy=None):
    """x (..., D) as float64 arrays. Returns {name: (value, bound)}."""
    D = x.shape[-1]
    x2 = x.reshape(-1, D)
    mean = x2.mean(1, keepdims=True) if D else np.zeros((len(x2), 1))
    d = x2 - mean
    rstd = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    n = d * rstd
    k = _sum_steps(D) * U
    # n: the mean's error is k of the mean distance (the sum of what is left of
    # it after its first rounding, whose own error is k^2 of the mean size), the
    # square root halves the sum of squares' k; a few roundings of its own
    size = np.abs(d).mean(1, keepdims=True) + k * np.abs(x2).mean(1, keepdims=True)
    en = (2 * k + 8 * U) * (np.abs(n) + size * rstd)
    wv = np.ones(D) if w is None else w
    bv = np.zeros(D) if b is None else b
    out = {"y": (n * wv + bv, en * np.abs(wv) + 2 * U * (np.abs(n * wv) + np.abs(bv)))}
    if dy is not None:
        dy2 = dy.reshape(-1, D)
        g = dy2 * wv
        s1, s2 = g.mean(1, keepdims=True), (g * n).mean(1, keepdims=True)
        a1, a2 = np.abs(g).mean(1, keepdims=True), np.abs(g * n).mean(1, keepdims=True)
        e1 = k * a1 + U * a1
        e2 = (k + 4 * U) * a2 + (np.abs(g) * en).mean(1, keepdims=True)
        dx = rstd * (g - s1 - n * s2)
        mag = np.abs(g) + a1 + np.abs(n) * a2
        ex = rstd * (8 * U * mag + e1 + np.abs(n) * e2 + en * np.abs(s2)) + k * np.abs(dx)
        R = len(x2)
        kr = (16 + min(R, 512 + R // 256)) * U
        out["x"] = dx, ex
        out["weight"] = (dy2 * n).sum(0), (kr * np.abs(dy2 * n) + np.abs(dy2) * en).sum(0)
        out["bias"] = dy2.sum(0), kr * np.abs(dy2).sum(0)
    return {q: tuple(t.reshape(x.shape) if q in ("x", "y") else t for t in v)
            for q, v in out.items()}


def gated(x, gate, z, state, lengths, dy=None, dfinal=None):
    """x (B, T, D) etc. as float64 arrays. Returns {name: (value, bound)}, the
    gradients under "d" + name.

    r = 1 - a is off by K roundings of itself (the exponent's, |gate| / 2 and
    one, the instruction's two and a half, the reciprocal's two). A step is two
    operations, h - r h and + r x, whose roundings are of results up to |h| and
    up to the new state; a tile's map, applied the same way, rounds what it
    starts from once more."""
    Bn, T, D = x.shape
    K = (8 + np.abs(np.where(np.isfinite(gate), gate, 0))) * U
    a, r = sigmoid(gate), sigmoid(-gate)
    h, hm, he = (np.zeros((Bn, T + 1, D)) for _ in range(3))
    if state is not None:
        h[:, 0], hm[:, 0] = state, np.abs(state)
    n = [T] * Bn if lengths is None else [int(min(max(v, 0), T)) for v in lengths]
    y, ye = np.zeros((Bn, T, D)), np.zeros((Bn, T, D))
    final, fe = np.zeros((Bn, D)), np.zeros((Bn, D))
    g = {q: [np.zeros((Bn, T, D)), np.zeros((Bn, T, D))] for q in ("dx", "dgate", "dz")}
    ds, dse = np.zeros((Bn, D)), np.zeros((Bn, D))
    for b in range(Bn):
        for t in range(n[b]):
            at, rt, xt = a[b, t], r[b, t], np.abs(x[b, t])
            h[b, t + 1] = at * h[b, t] + rt * x[b, t]
            hm[b, t + 1] = at * hm[b, t] + rt * xt
            he[b, t + 1] = at * he[b, t] + 4 * (U * (hm[b, t + 1] + at * hm[b, t]) +
                                                K[b, t] * rt * (xt + hm[b, t]))
        m = n[b]
        final[b], fe[b] = h[b, m], he[b, m]
        zb = None if z is None else z[b, :m]
        s = None if z is None else sigmoid(zb)
        silu = 1.0 if z is None else zb * s
        kz = 0.0 if z is None else (10 + np.abs(zb)) * U  # of silu and of its slope
        y[b, :m] = h[b, 1:m + 1] * silu
        ye[b, :m] = np.abs(silu) * (he[b, 1:m + 1] + (kz + 2 * U) * hm[b, 1:m + 1])
        if dy is None:
            continue
        dyb = dy[b, :m]
        if z is not None:
            slope, sm = s * (1 + zb * (1 - s)), s * (1 + np.abs(zb) * (1 - s))
            g["dz"][0][b, :m] = dyb * h[b, 1:m + 1] * slope
            g["dz"][1][b, :m] = np.abs(dyb) * sm * (he[b, 1:m + 1] +
                                                    (kz + 4 * U) * hm[b, 1:m + 1])
        G = np.zeros(D) if dfinal is None else dfinal[b].copy()
        Gm, Ge = np.abs(G), np.zeros(D)
        for t in range(m - 1, -1, -1):
            e = dyb[t] * (1.0 if z is None else silu[t])
            G = G + e
            Gm = Gm + np.abs(e)
            Ge = Ge + 4 * U * Gm + (0.0 if z is None else 4 * kz[t]) * np.abs(e)
            at, rt, kt = a[b, t], r[b, t], K[b, t]
            g["dx"][0][b, t] = rt * G
            g["dx"][1][b, t] = rt * Ge + (kt * rt + 4 * U * rt) * Gm
            d, dm = h[b, t] - x[b, t], hm[b, t] + np.abs(x[b, t])
            g["dgate"][0][b, t] = d * G * at * rt
            g["dgate"][1][b, t] = at * rt * (dm * Ge + he[b, t] * Gm + (2 * kt + 8 * U) * dm * Gm)
            Ge = at * Ge + 4 * (kt * rt + 2 * U * at) * Gm
            G, Gm = at * G, at * Gm
        ds[b], dse[b] = G, Ge
    out = {"y": (y, ye), "final": (final, fe)}
    if dy is not None:
        out.update({q: tuple(v) for q, v in g.items()})
        out["dstate"] = ds, dse
    return out


def sample(logits, u, temperature, top_k, top_p, min_p):
    """logits (rows, V); settings one a row. The definition, row by row."""
    out = []
    for r in range(logits.shape[0]):
        x = logits[r]
        ids = np.flatnonzero(x > -np.inf)  # NaN is not
        if not len(ids):
            out.append(-1)
            continue
        ids = ids[np.argsort(-x[ids], kind="stable")]
        if top_k[r] > 0:
            ids = ids[:int(top_k[r])]
        if not temperature[r] > 0:
            out.append(int(ids[0]))
            continue
        top = x[ids[0]]
        with np.errstate(invalid="ignore"):
            w = np.where(x[ids] == top, 1.0, np.exp((x[ids] - top) / temperature[r]))
        before = np.concatenate([[0.0], np.cumsum(w)])
        keep = np.ones(len(ids), bool)
        if top_p[r] < 1:
            keep &= before[:-1] < max(top_p[r], 0) * before[-1]
        if min_p[r] > 0:
            keep &= w >= min_p[r]
        keep[0] = True
        m = int(keep.sum())  # a first part
        uu = min(max(u[r], 0.0), 1 - 2.0 ** -24) if u[r] == u[r] else 0.0
        at = int((before[1:m + 1] <= uu * before[m]).sum())
        live = int((w[:m] > 0).sum())
        out.append(int(ids[min(at, live - 1)]))
    return np.array(out)
