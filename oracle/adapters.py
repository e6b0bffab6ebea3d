"""Oracle of what is trained beside frozen weights, in NumPy and fp64: low-rank adapters and their
gradients, the experts' balance loss, and the gradient of the router's logits.

Results come with the sums of magnitudes that error bounds refer to.
"""
import numpy as np


def _rows(index, L):
    return [(e, np.flatnonzero(index == e)) for e in range(L)]


def forward(x, a, b, index, scale, base):
    """(y, h, magnitudes of y's sum without base, magnitudes of h)."""
    x, a, b, base = (np.asarray(t, np.float64) for t in (x, a, b, base))
    M, R = x.shape[0], a.shape[1]
    y, mag = base.copy(), np.zeros_like(base)
    h, hmag = np.zeros((M, R)), np.zeros((M, R))
    for e, rows in _rows(index, a.shape[0]):
        if rows.size:
            h[rows], hmag[rows] = x[rows] @ a[e].T, np.abs(x[rows]) @ np.abs(a[e]).T
            y[rows] += scale[e] * (h[rows] @ b[e])
            mag[rows] = abs(scale[e]) * (hmag[rows] @ np.abs(b[e]))
    return y, h, mag, hmag


def backward(x, a, b, index, scale, h, dy, base):
    """({dx, da, db}, the same of magnitudes; dx's without base)."""
    x, a, b, h, dy, base = (np.asarray(t, np.float64) for t in (x, a, b, h, dy, base))
    out = {"dx": base.copy(), "da": np.zeros(a.shape), "db": np.zeros(b.shape)}
    mag = {"dx": np.zeros_like(base), "da": np.zeros(a.shape), "db": np.zeros(b.shape)}
    for e, rows in _rows(index, a.shape[0]):
        if not rows.size:
            continue
        for to, f in ((out, lambda t: t), (mag, np.abs)):
            xe, dye, he, s = f(x[rows]), f(dy[rows]), f(h[rows]), f(np.float64(scale[e]))
            dh = s * (dye @ f(b[e]).T)
            to["dx"][rows] += dh @ f(a[e])
            to["da"][e] = dh.T @ xe
            to["db"][e] = s * (he.T @ dye)
    return out, mag


def scores(logits, score):
    """(p, t) of bl_route_experts' scores and the same divided by their row's sum; NaN and -inf are
    left out, +inf is the largest finite fp32 value. t is found from logarithms, so that no row's
    scores are too small for it."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    ok = l > -np.inf
    with np.errstate(all="ignore"):
        log = l if score == "softmax" else np.where(ok, -np.logaddexp(0, -l), -np.inf)
        top = np.max(log, axis=1, keepdims=True)
        w = np.where(ok, np.exp(log - np.where(np.isfinite(top), top, 0)), 0.0)
        total = w.sum(1, keepdims=True)
        t = np.where(total > 0, w / total, 0.0)
        p = t if score == "softmax" else np.where(ok, np.exp(log), 0.0)
    return p, t


def sequence_of_rows(offsets, M):
    """The sequence of each row; -1 for rows of none."""
    seq = np.full(M, -1)
    for s in range(len(offsets) - 1):
        seq[max(offsets[s], 0):max(min(offsets[s + 1], M), 0)] = s
    return seq


def balance(logits, index, score, offsets=None):
    """(loss [S], count [S, E], coef [S, E])."""
    M, E = logits.shape
    offsets = [0, M] if offsets is None else offsets
    t = scores(logits, score)[1]
    S = len(offsets) - 1
    loss, count, coef = np.zeros(S), np.zeros((S, E), np.int64), np.zeros((S, E))
    seq = sequence_of_rows(offsets, M)
    held = (index >= 0) & (index < E)
    for s in range(S):
        rows = (seq == s) & held.any(1)
        count[s] = np.bincount(index[rows][held[rows]], minlength=E)
        if rows.any():
            coef[s] = E * count[s] / (float(count[s].sum()) * rows.sum())
            loss[s] = (coef[s] * t[rows].sum(0)).sum()
    return loss, count, coef


def route_weights(logits, index, score, renorm, factor):
    """bl_route_experts' weights of a given choice."""
    E = logits.shape[1]
    held = (index >= 0) & (index < E)
    w = np.where(held, np.take_along_axis(scores(logits, score)[0], np.where(held, index, 0), 1), 0.0)
    if renorm:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return factor * w


def route_backward(logits, index, score, renorm, factor, dweight=None, coef=None, dloss=None, offsets=None):
    """(dlogits, magnitudes of its terms). dweight [M, k] or None, coef [S, E] and dloss [S] or None."""
    M, E = logits.shape
    p, t = scores(logits, score)
    held = (index >= 0) & (index < E)
    d, mag = np.zeros((M, E)), np.zeros((M, E))
    slope = 1 - p if score == "sigmoid" else np.ones_like(p)
    if dweight is not None:
        at = np.where(held, index, 0)
        g = np.where(held, factor * np.asarray(dweight, np.float64), 0.0)
        ps = np.where(held, np.take_along_axis(p, at, 1), 0.0)
        if renorm:
            total = ps.sum(1, keepdims=True)
            u = np.divide(ps, total, out=np.zeros_like(ps), where=total > 0)
            v, vm = u * (g - (u * g).sum(1, keepdims=True)), u * (np.abs(g) + (u * np.abs(g)).sum(1, keepdims=True))
        else:
            v, vm = ps * g, ps * np.abs(g)
        rows = np.broadcast_to(np.arange(M)[:, None], at.shape)
        np.add.at(d, (rows[held], at[held]), v[held])
        np.add.at(mag, (rows[held], at[held]), vm[held])
        d, mag = d * slope, mag * slope
        if score == "softmax" and not renorm:
            d -= p * v.sum(1, keepdims=True)
            mag += p * vm.sum(1, keepdims=True)
    if coef is not None:
        seq = sequence_of_rows([0, M] if offsets is None else offsets, M)
        on = (seq >= 0) & held.any(1)
        to = np.where(on, seq, 0)
        c = np.asarray(coef, np.float64)[to] * on[:, None]
        q = np.asarray(dloss, np.float64)[to][:, None] * slope * t
        d += q * (c - (t * c).sum(1, keepdims=True))
        mag += np.abs(q) * (np.abs(c) + (t * np.abs(c)).sum(1, keepdims=True))
    return d, mag
