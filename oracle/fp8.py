"""Oracle of the 8-bit floating point operators in NumPy: e4m3 codes, block quantisers, the
block-scaled linear layer, routing to experts and the experts' gated products, in fp64.

Codes are decided in fp32 as the library's contract says (fl32 steps written out); sums and
scores are fp64. `*_scale` functions give the sums of magnitudes that error bounds refer to.
"""
import numpy as np

BLOCK = 128
FLOOR = np.float32(2.0 ** -100)


def _e4m3_table():
    v = np.empty(256, dtype=np.float64)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            mag = np.nan
        v[c] = -mag if c & 128 else mag
    return v


E4M3 = _e4m3_table()
_POS = E4M3[:127]                                  # 0 .. 448, rising


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    return E4M3[codes]


def e4m3_codes(t: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code of |t| < 464 (round to nearest, ties to the even code); NaN -> 0x7F."""
    t = np.asarray(t, dtype=np.float64)
    a = np.abs(np.nan_to_num(t))
    hi = np.searchsorted(_POS, a, side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.signbit(t), code + 128, code)
    return np.where(np.isnan(t), 0x7F, code).astype(np.uint8)


def _pad(a, axis):
    n = -a.shape[axis] % BLOCK
    width = [(0, 0)] * a.ndim
    width[axis] = (0, n)
    return np.pad(a, width)


def _codes_and_scales(blocks, axes):
    """blocks fp32 [..]; one scale over `axes`."""
    with np.errstate(all="ignore"):
        a = np.maximum(np.abs(blocks).max(axis=axes, keepdims=True), FLOOR).astype(np.float32)
        r = (np.float32(448) * (np.float32(1) / a)).astype(np.float32)
        t = (blocks * r).astype(np.float32)
        return e4m3_codes(t), (a / np.float32(448)).astype(np.float32), t


def silu_mul(v: np.ndarray) -> np.ndarray:
    """[M, 2 K] = [gate | up] -> silu(gate) * up in fp64."""
    g, u = np.split(v.astype(np.float64), 2, axis=1)
    with np.errstate(all="ignore"):
        return g / (1 + np.exp(-g)) * u


def quant_act(v: np.ndarray):
    """v [M, K] -> codes uint8 [M, K], scales fp32 [ceil(K/128), M], the scaled values fp32."""
    M, K = v.shape
    b = _pad(v.astype(np.float32), 1).reshape(M, -1, BLOCK)
    c, s, t = _codes_and_scales(b, 2)
    return c.reshape(M, -1)[:, :K], np.ascontiguousarray(s[:, :, 0].T), t.reshape(M, -1)[:, :K]


def quant_weight(W: np.ndarray):
    """W fp32 [N, K] -> codes uint8 [N, K], scales fp32 [ceil(N/128), ceil(K/128)]."""
    N, K = W.shape
    p = _pad(_pad(W.astype(np.float32), 0), 1)
    b = p.reshape(p.shape[0] // BLOCK, BLOCK, p.shape[1] // BLOCK, BLOCK)
    c, s, _ = _codes_and_scales(b, (1, 3))
    return c.reshape(p.shape)[:N, :K], s[:, 0, :, 0]


def act_values(codes, scales):
    return e4m3_values(codes) * np.repeat(scales.T.astype(np.float64), BLOCK, 1)[:, : codes.shape[1]]


def weight_values(codes, scales):
    N, K = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, 0)[:N], BLOCK, 1)[:, :K]
    return e4m3_values(codes) * s


def linear(codes, scales, wcodes, wscales):
    """-> y fp64 [M, N] and sum_k |x w|."""
    x, w = act_values(codes, scales), weight_values(wcodes, wscales)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def route(logits, k, bias=None, score="softmax", groups=1, kept=1, renorm=True, factor=1.0):
    """-> weight fp64 [M, k], index int [M, k] and the least gap between two different choice
    values of one row (inf where there is none): below the rounding of the scores the choice
    would not be decided."""
    M, E = logits.shape
    weight, index = np.zeros((M, k)), np.full((M, k), -1)
    gap = np.inf
    big = np.finfo(np.float32).max
    for m in range(M):
        l = logits[m].astype(np.float64)
        ok = l > -np.inf                           # False for NaN
        l = np.minimum(np.where(ok, l, -np.inf), big)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                p = 1 / (1 + np.exp(-l))
            c = p.copy()
        else:
            e = np.exp(l - l[ok].max()) * ok if ok.any() else np.zeros(E)
            p = e / e.sum() if ok.any() else e
            c = l.copy() if bias is None else p.copy()
        if bias is not None:
            c = c + bias.astype(np.float64)
        c = np.where(ok, c, -np.inf)
        u = np.unique(c[c > -np.inf])
        if u.size > 1:
            gap = min(gap, np.diff(u).min())
        if groups > 1:
            cg = c.reshape(groups, -1)
            top = -np.sort(-cg, axis=1)[:, :2]
            rank = top[:, 0].copy()
            if score == "sigmoid" and top.shape[1] > 1:
                rank = np.where(top[:, 1] > -np.inf, top[:, 0] + np.where(top[:, 1] > -np.inf, top[:, 1], 0), rank)
            best = sorted(range(groups), key=lambda i: (-rank[i], i))[:kept]
            ur = np.unique(rank[rank > -np.inf])
            if ur.size > 1:
                gap = min(gap, np.diff(ur).min())
            for i in range(groups):
                if i not in best:
                    cg[i] = -np.inf
            c = cg.reshape(-1)
        order = sorted((e for e in range(E) if c[e] > -np.inf), key=lambda e: (-c[e], e))[:k]
        index[m, : len(order)] = order
        weight[m, : len(order)] = p[order]
    if renorm:
        total = weight.sum(1, keepdims=True)
        weight = np.divide(weight, total, out=np.zeros_like(weight), where=total > 0)
    return weight * factor, index, gap


def experts(x, index, weight, wgu, sgu, wd, sd, rel):
    """x [M, H]; codes and scales as the library takes them. `rel`: relative error allowed in
    silu(gate) * up before its quantisation. -> y fp64 [M, H] and a bound on how far a result
    may be from it when every sum is right within `rel` of its magnitudes: codes of
    silu(gate) * up that lie within the allowed error of a rounding boundary may be the
    neighbouring code."""
    M, H = x.shape
    y, bound = np.zeros((M, H)), np.zeros((M, H))
    xc, xs, _ = quant_act(x)
    for m in range(M):
        for j in range(index.shape[1]):
            e = index[m, j]
            if not 0 <= e < wgu.shape[0]:
                continue
            gu, mag = zip(*(linear(xc[m:m + 1], xs[:, m:m + 1], wgu[e, i], sgu[e, i]) for i in (0, 1)))
            h = silu_mul(np.concatenate(gu, 1))
            # silu's slope is at most 1.1, |silu(g)| <= |g|
            dh = rel * (1.1 * mag[0] * np.abs(gu[1]) + np.abs(gu[0]) * mag[1] + 4 * np.abs(h))
            hc, hs, _ = quant_act(h)
            s = np.repeat(hs.T.astype(np.float64), BLOCK, 1)[:, : h.shape[1]]
            worst = np.repeat(_pad(dh, 1).reshape(1, -1, BLOCK).max(2), BLOCK, 1)[:, : h.shape[1]]
            t = np.abs(h) / s
            dt = (dh + worst) / s + 1e-6 * t       # the value's own error, its block maximum's, fl32 steps
            lo, hi = e4m3_values(e4m3_codes(np.maximum(t - dt, 0))), e4m3_values(e4m3_codes(np.minimum(t + dt, 448)))
            val = act_values(hc, hs)
            w = weight_values(wd[e], sd[e])
            dv = (hi - lo) * s + np.abs(val) * (worst / np.maximum(448 * s, 1e-300) + 1e-6)
            y[m] += weight[m, j] * (val @ w.T)[0]
            bound[m] += abs(weight[m, j]) * ((dv + rel * np.abs(val)) @ np.abs(w).T)[0]
    return y, bound
