"""Norm, microscaled formats and sampling from their definitions, in 64 bits on the host: what the tests of these
operators compare with."""
import numpy as np

# name: (largest exponent, values of the codes without sign)
GRIDS = {"fp4": (2, np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])),
         "fp8": (8, np.array([(8 + c % 8 if c >= 8 else c % 8) * 2.0 ** (max(c // 8, 1) - 10) for c in range(127)]))}


def sums(x, delta):
    """The residual's addition: in float32, rounded to x's type."""
    with np.errstate(over="ignore", invalid="ignore"):
        return (x.astype(np.float32) + delta.astype(np.float32)).astype(x.dtype)


def norm(s, weight, eps):
    s = s.astype(np.float64)
    with np.errstate(all="ignore"):
        y = s / np.sqrt((s * s).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
        return y if weight is None else y * weight.astype(np.float64)


def blocks(x):
    return x.reshape(x.shape[:-1] + (-1, 32))


def scales(x, form):
    """Scale bytes of rows [...][cols]."""
    b = np.abs(blocks(x.astype(np.float64)))
    bad = ~np.isfinite(b).all(-1)
    top = np.where(np.isfinite(b), b, 0).max(-1)
    e = np.frexp(top)[1] - 1 - GRIDS[form][0]
    return np.where(bad, 255, np.where(top > 0, np.clip(e, -127, 127) + 127, 0)).astype(np.uint8)


def codes(x, form):
    """Codes (one per element) of rows of finite values, with the scales above."""
    grid = GRIDS[form][1]
    s = scales(x, form).astype(np.int64)
    v = np.ldexp(blocks(x.astype(np.float64)), -(s - 127)[..., None])
    m = np.abs(v)
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, m, "left"), np.searchsorted(mid, m, "right")
    c = np.where(lo % 2 == 0, lo, hi)
    return (c + np.where(np.signbit(v), 128 if form == "fp8" else 8, 0)).reshape(x.shape).astype(np.uint8)


def packed(c, form):
    return c if form == "fp8" else (c[..., 0::2] | c[..., 1::2] << 4).astype(np.uint8)


def unpacked(c, form):
    return c if form == "fp8" else np.stack([c & 15, c >> 4], -1).reshape(c.shape[:-1] + (-1,))


def elements(c, form):
    """Values of codes (one per element), unscaled."""
    grid = np.append(GRIDS[form][1], [np.nan] if form == "fp8" else [])
    half = 128 if form == "fp8" else 8
    return np.where(c >= half, -1.0, 1.0) * grid[c % half]


def values(c, s, form):
    """Values of packed codes and scale bytes."""
    v = blocks(elements(unpacked(c, form), form))
    s = s.astype(np.int64)[..., None]
    with np.errstate(invalid="ignore"):
        return np.where(s == 255, np.nan, np.ldexp(v, np.minimum(s, 254) - 127)).reshape(v.shape[:-2] + (-1,))


def product(a, w, bias, cut=False):
    """The product, and an upper bound of its error by the stated arithmetic: a sum in float32 of parts of eight products,
    at most 40 parts of the whole and the bias, each addition within 2^-24 of the magnitudes' sum, and 2^-20 of that
    sum for the groups inside an instruction (eight products aligned with their largest, 2^-23 of it lost of each).  cut: each
    of eight neighbouring products may lose 2^-13 of their largest besides."""
    k = a.shape[1]
    out, size = a @ w.T, np.abs(a) @ np.abs(w.T)
    if bias is not None:
        out, size = out + bias, size + np.abs(bias)
    tol = size * (2.0 ** -20 + (k // 8 + 41) * 2.0 ** -24)
    if cut:
        a, w = np.abs(a), np.abs(w)
        for i in range(0, k, 8):
            top = np.zeros(out.shape)
            for j in range(i, i + 8):
                np.maximum(top, np.multiply.outer(a[:, j], w[:, j]), out=top)
            tol = tol + 8 * 2.0 ** -13 * top
    return out, tol


def sample(l, u, t=None, k=None, p=None, m=None):
    """(token, prob, kept, gap) of one row; gap: how near the choices came to another outcome, relative to the sums."""
    l = l.astype(np.float64)
    ok = np.flatnonzero(l > -np.inf)                       # (neither -inf nor NaN)
    if not len(ok):
        return -1, 0.0, 0, 1.0
    t = 1.0 if t is None else float(t)
    best = l[ok].max()
    if not t > 0:
        return int(ok[l[ok] == best][0]), 1.0, 1, 1.0
    ids = ok[np.lexsort((ok, -l[ok]))]
    with np.errstate(all="ignore"):
        w = np.where(l[ids] == best, 1.0, 0.0 if best == np.inf else np.exp((l[ids] - best) / t))
    n, gap = len(ids), 1.0
    if k is not None and k > 0:
        n = min(n, int(k))
    if p is not None and p < 1:
        before = np.cumsum(w[:n]) - w[:n]
        total = w[:n].sum()
        kept = max(1, int((before < float(p) * total).sum()))
        edge = np.append(before, total)[[kept - 1, kept]] / total - float(p)
        gap = min(gap, np.abs(edge[np.arange(2) >= (kept == 1)]).min() if kept < n or kept > 1 else 1.0)
        n = kept
    if m is not None and m > 0:
        lim = min(float(m), 1.0)
        gap = min(gap, np.abs(w[:n] - lim)[1:].min() if n > 1 else 1.0)
        n = max(1, int((w[:n] >= lim).sum()))
    order = np.argsort(ids[:n])
    ids, w = ids[:n][order], w[:n][order]
    c = np.cumsum(w)
    x = min(max(float(u), 0.0), np.nextafter(1.0, 0.0)) * c[-1] if u == u else 0.0
    at = min(int(np.searchsorted(c, x, "right")), n - 1)
    if u >= 1:
        at = int(np.flatnonzero(w > 0)[-1])
    elif x > 0:
        gap = min(gap, np.abs(c - x).min() / c[-1])
    return int(ids[at]), w[at] / c[-1], n, gap
