"""The operators around the expert layer in float64 NumPy, for the tests: written
from the formulas, sharing nothing with the package.  The joint's functions also
give the bounds within which sums and roundings of 32 bits stay."""
import numpy as np

U = 2.0 ** -24
# additions in a row behind a sum over columns: a lane's 32, five shuffles, 16 warps
D = 53


def inv_rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def joint(x, y, after, gate, before, a, b, eps):
    """(h, r) and their bounds before the rounding to the output's type."""
    if y is None:
        h, eh = x, np.zeros_like(x)
    else:
        n = y * inv_rms(y, eps) * after if after is not None else y
        t = b * (n if gate is None else gate * n)
        h = a * x + t
        eh = (D / 2 + 10) * U * np.abs(t) + 2 * U * (np.abs(a * x) + np.abs(t))
    if before is None:
        return h, None, eh, None
    ih = inv_rms(h, eps)
    r = h * ih * before
    # through the mean: by Cauchy-Schwarz no more than |eh| / |h| of every element
    size = np.sqrt((h * h).sum(1, keepdims=True))
    through = np.sqrt((eh * eh).sum(1, keepdims=True)) / np.where(size > 0, size, 1.0)
    return h, r, eh, np.abs(ih * before) * eh + np.abs(r) * (through + (D / 2 + 6) * U)


def joint_grad(dr, dh, h, y, after, gate, before, a, b, eps):
    """Gradients as a dict name -> (value, bound); sums over rows are left to
    :func:`row_sum` (values of each row under the sums' names)."""
    out = {}
    g = np.zeros_like(h) if dh is None else dh
    eg = np.zeros_like(h)
    mag = np.abs(g)
    if before is not None:
        ih = inv_rms(h, eps)
        u = dr * before
        back = h * ih ** 3 * (u * h).mean(1, keepdims=True)
        g = g + ih * u - back
        mag = mag + np.abs(ih * u) + np.abs(h) * ih ** 3 * np.abs(u * h).mean(1, keepdims=True)
        eg = (2.5 * D + 12) * U * mag
        t = dr * h * ih
        out["dbefore"] = (t, (D / 2 + 6) * U * np.abs(t))
    out["dx"] = (a * g, np.abs(a) * (eg + U * np.abs(g)))
    if y is None:
        return out
    g, eg = b * g, np.abs(b) * (eg + U * np.abs(g))
    iy = inv_rms(y, eps) if after is not None else None
    n = y * iy * after if after is not None else y
    if gate is not None:
        out["dgate"] = (g * n, eg * np.abs(n) + (D / 2 + 8) * U * np.abs(g * n))
        g, eg = g * gate, np.abs(gate) * eg + U * np.abs(g * gate)
    if after is not None:
        t = g * y * iy
        out["dafter"] = (t, eg * np.abs(y * iy) + (D / 2 + 6) * U * np.abs(t))
        w, ew = g * after, np.abs(after) * eg + U * np.abs(g * after)
        g = iy * w - y * iy ** 3 * (w * y).mean(1, keepdims=True)
        eg = iy * ew + np.abs(y) * iy ** 3 * (ew * np.abs(y)).mean(1, keepdims=True) + (2.5 * D + 12) * U * (
            np.abs(iy * w) + np.abs(y) * iy ** 3 * np.abs(w * y).mean(1, keepdims=True))
    out["dy"] = (g, eg)
    return out


def row_sum(value, bound):
    """Sums over rows: a group's rows, 16 groups, a slice's 32 parts, eight slices."""
    depth = value.shape[0] / 100 + 64
    return value.sum(0), bound.sum(0) + depth * U * np.abs(value).sum(0)


def choose(z, k, mask, renormalize):
    """(idx, w, counts, losses, p, lse, live)."""
    t, e = z.shape
    idx, w = np.full((t, k), -1, np.int64), np.zeros((t, k))
    p, lse, live = np.zeros((t, e)), np.zeros(t), np.zeros(t, bool)
    counts = np.zeros(e + 1, np.int64)
    for i in range(t):
        if mask is not None and not mask[i] or (z[i] == -np.inf).all():
            continue
        live[i] = True
        counts[e] += 1
        if not (z[i] < np.inf).all():            # NaN or +inf
            w[i], p[i], lse[i] = np.nan, np.nan, np.nan
            continue
        top = z[i].max()
        ex = np.exp(z[i] - top)
        lse[i] = top + np.log(ex.sum())
        p[i] = ex / ex.sum()
        by = sorted((j for j in range(e) if z[i, j] > -np.inf), key=lambda j: (-z[i, j], j))[:k]
        idx[i, :len(by)] = by
        w[i, :len(by)] = ex[by] / (ex[by].sum() if renormalize else ex.sum())
        counts[by] += 1
    n = max(1, counts[e])
    f, mean = counts[:e] / (k * n), p[live].sum(0) / n
    losses = np.array([e * (f * mean).sum(), (lse[live] ** 2).sum() / n])
    return idx, w, counts, losses, p, lse, live


def choose_grad(z, idx, counts, dw, dlosses, mask, renormalize):
    """The gradient for the logits and the sum of its terms' magnitudes."""
    t, e = z.shape
    k = idx.shape[1]
    _, _, _, _, p, lse, live = choose(z, k, mask, renormalize)
    dz, mag = np.zeros((t, e)), np.zeros((t, e))
    n = max(1, counts[e])
    for i in np.nonzero(live)[0]:
        if np.isnan(lse[i]):
            dz[i] = np.nan
            continue
        if dw is not None:
            d, part = np.zeros(e), np.zeros(e, bool)
            for s in range(k):
                if 0 <= idx[i, s] < e:
                    d[idx[i, s]] += dw[i, s]
                    part[idx[i, s]] = True
            wt = p[i]
            if renormalize:
                total = (p[i] * part).sum()
                wt = p[i] * part / total if total > 0 else np.zeros(e)
            dot, adot = (wt * d).sum(), (wt * np.abs(d)).sum()
            dz[i] += wt * (d - dot)
            mag[i] += wt * (np.abs(d) + adot)
        if dlosses is not None:
            c = counts[:e]
            f0, f1 = dlosses[0] * e / (k * n * n), dlosses[1] * 2 / n
            dz[i] += f0 * p[i] * (c - (p[i] * c).sum()) + f1 * lse[i] * p[i]
            mag[i] += np.abs(f0) * p[i] * (c + (p[i] * c).sum()) + np.abs(f1 * lse[i]) * p[i]
    return dz, mag
