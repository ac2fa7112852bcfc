"""Plain references in 64 bits of the operators around a decode step's products: sampling, head norms with rotation, experts."""
import numpy as np


def prefix_order(x):
    """Ids of one row in descending order, equal logits (+0 and -0 too) by the lower id."""
    return np.lexsort((np.arange(x.size), -(x.astype(np.float64) + 0.0)))


def sample(x, noise, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The ids that a row may give: one, but for draws closer than float32 sums and 64-bit scores can tell.  A top-p border
    may lie 2^-20 of the mass to either side (the weights' approximation, 2^-22 each, and their integers)."""
    n = x.size
    x64 = x.astype(np.float64)
    if np.isnan(x).any() or np.isneginf(x).all():
        return {-1}
    order = prefix_order(x)
    if np.isposinf(x).any() or not temperature > 2.0 ** -100 or top_k == 1 or top_p <= 0:
        return {int(order[0])}
    z = (x64 - x64[order[0]]) / np.float64(temperature)
    w = np.exp(z)
    ws = w[order]
    kept_k = top_k if 0 < top_k < n else n
    found = set()
    for slack in (-(2.0 ** -20), 0.0, 2.0 ** -20):
        for m_slack in (-(2.0 ** -20), 0.0, 2.0 ** -20):
            keep = np.arange(n) < kept_k
            if top_p < 1:
                mass = np.where(keep, ws, 0.0)
                before = np.cumsum(mass) - mass
                keep &= before < np.float64(top_p) * mass.sum() * (1 + slack)
                keep[0] = True
            if min_p > 0:
                keep &= ws >= min(np.float64(min_p), 1.0) * (1 + m_slack if min_p < 1 else 1.0)
                keep[0] = True
            ids = order[keep]
            ids = ids[(noise[ids] > 0) & (ws[keep] > 0) & ~np.isneginf(x[ids])]
            if ids.size == 0:
                found.add(int(order[0]))
                continue
            with np.errstate(divide="ignore"):
                s = z[ids] - np.log(noise[ids].astype(np.float64))
            best = s.max()
            if not np.isfinite(best):
                found.add(int(order[0]))
                continue
            near = ids[s >= best - 2.0 ** -40 * max(1.0, abs(best))]
            found.add(int(near.min()))
    return found


def qk_rope(x, weight, eps, pos, freq, halves, factor=1.0):
    """x (rows, heads, dim) in 64 bits, normed and turned; and |a| + |b| of each value's pair (|s| for the others)."""
    s = x.astype(np.float64)
    if weight is not None:
        s = s / np.sqrt((s ** 2).mean(axis=2, keepdims=True) + eps) * weight.astype(np.float64)
    y, mag = s.copy(), np.abs(s)
    if freq is None:
        return y, mag
    half = freq.size
    t = pos.astype(np.longdouble)[:, None, None] * freq.astype(np.longdouble)  # 64 bits are too few for 2^31 * 100 radians
    cos, sin = np.cos(t).astype(np.float64), np.sin(t).astype(np.float64)
    ia = np.arange(half) if halves else 2 * np.arange(half)
    ib = ia + half if halves else ia + 1
    a, b = s[..., ia], s[..., ib]
    y[..., ia] = (a * cos - b * sin) * factor
    y[..., ib] = (a * sin + b * cos) * factor
    mag[..., ia] = mag[..., ib] = (np.abs(a) + np.abs(b)) * abs(factor)
    return y, mag


def act(name, g):
    if name == "silu":
        with np.errstate(over="ignore"):
            return g / (1 + np.exp(-g))
    return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def moe(w1, w3, w2, x, logits, top, renorm, scale, name, parts):
    """w1, w3 (experts, hidden, dim), w2 (experts, dim, hidden) float32 values; x (tokens, dim); in 64 bits.  Returns out, its bound
    before the output's own rounding, ids and shares.

    Bound.  A product's sum of n terms: blocks of 32 on the tensor core, then n / 32 float32 additions, each at most 2^-23 of
    the sum of magnitudes A (whatever the rounding inside an MMA): (n / 32 + 40) 2^-23 A; x itself in 22 bits (2^-22 A).  h = act(g) u:
    |dh| <= 1.13 |u| dg + |act(g)| du (the slope of either activation is below 1.13) + 2^-20 (1 + |g|) |h| for the float32 functions, and
    its halves' rounding, 2^-11 |h| for one and 2^-22 for two, or 2^-35 of the largest where that is more (a block's second half keeps four bits fewer of its small values).  The shares: 2^-20 relative (exponentials, sums, a quotient), and the
    difference of a logit and the maximum, d, rounded to float32: e^(d (1 + 2^-24)) is off by |d| 2^-24.  The shares' relative bound is
    the fifth result."""
    tokens, experts = logits.shape
    dim, hidden = w2.shape[1], w2.shape[2]
    out, bound = np.zeros((tokens, dim)), np.zeros((tokens, dim))
    ids, shares, share_rel = np.full((tokens, top), -1, np.int32), np.zeros((tokens, top)), np.zeros((tokens, top))
    for t in range(tokens):
        l = logits[t].astype(np.float64)
        if np.isnan(l).any() or np.isposinf(l).any():
            out[t] = np.nan
            shares[t] = np.nan
            continue
        order = [e for e in prefix_order(logits[t]) if not np.isneginf(l[e])][:top]
        if not order:
            continue
        m = l[order[0]]
        p = np.exp(l - m)
        p = p[order] / (p[order].sum() if renorm else p.sum())
        ids[t, :len(order)], shares[t, :len(order)] = order, p
        rel = 2.0 ** -20 + (m - l[order]) * 2.0 ** -24
        share_rel[t, :len(order)] = rel
        xt = x[t].astype(np.float64)
        for e, pe, re in zip(order, p, rel):
            g, u = w1[e].astype(np.float64) @ xt, w3[e].astype(np.float64) @ xt
            ga, ua = np.abs(w1[e].astype(np.float64)) @ np.abs(xt), np.abs(w3[e].astype(np.float64)) @ np.abs(xt)
            c = (dim / 32 + 42) * 2.0 ** -23
            h = act(name, g) * u
            dh = (1.13 * np.abs(u) * c * ga + np.abs(act(name, g)) * c * ua + 1.13 * c * c * ga * ua +
                  (2.0 ** -20 * (1 + np.abs(g)) + (2.0 ** -11 if parts == 1 else 2.0 ** -22)) * np.abs(h) + 2.0 ** -35 * np.abs(h).max() + 1e-33)
            a2 = np.abs(w2[e].astype(np.float64))
            out[t] += pe * scale * (w2[e].astype(np.float64) @ h)
            bound[t] += pe * abs(scale) * (a2 @ dh + ((hidden / 32 + 40) * 2.0 ** -23 + re) * (a2 @ np.abs(h)))
    return out, bound, ids, shares, share_rel
