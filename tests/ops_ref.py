"""Plain references of the operators between the products: the rules of the 8-bit cache and norm in
float32 steps (numpy), the attention, norm and log probabilities in 64 bits."""
import numpy as np

F = np.float32


def f32_of_bf16(codes):
    return (np.asarray(codes, np.uint16).astype(np.uint32) << 16).view(np.float32)


def half_step(x):
    """trunc(x + copysign(0.5, x)) in float32."""
    x = np.asarray(x, F)
    return np.trunc((x + np.copysign(F(0.5), x)).astype(F))


def q8_levels(x, inv):
    return np.clip(half_step((x * inv).astype(F)), -127, 127).astype(np.int8)


class Cache:
    """The paged cache as numpy arrays, with the writer's rule applied page by page."""

    def __init__(self, pages, heads, page, dim):
        self.page = page
        self.lev = [np.zeros((pages, heads, page, dim), np.int8) for _ in range(2)]
        self.scale = [np.zeros((pages, heads), F) for _ in range(2)]

    def write(self, table, lens, counts, k, v):
        """k, v: float32 (rows, heads, dim); counts: rows of each sequence."""
        row = 0
        for s, n in enumerate(counts):
            pos, end = lens[s] - n, lens[s]
            while pos < end:
                pid, lo = table[s][pos // self.page], pos % self.page
                m = min(end - pos, self.page - lo)
                for which, x in ((0, k), (1, v)):
                    self._page(which, pid, lo, x[row:row + m])
                pos += m
                row += m

    def _page(self, which, pid, lo, x):
        lev, scale = self.lev[which][pid], self.scale[which][pid]
        for h in range(lev.shape[0]):
            top = F(np.max(np.abs(x[:, h])))
            want = F(0) if top < F(1e-30) else F(top * F(1 / 127))
            had = scale[h] if lo > 0 else F(0)
            d = max(want, had)
            if lo > 0 and d > had:
                lev[h, :lo] = half_step(lev[h, :lo].astype(F) * F(had / d)).astype(np.int8)
            inv = F(F(1) / d) if d > 0 else F(0)
            lev[h, lo:lo + len(x)] = q8_levels(x[:, h], inv)
            scale[h] = d

    def values(self, which, table_row, length):
        """float32 (length, heads, dim)."""
        pages = np.asarray(table_row[: -(-length // self.page)], np.int64)
        x = self.lev[which][pages].astype(F) * self.scale[which][pages][:, :, None, None]
        return np.moveaxis(x, 1, 2).reshape(-1, x.shape[1], x.shape[3])[:length]


def attend(q, k, v, first, scale, causal=True, window=0):
    """One sequence in 64 bits: q (n, heads, dim) at positions first.., k, v (length, kv_heads, dim).
    Returns out, sum_j p_j |v_j|, and max_j scale * sum |q_d k_jd| and max |z| of each row and head."""
    n, heads, dim = q.shape
    length, kvh = k.shape[0], k.shape[1]
    out = np.zeros((n, heads, dim))
    mag = np.zeros((n, heads, dim))
    amp = np.zeros((n, heads))
    pos = first + np.arange(n)[:, None]
    j = np.arange(length)[None, :]
    seen = np.ones((n, length), bool) if not causal else j <= pos
    if window:
        seen = seen & (j > pos - window)
    for h in range(heads):
        g = h // (heads // kvh)
        kk, vv, qq = k[:, g].astype(np.float64), v[:, g].astype(np.float64), q[:, h].astype(np.float64)
        z = np.where(seen, scale * (qq @ kk.T), -np.inf)
        some = seen.any(axis=1)
        m = np.where(some, z.max(axis=1, initial=-np.inf), 0.0)
        p = np.exp(z - m[:, None])
        total = p.sum(axis=1)
        p = p / np.where(some, total, 1.0)[:, None]
        out[:, h] = p @ vv
        mag[:, h] = p @ np.abs(vv)
        amp[:, h] = np.where(seen, abs(scale) * (np.abs(qq) @ np.abs(kk).T), 0.0).max(axis=1, initial=0.0)
    return out, mag, amp


def attend_bound(mag, amp, out, dim, length, bf16):
    """How far qmv_attend may be from 64 bits.  A score's error is a float32 sum of dim products (and
    22 bits of a float32 q): dz <= amp (dim + 8) 2^-23; the weights and their sum each carry it, their own
    rounding (2^-11 as halves, 2^-21 as pairs), and float32 sums over the keys; the output is rounded once."""
    dz = amp * (dim + 8) * 2.0 ** -23
    rel = 2 * dz + (2.0 ** -10 if bf16 else 2.0 ** -20) + (length + 64) * 2.0 ** -24
    return rel[:, :, None] * mag + (2.0 ** -8 * np.abs(out) if bf16 else 0.0) + 1e-30


def half_weights(q, k, v_lev, v_scale, first, scale, causal=True, window=0):
    """What the prompt kernel's rounding to half adds to attend_bound: weights times V scale below 2^-21 of
    the row's largest are multiples of 2^-32 of it, so each key may be off by that times its level.
    v_lev, v_scale: levels (length, kv_heads, dim) and scales (length, kv_heads)."""
    n, heads, dim = q.shape
    length, kvh = k.shape[0], k.shape[1]
    pos, j = first + np.arange(n)[:, None], np.arange(length)[None, :]
    seen = np.ones((n, length), bool) if not causal else j <= pos
    if window:
        seen = seen & (j > pos - window)
    add = np.zeros((n, heads, dim))
    for h in range(heads):
        g = h // (heads // kvh)
        z = np.where(seen, scale * (q[:, h].astype(np.float64) @ k[:, g].astype(np.float64).T), -np.inf)
        p = np.exp(z - z.max(axis=1, keepdims=True))
        w = p / p.sum(axis=1, keepdims=True) * v_scale[:, g].astype(np.float64)
        add[:, h] = 2.0 ** -32 * w.max(axis=1, keepdims=True) * (seen @ np.abs(v_lev[:, g].astype(np.float64)))
    return add


def rmsnorm(x, res, w, eps):
    """64 bits: s, y."""
    s = x.astype(np.float64) + (0.0 if res is None else res.astype(np.float64))
    r = 1.0 / np.sqrt((s ** 2).mean(axis=1, keepdims=True) + eps)
    return s, s * w.astype(np.float64) * r


def logprobs(x):
    """64 bits: log probabilities and entropy of each row (masked ids: -inf, no entropy)."""
    x = x.astype(np.float64)
    m = x.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        none = np.isneginf(m)
        d = np.where(none, -np.inf, x - np.where(none, 0.0, m))
        lz = np.log(np.exp(d).sum(axis=1, keepdims=True))
        lp = np.where(none, -np.inf, d - lz)
        p = np.exp(lp)
        h = -np.where(p > 0, p * lp, 0.0).sum(axis=1)
    return lp, h


def top_ids(x, n):
    """The n largest of each row, equal ones by the lower id."""
    key = np.where(np.isnan(x), np.inf, x) + 0.0
    return np.stack([np.lexsort((np.arange(r.size), -r))[:n] for r in key])


def near_half(inv):
    """The float32 values below half a step (0.5 / inv) whose level depends on the product's own rounding: rounded before the
    half is added it gives 1, in one rounding of the whole 0.  May be empty: about three in ten have one."""
    x = np.full(16, F(np.float64(0.5) / np.float64(inv)))
    for i in range(1, x.size):
        x[i] = np.nextafter(x[i - 1], F(0))
    twice = np.trunc(((x * F(inv)).astype(F) + F(0.5)).astype(F))
    once = np.trunc((x.astype(np.float64) * np.float64(inv) + 0.5).astype(F))  # 48-bit product, exact in 64 bits
    return x[twice != once]
