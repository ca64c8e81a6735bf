"""Plain reference of the cache in 8 bits, of attention with sinks and of sampling (numpy, 64-bit): test
infrastructure, no code of the package."""
import numpy as np

from paged_reference import EPS, Pages


# ------------------------------------------------------------------ e4m3
def e4m3_values():
    """The value of each code: sign, 4 bits of exponent (bias 7), 3 of fraction; 0x7F and 0xFF are NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if c & 127 == 127 else -v if c & 128 else v
    return out


VALUES = e4m3_values()


def e4m3_codes(x):
    """x (float64) rounded to the nearest code, ties to an even one, beyond 448 to 448; NaN to 0x7F."""
    mags = VALUES[:127]                         # rising, 0 .. 448
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.searchsorted(mags, a)               # first code whose value is at least a
    lo = np.maximum(hi - 1, 0)
    up, down = mags[hi] - a, a - mags[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(mags[hi] == a, hi, code)
    code = np.where(np.isnan(x), 127, code).astype(np.uint8)
    return code | np.where(np.signbit(x) & ~np.isnan(x), 128, 0).astype(np.uint8)


def scale_for(amax):
    """The least power of two s >= 2^-126 with amax <= 448 s; 0 for 0."""
    if amax == 0:
        return 0.0
    s = 2.0 ** -126
    while amax > 448.0 * s:
        s *= 2
    return s


class QPages(Pages):
    """Pages in 8 bits: pools hold codes (uint8), scales are one [n_pages, heads, blocks] array per pool."""

    def __init__(self, *args, block_rows, scales, **kw):
        super().__init__(*args, **kw)
        self.block_rows, self.scales = block_rows, list(scales)

    def resize(self, new):
        table, lens = self.table.copy(), self.lens.copy()
        err = super().resize(new)
        if err is None:
            for s, n in enumerate(new):
                old = int(lens[s])
                j = self._pages(old) - 1
                if n > old and old % self.page_rows and table[s, j] != self.table[s, j]:  # copied
                    blocks = -(-(old % self.page_rows) // self.block_rows)
                    for sc in self.scales:
                        sc[self.table[s, j], :, :blocks] = sc[table[s, j], :, :blocks]
        return err

    def compact(self):
        used = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        holes = [p for p in range(len(used)) if self.refs[p] == 0]
        for src, dst in zip([p for p in used if p >= len(used)], holes):
            for sc in self.scales:
                sc[dst] = sc[src]
        return super().compact()

    def write(self, i, rows, starts):
        """rows [tokens, heads, head_dim] float64 into pool i."""
        pool, scales, block = self.pools[i], self.scales[i], self.block_rows
        for s in range(len(self.lens)):
            at, end, pos = starts[s], starts[s + 1], int(self.lens[s]) - (starts[s + 1] - starts[s])
            while at < end:
                p, r = self.row(s, pos)
                first = r - r % block
                n = min(end - at, first + block - r, self.page_rows - r)
                for h in range(pool.shape[1]):
                    x = rows[at:at + n, h]
                    fine = np.abs(x[np.isfinite(x)])
                    old = np.float64(scales[p, h, first // block]) if r > first else 0.0
                    now = max(old, scale_for(fine.max() if fine.size else 0.0))
                    if now != old:
                        pool[p, h, first:r] = e4m3_codes(VALUES[pool[p, h, first:r]] * (old / now))
                    with np.errstate(invalid="ignore"):
                        pool[p, h, r:r + n] = e4m3_codes(x / now if now else x * 0.0)
                    scales[p, h, first // block] = now
                at, pos = at + n, pos + n


# ------------------------------------------------------------------ attention
def seen(nq, nk, window, sinks):
    """[nq, nk]: which keys the queries see, the last query at the last key."""
    gap = np.arange(nq)[:, None] + (nk - nq) - np.arange(nk)
    see = gap >= 0
    if window:
        see &= (gap < window) | (np.arange(nk) < sinks)
    return see


def attend_seen(q, k, v, see, scale, kind, weight=None, least=0.0, big=None):
    """softmax(scale q k^T) v over the keys seen, in 64 bits, and the largest error a kernel may make:
    q [nq, hq, hd], k and v [nk, hkv, hd].

    The bound is that of paged_reference.attend: the result is rounded once (u |out|); a weight p is off by
    at most `weight` of itself (one 16-bit term: u, the default) and by `least` of the largest; a score is a
    32-bit sum of hd products, each step off by at most 2^-23 of the sum of magnitudes B, which moves a weight
    by a factor of at most exp(2 d); sums of the products with v in 32 bits: 2^-16 of sum p |v|.
    big [nk, hkv]: what `least` is a part of, where V has scales: the weight times the key's scale, V's codes
    (at most 448) coming after it."""
    nq, hq, hd = q.shape
    group = hq // k.shape[1]
    u = EPS[kind]
    weight = u if weight is None else weight
    out, tol = np.zeros((nq, hq, hd)), np.zeros((nq, hq, hd))
    rows = np.flatnonzero(see.any(1))
    if not len(rows):
        return out, tol + 1e-30
    see = see[rows]
    for h in range(hq):
        kk, vv, qq = k[:, h // group], v[:, h // group], q[rows, h]
        kk, vv = np.where(see.any(0)[:, None], kk, 0.0), np.where(see.any(0)[:, None], vv, 0.0)
        s = np.where(see, qq @ kk.T * scale, -np.inf)
        e = np.exp(s - s.max(1, keepdims=True))
        l = e.sum(1, keepdims=True)
        p = e / l
        o = p @ vv
        b = np.where(see, abs(scale) * (np.abs(qq) @ np.abs(kk).T), 0.0).max(1, keepdims=True)
        t = u * np.abs(o) + (weight + 2 * hd * 2.0 ** -23 * b + 2.0 ** -16) * (p @ np.abs(vv))
        if big is not None:
            f = big[:, h // group]
            codes = np.where(f > 0, 448.0, 0.0)
            t += least * (p * f).max(1, keepdims=True) * (see @ codes)[:, None]
        elif least:
            t += least * (see @ np.abs(vv)) / l
        if kind == "fp16":
            t += 2.0 ** -25  # half a step of a subnormal result
        out[rows, h], tol[rows, h] = o, t
    return out, tol * (1 + 2 * u) + 1e-30


# ------------------------------------------------------------------ sampling
def draw(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, tokens kept, probability, room): room is how far, as a part of the sum, the nearest border lies
    that decides the token, and (kept, room) the same for the number kept."""
    x = np.asarray(x, np.float64)
    none = (-1, 0, 0.0, np.inf, np.inf)
    if not (0 <= temperature < np.inf and 0 <= top_p <= 1 and 0 <= min_p <= 1 and 0 <= u <= 1):
        return none
    valid = np.flatnonzero(x == np.inf if (x == np.inf).any() else x > -np.inf)
    if not len(valid):
        return none
    order = valid[np.lexsort((valid, -x[valid]))]
    if temperature == 0:
        return int(order[0]), 1, 1.0, np.inf, np.inf
    top = x[order[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.where(x[order] == top, 0.0, (x[order] - top) / temperature)
    w = np.exp(z)
    if 0 < top_k < len(order):
        order, w = order[:top_k], w[:top_k]
    n, near = len(order), np.inf
    if top_p < 1:
        c = np.cumsum(w)
        n = min(n, int((c < top_p * c[-1]).sum()) + 1)
        near = np.abs(c - top_p * c[-1]).min() / c[-1]
    if min_p > 0:
        n = min(n, int((w >= min_p).sum()))
        below = w[w < 1]  # (the largest logit's weight is 1 on any side)
        near = min(near, np.abs(below - min_p).min() if below.size else np.inf)
    order, w = order[:n], w[:n]
    by = np.argsort(order)
    order, w = order[by], w[by]
    c = np.cumsum(w)
    i = int((c <= u * c[-1]).sum())
    if i >= n:
        i = int(np.flatnonzero(w > 2.0 ** -43)[-1])
    return int(order[i]), n, w[i] / c[-1], np.abs(c - u * c[-1]).min() / c[-1], near
