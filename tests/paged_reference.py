"""Plain reference of the paged cache and of the attention that reads it (numpy, 64-bit):
test infrastructure, no code of the package."""
import numpy as np

EPS = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a step, relative


class Pages:
    """The bookkeeping of a paged cache, one sequence and one page at a time, and the rows as
    a list of [n_pages, heads, page_rows, head_dim] arrays."""

    def __init__(self, n_pages, page_rows, n_seqs, max_pages, pools=()):
        self.page_rows, self.max_pages = page_rows, max_pages
        self.table = np.full((n_seqs, max_pages), -1, np.int32)
        self.lens = np.zeros(n_seqs, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        self.pools = list(pools)

    def _pages(self, n):
        return -(-int(n) // self.page_rows)

    def resize(self, new):
        """None, or the error's name (then nothing changed)."""
        cap = self.max_pages * self.page_rows
        if any(n < -1 or n > cap for n in new):
            return "MSM_ERR_INVALID_ARG"
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        plan = []
        for s, n in enumerate(new):
            old = int(self.lens[s])
            n = old if n == -1 else int(n)
            have, want = self._pages(old), self._pages(n)
            leave = n > old and old % self.page_rows != 0 and self.refs[self.table[s, have - 1]] > 1
            plan.append((s, old, n, have, want, leave))
        if sum(max(0, want - have) + leave for _, _, _, have, want, leave in plan) > len(free):
            return "MSM_ERR_OOM"
        taken = iter(free)
        for s, old, n, have, want, leave in plan:
            if leave:
                src, dst = int(self.table[s, have - 1]), next(taken)
                for pool in self.pools:
                    pool[dst, :, :old % self.page_rows] = pool[src, :, :old % self.page_rows]
                self.table[s, have - 1] = dst
                self.refs[dst] += 1
                self.refs[src] -= 1
            for j in range(have, want):
                self.table[s, j] = next(taken)
                self.refs[self.table[s, j]] += 1
            for j in range(want, have):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.lens[s] = n
        return None

    def fork(self, parent):
        for s, p in enumerate(parent):
            if p == -1:
                continue
            if p < 0 or p >= len(parent) or p == s or parent[p] != -1 or self.lens[s] != 0:
                return "MSM_ERR_INVALID_ARG"
        for s, p in enumerate(parent):
            if p == -1:
                continue
            for j in range(self._pages(self.lens[p])):
                self.table[s, j] = self.table[p, j]
                self.refs[self.table[p, j]] += 1
            self.lens[s] = self.lens[p]
        return None

    def compact(self):
        used = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        n = len(used)
        holes = [p for p in range(n) if self.refs[p] == 0]
        to = dict(zip([p for p in used if p >= n], holes))
        for src, dst in to.items():
            for pool in self.pools:
                pool[dst] = pool[src]
            self.refs[dst], self.refs[src] = self.refs[src], 0
        for s in range(len(self.lens)):
            for j in range(self._pages(self.lens[s])):
                self.table[s, j] = to.get(int(self.table[s, j]), self.table[s, j])

    def row(self, s, r):
        return int(self.table[s, r // self.page_rows]), r % self.page_rows

    def write(self, pool, rows, starts):
        for s in range(len(self.lens)):
            n = starts[s + 1] - starts[s]
            for i in range(n):
                p, r = self.row(s, int(self.lens[s]) - n + i)
                pool[p, :, r] = rows[starts[s] + i]

    def gather(self, pool, s):
        """[rows][heads][head_dim] of sequence s."""
        out = np.empty((int(self.lens[s]), pool.shape[1], pool.shape[3]), pool.dtype)
        for r in range(len(out)):
            p, i = self.row(s, r)
            out[r] = pool[p, :, i]
        return out

    def check(self):
        """The invariants of a cache."""
        count = np.zeros_like(self.refs)
        for s in range(len(self.lens)):
            n = self._pages(self.lens[s])
            assert (self.table[s, :n] >= 0).all() and (self.table[s, n:] == -1).all()
            np.add.at(count, self.table[s, :n], 1)
        assert np.array_equal(count, self.refs)


def attend(q, k, v, shift, window, scale, kind):
    """Causal attention of one sequence in 64 bits.  q [nq, hq, hd], k and v [nk, hkv, hd]
    float64 holding 16-bit values; query i sees the keys j with 0 <= i + shift - j (< window).
    Returns out and the largest error a kernel may make, element by element.

    The bound, for 16-bit type `kind` with half a step u (relative), p the softmax weights:
      - the result is rounded once:                                      u |out|
      - each weight is rounded to 16 bits before its product with v:     u sum p |v|
        (fp16 also has an absolute half step, 2^-25, below 2^-14; a weight is at most its
        final value times the sum l of the unnormalised ones):           2^-25 sum |v| / l
      - the scores are 32-bit sums of hd products, each step off by at most 2^-23 of the sum
        of magnitudes B (tensor cores may truncate), as are the sums of the weights' products
        over at most nk keys in partial sums of 16 and more; a score's error d moves every
        weight by at most a factor exp(2 d):  (2 hd 2^-23 scale B + 2^-16) sum p |v|
    The window, the causal mask and rows without keys are exact."""
    nq, hq, hd = q.shape
    nk, hkv, _ = k.shape
    group = hq // hkv
    u = EPS[kind]
    out, tol = np.zeros((nq, hq, hd)), np.zeros((nq, hq, hd))
    j = np.arange(nk)
    for i in range(nq):
        gap = i + shift - j
        see = (gap >= 0) & ((gap < window) if window else True)
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[see, h // group], v[see, h // group]
            s = kk @ q[i, h] * scale
            e = np.exp(s - s.max())
            l = e.sum()
            p = e / l
            out[i, h] = p @ vv
            mag = p @ np.abs(vv)
            b = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
            tol[i, h] = u * np.abs(out[i, h]) + (u + 2 * hd * 2.0 ** -23 * b + 2.0 ** -16) * mag
            if kind == "fp16":
                tol[i, h] += 2.0 ** -25 * np.abs(vv).sum(0) / l
    return out, tol * (1 + 2 * u) + 1e-30


def attend_matrix(q, k, v, shift, window, scale, kind, terms=1, least=None):
    """attend() with a head's queries and keys as one matrix (for batches of many rows).

    terms = 2: the bound where a weight p is held as two 16-bit terms.  The first one is p (1 - 2 u)
    rounded, so the rest is between 0 and p (1 - (1 - 2 u) (1 - u)) < 3 u p, of which its rounding
    takes at most half a step: 3 u^2 p; fp16 weights are at most 2^14 then, so half of their smallest
    step, 2^-25, is 2^-39 of the largest weight.
    least: half of the smallest fp16 step, as a part of the largest weight (2^-25 where that is 1)."""
    nq, hq, hd = q.shape
    nk, hkv, _ = k.shape
    group = hq // hkv
    u = EPS[kind]
    weight = u if terms == 1 else 3 * u * u
    least = least or 2.0 ** (-25 if terms == 1 else -39)
    out, tol = np.zeros((nq, hq, hd)), np.zeros((nq, hq, hd))
    gap = np.arange(nq)[:, None] + shift - np.arange(nk)
    see = (gap >= 0) & ((gap < window) if window else True)
    rows = np.flatnonzero(see.any(1))
    see = see[rows]
    if not len(rows):
        return out, tol + 1e-30
    for h in range(hq):
        kk, vv, qq = k[:, h // group], v[:, h // group], q[rows, h]
        s = np.where(see, qq @ kk.T * scale, -np.inf)
        e = np.exp(s - s.max(1, keepdims=True))
        l = e.sum(1, keepdims=True)
        p = e / l
        o = p @ vv
        b = np.where(see, abs(scale) * (np.abs(qq) @ np.abs(kk).T), 0.0).max(1, keepdims=True)
        t = u * np.abs(o) + (weight + 2 * hd * 2.0 ** -23 * b + 2.0 ** -16) * (p @ np.abs(vv))
        if kind == "fp16":
            t += least * (see @ np.abs(vv)) / l
        out[rows, h], tol[rows, h] = o, t
    return out, tol * (1 + 2 * u) + 1e-30
