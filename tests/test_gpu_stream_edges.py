"""Writes into 8-bit blocks whose scales come from elsewhere, and sampling with the numbers at the ends of their ranges, against
the reference in stream_reference.py."""
import numpy as np
import pytest

from stream_reference import draw
from test_gpu_paged import _mods, f64, ints, randn
from test_gpu_stream import Both, INF, NAN, codes, logits

pytestmark = pytest.mark.gpu


def set_scales(c, make):
    """New scales of every block, on the GPU and in the reference: make(pool, shape)."""
    torch, _ = _mods()
    for i, (t, r) in enumerate(zip(c.gpu.k_scales + c.gpu.v_scales, c.ref.scales)):
        new = np.asarray(make(i, r.shape), np.float32)
        t.copy_(torch.from_numpy(new))
        r[:] = new


# ------------------------------------------------------------------ writes behind scales of other origin
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -127, 2.0 ** -128, 2.0 ** -130, 3 * 2.0 ** -148, 2.0 ** -149, 0.0])
def test_zeros_behind_rows_of_the_smallest_scales(kind, scale):
    """A scale that is not negative may be so small that its reciprocal is no number: 0 stays 0 over it."""
    c = Both(np.random.default_rng(1), 1, 8, 16, 8, 2, 64, 2, 4, kind)
    c.call("resize", [3, 21])
    c.write([3, 21], 1)
    set_scales(c, lambda i, shape: np.full(shape, scale))
    c.call("resize", [5, 24])
    c.write([2, 3], 2, sizes=0.0)
    assert not c.gpu.attention(0, randn(kind, 2, 4, 64, seed=3).cuda()).isnan().any()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,hd,older,new", [(16, 64, 3, 1), (16, 128, 3, 13), (100, 128, 30, 60), (300, 128, 100, 190),
                                               (70, 64, 1, 69)])
def test_quotients_next_to_the_borders_of_codes(kind, rows, hd, older, new):
    """Blocks that keep a scale which is no power of two: elements that lie on a border between two codes but for the
    rounding of the scale, and any others.  (The reference's quotient has 53 bits.  An element has at most 11 and a scale 24, so
    a quotient that is not on a border is at least 2^-30 of itself away from it: the reference decides all of them.)"""
    torch, _ = _mods()
    rng = np.random.default_rng(rows + new)
    n, heads = 12, 3
    c = Both(rng, 1, n, rows, rows, heads, hd, n, 1, kind)
    c.call("resize", [older] * n)
    c.write([older] * n, 1)
    digits, least, most = (128, -60, 60) if kind == "bf16" else (1024, -18, -8)
    unit = rng.integers(digits, 2 * digits, (n, 2 * heads)) * 2.0 ** rng.integers(least, most, (n, 2 * heads))
    tie = rng.integers(8, 16, (n, 2 * heads)) * 2 + 1                              # 17 .. 31: halfway between codes 8 .. 16
    step = rng.integers(-1, 2, (n, 2 * heads))
    scale = (unit / (tie / 16.0)).astype(np.float32)
    scale = (scale.view(np.int32) + step.astype(np.int32)).view(np.float32)     # the nearest one and its neighbours
    page = c.ref.table[:, 0]

    def make(i, shape):
        s = np.ones(shape, np.float32)
        s[page, :, 0] = scale[:, i * heads:(i + 1) * heads]
        return s
    set_scales(c, make)

    def change(kv):
        shape = (n, new, 2 * heads, hd)
        x = unit[:, None, :, None] * 2.0 ** rng.integers(-9, 7, shape) * rng.choice([-1.0, 1.0], shape)
        other = scale[:, None, :, None] * rng.uniform(-220.0, 220.0, shape) * 2.0 ** rng.integers(-10, 1, shape)
        x = np.where(rng.random(shape) < 0.6, x, other)
        x = torch.from_numpy(x.reshape(n * new, 2 * heads, hd)).to(kv.dtype)
        kv[:n * new] = x
    c.call("resize", [older + new] * n)
    c.write([new] * n, 2, change=change)
    assert np.array_equal(c.ref.scales[0][page, :, 0], scale[:, :heads])        # (none of the rows made them grow)


@pytest.mark.parametrize("rows,block,older,new", [(16, 8, 3, 5), (100, 100, 40, 50), (300, 300, 250, 40)])
def test_scales_that_are_no_powers_of_two_grow_and_stay(rows, block, older, new):
    """Scales as a cache may have that was quantised elsewhere (the largest magnitude over 448).  (20 bits of them, so that a code,
    4 bits, times old / new has the 24 that the product is taken in.)"""
    rng = np.random.default_rng(rows)
    c = Both(rng, 1, 8, rows, block, 2, 128, 4, 2)
    c.call("resize", [older] * 4)
    c.write([older] * 4, 1)

    def make(i, shape):
        s = (rng.uniform(0.3, 4.0, shape) / 448).astype(np.float32)
        return (s.view(np.uint32) & np.uint32(0xFFFFFFF0)).view(np.float32)
    set_scales(c, make)
    for step, sizes in enumerate((0.02, 1.0, 40.0)):
        old = c.ref.lens.copy()
        c.call("resize", [int(n) + new for n in old] if step < 1 else [int(n) + 1 for n in old])
        c.write(c.ref.lens - old, step + 2, sizes=sizes)


def write_special(kind, rows, older, new, pattern, old_scale):
    """Codes and scales after rows of zeros with some special elements, behind `older` rows."""
    torch, msm = _mods()
    hd = 128
    c = msm.PagedCache.allocate(1, 3, rows, 1, hd, 2, 1, dtype=torch.float8_e4m3fn)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[kind]
    c.resize(ints([older, 0]))
    if older:
        c.write(0, torch.zeros(older, 1, hd, dtype=dt, device="cuda"), torch.zeros(older, 1, hd, dtype=dt, device="cuda"),
                ints([0, older, older]))
    for t in c.k_scales + c.v_scales:
        t.fill_(old_scale)
    c.resize(ints([older + new, 0]))
    x = torch.zeros(new, 1, hd, dtype=dt)
    for (r, d), v in pattern.items():
        x[r, 0, d] = v
    x = x.cuda()
    c.write(0, x, x, ints([0, new, new]))
    got = c.attention(0, torch.ones(2, 1, hd, dtype=dt, device="cuda"))
    c.sync()
    p = int(c.table[0, 0])
    return [(codes(k)[p, 0, older:older + new], float(s[p, 0, 0])) for k, s in ((c.k_pages[0], c.k_scales[0]),
                                                                              (c.v_pages[0], c.v_scales[0]))], got


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,older,new", [(16, 0, 3), (16, 5, 4), (16, 3, 1), (200, 0, 150), (200, 120, 70)])
def test_infinities_where_nothing_else_gives_a_scale(kind, rows, older, new):
    """The only elements other than 0 are infinite: the scale is 0, or the one that the block has, and their codes are +-448."""
    for old_scale in (0.0, 2.0 ** -149, 2.0 ** -130, 0.3):
        pattern = {(0, 3): INF, (new - 1, 100): -INF, (0, 64): -0.0}
        held, got = write_special(kind, rows, older, new, pattern, old_scale)
        want = np.zeros((new, 128), np.uint8)
        want[0, 3], want[new - 1, 100], want[0, 64] = 0x7E, 0xFE, 0x80
        for code, scale in held:
            assert np.array_equal(code, want) and scale == np.float32(old_scale if older else 0.0)
        assert not got.isnan().any()
        pattern[new - 1, 7] = NAN
        held, _ = write_special(kind, rows, older, new, pattern, old_scale)
        for code, scale in held:
            assert code[new - 1, 7] & 0x7F == 0x7F
            code[new - 1, 7] = 0
            assert np.array_equal(code, want) and scale == np.float32(old_scale if older else 0.0)


# ------------------------------------------------------------------ sampling
def drawn(x, u, **par):
    """Draws and compares every row; (tokens, kept, rows too near a border to be decided).  A weight w is off by at most
    1.1 x 2^-30 w (two roundings of 1/2 .. 1 to 2^-31) + 2^-43 (the largest logit's by nothing), so sums, which are at least 1, by 1.1 x 2^-30
    of the share of the others + 2^-43 for each of them.  Borders nearer than that are not compared.  (min_p is one that no
    weight is near to.)"""
    torch, msm = _mods()
    n = len(x)
    kept, probs = torch.full((n,), -7, dtype=torch.int32, device="cuda"), torch.full((n,), NAN, device="cuda")
    dev = {k: torch.tensor(np.asarray(v), dtype=torch.int32 if k == "top_k" else torch.float32).cuda() for k, v in par.items()}
    u = torch.as_tensor(np.asarray(u), dtype=torch.float32).cuda()
    tokens = msm.sample(x, u, probs=probs, kept=kept, **dev).cpu().numpy()
    kept, probs = kept.cpu().numpy(), probs.cpu().double().numpy()
    host = {k: v.cpu().double().numpy() for k, v in dev.items()}
    rows, close = f64(x), 0
    for i, row in enumerate(rows):
        one = {k: int(v[i]) if k == "top_k" else float(v[i]) for k, v in host.items()}
        token, m, p, room, near = draw(row, float(u[i].double()), **one)
        if "min_p" in one:
            near = draw(row, 0.5, **{k: v for k, v in one.items() if k != "min_p"})[4]
        t, top = one.get("temperature", 1.0), np.fmax.reduce(row)
        with np.errstate(invalid="ignore", over="ignore"):
            w = np.exp(np.where(row == top, 0.0, (row - top) / t)) if t else (row == top) * 1.0
        w = np.nan_to_num(w, nan=0.0)
        limit = 1.1 * 2.0 ** -30 * (1 - (w == 1).sum() / max(1.0, w.sum())) + 2.0 ** -43 * ((w > 0) & (w < 1)).sum()
        if min(room, near) <= limit:
            close += 1
            continue
        assert (tokens[i], kept[i]) == (token, m), (i, one, room, near, tokens[i], token, kept[i], m)
        assert abs(probs[i] - p) <= 2.0 ** -20 * p + 2.0 ** -40, (i, probs[i], p)
    return tokens, kept, close


def tails(n, vocab, many, levels, seed, dtype="fp32"):
    """Rows of one logit far above `many` others, weights of 2^-17 to 2^-22 of its own at `levels` different values (0: all
    different), and nothing else: the first histogram's last class begins at 2^-16."""
    torch, _ = _mods()
    rng = np.random.default_rng(seed)
    x = np.full((n, vocab), -INF, np.float32)
    for i in range(n):
        at = rng.permutation(vocab)[:many + 1]
        t = rng.uniform(17.0, 22.0, levels or many)
        x[i, at[1:]] = 5.0 - np.log(2.0) * (rng.choice(t, many) if levels else t)
        x[i, vocab // 2] = 5.0
    return torch.from_numpy(x).to({"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]).cuda(), rng


@pytest.mark.parametrize("vocab,many,levels,dtype", [(3000, 2500, 0, "fp32"), (3000, 2500, 7, "fp32"), (40000, 5000, 0, "fp32"),
                                                     (60000, 8000, 300, "fp32"), (131072, 8000, 0, "bf16"), (9000, 400, 0, "fp32")])
def test_borders_and_draws_among_the_smallest_weights(vocab, many, levels, dtype):
    """The border of top-k, top-p and min-p and the token lie in the first histogram's last class.  Borders of sums are some
    2^-19.5 of the sum apart, 1,000 times what decides, and min-p's number lies between two weights: of a case's 128 rows and 250
    borders 0.7 at most are too near one on average."""
    n = 16
    x, rng = tails(n, vocab, many, levels, vocab + many + levels, dtype)
    w = np.exp(f64(x) - 5.0)
    tail = (w.sum(1) - 1) / w.sum(1)
    front = w[:, :vocab // 2].sum(1) / w.sum(1)
    u = front * rng.uniform(0.001, 0.2, n)      # a token in front of the large one, where the border leaves enough of them
    p = 1 - tail * rng.uniform(0.1, 0.9, n)
    k = rng.integers(many // 8, many, n)
    m = []
    for i in range(n):                          # halfway between two weights, of the wider half of the gaps
        v = np.unique(w[i][(w[i] > 0) & (w[i] < 1)])
        gaps = np.diff(v)
        g = rng.choice(np.flatnonzero(gaps >= np.median(gaps)))
        m.append((v[g] + v[g + 1]) / 2)
    near = others = 0
    for par in ({}, dict(top_p=p), dict(top_k=k), dict(top_k=k, top_p=p), dict(min_p=m), dict(top_k=k, min_p=m),
                dict(top_p=p, min_p=m), dict(top_k=k, top_p=p, min_p=m)):
        tokens, kept, close = drawn(x, u, **par)
        near += close
        others += int((tokens != vocab // 2).sum())
        if par:
            assert (kept <= many).all() and (kept > 1).mean() > 0.7, par
    assert near <= 4
    assert others > 8 * n * 0.6


@pytest.mark.parametrize("vocab", [40, 2500, 33000])
def test_equal_logits_with_borders_between_two_of_them(vocab):
    """All rows are decided: top-p and the random number lie halfway between borders."""
    torch, _ = _mods()
    rng = np.random.default_rng(vocab)
    n = 12
    k = rng.integers(1, vocab + 1, n)
    m = rng.integers(0, vocab, n)
    j = np.array([rng.integers(0, i + 1) for i in m])
    for x in (torch.full((n, vocab), 3.25, device="cuda"), torch.full((n, vocab), -7.0, dtype=torch.float16, device="cuda")):
        tokens, kept, close = drawn(x, (j + 0.5) / (m + 1), top_p=(m + 0.5) / vocab)
        assert close == 0 and (tokens == j).all() and (kept == m + 1).all()
        tokens, kept, close = drawn(x, (np.minimum(j, k - 1) + 0.5) / k, top_k=k)
        assert close == 0 and (tokens == np.minimum(j, k - 1)).all() and (kept == k).all()


def test_masked_rows_are_all_decided():
    """The rows of test_rows_without_a_choice_and_masked_rows (where the border of top-p 0.5 among equal weights lies
    on the target) with numbers between the borders."""
    torch, _ = _mods()
    x, u = logits(10, 5000, "fp32", 1)
    x[0], x[1], x[2, :], x[2, 4321], x[3, ::2] = -INF, NAN, -INF, -3.0, NAN
    x[4, 1:], x[5] = torch.finfo(torch.float32).min, torch.finfo(torch.float32).min
    x[6, 17], x[6, 99], x[7, 5], x[8, 100:] = INF, INF, torch.finfo(torch.float32).max, -INF
    for y in (x, x.bfloat16()):
        for par in ({}, dict(top_k=[50] * 10), dict(top_p=[0.8003] * 10), dict(min_p=[0.1] * 10), dict(temperature=[1e-38] * 10),
                    dict(temperature=[3e38] * 10, top_p=[0.50013] * 10), dict(top_k=[4999] * 10, top_p=[0.99903] * 10)):
            tokens, _, close = drawn(y, u, **par)
            none = [0, 1] if y.dtype == torch.float32 else [0, 1, 5]    # (the lowest fp32 value is -inf in bf16)
            assert close == 0 and list(np.flatnonzero(tokens == -1)) == none, par


def test_zeros_of_either_sign():
    """-0 is 0, as temperature, top-p, min-p and random number."""
    torch, msm = _mods()
    for vocab in (5, 3000, 40000):
        x, u = logits(6, vocab, "fp32", vocab)
        plus, minus = torch.zeros(6, device="cuda"), torch.full((6,), -0.0, device="cuda")
        ud = torch.as_tensor(u, dtype=torch.float32).cuda()
        for name in ("temperature", "top_p", "min_p", "random"):
            got = []
            for z in (plus, minus):
                kept, probs = torch.full((6,), -7, dtype=torch.int32, device="cuda"), torch.full((6,), NAN, device="cuda")
                par = dict(random=ud, kept=kept, probs=probs)
                par[name] = z
                if name == "random":
                    par["top_p"] = torch.full((6,), 0.7, device="cuda")
                got.append((msm.sample(x, **par), kept, probs))
            for a, b in zip(*got):
                assert torch.equal(a, b), name
            host = {name: -0.0} if name != "random" else dict(top_p=float(np.float32(0.7)))
            for i in range(6):
                want = draw(f64(x[i]), -0.0 if name == "random" else float(ud[i]), **host)
                assert (int(got[1][0][i]), int(got[1][1][i])) == want[:2], (name, i)
