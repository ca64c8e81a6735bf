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
