"""Writes into 8-bit blocks whose scales come from elsewhere, against the reference in stream_reference.py."""
import numpy as np
import pytest

from test_gpu_paged import _mods, ints, randn
from test_gpu_stream import Both, INF, NAN, codes

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
