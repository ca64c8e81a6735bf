"""Writes into 8-bit blocks whose scales come from elsewhere, against the reference in stream_reference.py."""
import numpy as np
import pytest

from test_gpu_paged import _mods, ints, randn
from test_gpu_stream import Both

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
