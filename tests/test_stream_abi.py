"""The cache in 8 bits, sinks and sampling without a GPU: every refusal that the header names is found on
the host, before the device is touched; and the reference against its own definitions."""
import ctypes

import numpy as np
import pytest

import moe_decode_megakernel_warp_gb300 as msm
from stream_reference import VALUES, draw, e4m3_codes, scale_for, seen
from test_paged_abi import BUF, INVALID, UNSUPPORTED, pages


def qpages(scales=(BUF, BUF), block_rows=8, **over):
    base = pages(**{"dtype": msm.MSM_E4M3, **over})
    ks, ka = msm._ptr_array(list(scales))
    q = msm.MsmQPages(base, block_rows, ks, ks)
    q.keep = (ka, base)
    return q


def calls(c):
    return [lambda: msm.msm_qpages_resize(c, BUF), lambda: msm.msm_qpages_fork(c, BUF),
            lambda: msm.msm_qpages_compact(c), lambda: msm.msm_qpages_sync(c),
            lambda: msm.msm_qpages_write(c, 0, msm.MSM_BF16, BUF, BUF, (128, 64), (128, 64), BUF, 1),
            lambda: msm.msm_qpages_attention(c, 0, msm.MSM_BF16, BUF, (128, 64), 2, 1.0, 0, 0, BUF, (128, 64), BUF, 1 << 30)]


@pytest.mark.parametrize("over,want", [
    (dict(dtype=msm.MSM_BF16), INVALID), (dict(dtype=msm.MSM_FP32), INVALID), (dict(n_pages=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(n_kv_heads=1 << 16), UNSUPPORTED), (dict(block_rows=0), INVALID),
    (dict(block_rows=-1), INVALID), (dict(block_rows=17), INVALID), (dict(scales=(BUF, 0)), INVALID),
    (dict(scales=(BUF + 2, BUF)), INVALID), (dict(ptrs=[BUF, BUF + 8]), INVALID), (dict(table=None), INVALID)])
def test_every_call_refuses_a_bad_description(over, want):
    c = qpages(**over)
    for call in calls(c):
        assert call() == want
    assert msm.msm_qpages_attention_workspace(c, 2) == 0


def test_null_descriptions():
    lib = msm.lib()
    assert lib.msm_qpages_resize(None, None, None) == INVALID
    assert lib.msm_qpages_fork(None, None, None) == INVALID
    assert lib.msm_qpages_compact(None, None) == INVALID
    assert lib.msm_qpages_sync(None, None) == INVALID
    assert lib.msm_qpages_write(None, 0, 0, None, None, 0, 0, 0, 0, None, 0, None) == INVALID
    assert lib.msm_qpages_attention(None, 0, 0, None, 0, 0, 0, 0.0, 0, 0, None, 0, 0, None, 0, None) == INVALID
    assert lib.msm_paged_attention_sinks(None, 0, None, 0, 0, 0, 0.0, 0, 0, None, 0, 0, None, 0, None) == INVALID
    assert lib.msm_prompt_attention_sinks(None, 0, None) == INVALID
    assert lib.msm_sample(None, None) == INVALID
    q = qpages()
    q.k_scales = None
    assert msm.msm_qpages_compact(q) == INVALID


def test_the_calls_of_16_bits_refuse_8():
    c = pages(dtype=msm.MSM_E4M3)
    assert msm.msm_pages_resize(c, BUF) == INVALID and msm.msm_pages_compact(c) == INVALID
    assert msm.msm_paged_attention_workspace(c, 2) == 0


def test_arguments_of_the_8_bit_calls():
    c = qpages()
    assert msm.msm_qpages_resize(c, None) == INVALID and msm.msm_qpages_resize(c, BUF + 2) == INVALID
    assert msm.msm_qpages_fork(c, None) == INVALID
    ok = dict(layer=0, dtype=msm.MSM_FP16, k=BUF, v=BUF, k_strides=(128, 64), v_strides=(128, 64), starts=BUF, n_tokens=1)
    for bad in (dict(layer=2), dict(layer=-1), dict(dtype=msm.MSM_E4M3), dict(dtype=msm.MSM_FP32), dict(dtype=-1),
                dict(k=None), dict(v=BUF + 8), dict(k_strides=(129, 64)), dict(v_strides=(128, -64)),
                dict(k_strides=(1 << 31, 64)), dict(starts=None), dict(starts=BUF + 2), dict(n_tokens=-1)):
        assert msm.msm_qpages_write(c, **{**ok, **bad}) == INVALID, bad
    assert msm.msm_qpages_write(c, **{**ok, "n_tokens": 0, "k": None}) == msm.MSM_OK  # nothing to do
    ok = dict(layer=0, dtype=msm.MSM_BF16, q=BUF, q_strides=(256, 64), n_q_heads=4, scale=0.125, window=5, sinks=1,
              out=BUF, out_strides=(256, 64), workspace=BUF, workspace_bytes=1 << 30)
    for bad, want in ((dict(layer=2), INVALID), (dict(dtype=2), INVALID), (dict(q=None), INVALID),
                      (dict(q=BUF + 2), INVALID), (dict(out=BUF + 8), INVALID), (dict(n_q_heads=3), INVALID),
                      (dict(n_q_heads=6), UNSUPPORTED), (dict(scale=float("nan")), INVALID), (dict(window=-1), INVALID),
                      (dict(sinks=-1), INVALID), (dict(out_strides=(256, 32)), INVALID), (dict(workspace=None), INVALID),
                      (dict(workspace=BUF + 4), INVALID)):
        assert msm.msm_qpages_attention(c, **{**ok, **bad}) == want, bad
    assert msm.msm_qpages_attention_workspace(c, 5) == 0 and "multiple" in msm.msm_last_error()


def test_negative_sinks():
    c = pages()
    assert msm.msm_paged_attention_sinks(c, 0, BUF, (256, 64), 4, 0.1, 5, -1, BUF, (256, 64), BUF, 1 << 30) == INVALID
    assert "sinks" in msm.msm_last_error()
    p = msm.MsmPrompt(device=0, dtype=msm.MSM_FP16, n_seqs=2, n_q=10, n_k=10, n_q_heads=4, n_kv_heads=2, head_dim=128,
                      window=3, scale=0.1, q=BUF, k=BUF, v=BUF, out=BUF, q_token_stride=512, q_head_stride=128,
                      k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128,
                      out_token_stride=512, out_head_stride=128, q_starts=BUF, k_starts=BUF)
    assert msm.msm_prompt_attention_sinks(p, -1) == INVALID
    assert "sinks" in msm.msm_last_error()


def test_arguments_of_sampling():
    ok = dict(device=0, dtype=msm.MSM_FP32, n_rows=2, vocab=100, logits=BUF, row_stride=100, random=BUF, tokens=BUF)
    for bad, want in ((dict(dtype=msm.MSM_E4M3), INVALID), (dict(dtype=9), INVALID), (dict(n_rows=-1), INVALID),
                      (dict(vocab=0), INVALID), (dict(vocab=(1 << 20) + 1, row_stride=1 << 21), UNSUPPORTED),
                      (dict(n_rows=1 << 24), UNSUPPORTED), (dict(row_stride=-1), INVALID), (dict(logits=None), INVALID),
                      (dict(random=None), INVALID), (dict(tokens=None), INVALID), (dict(logits=BUF + 2), INVALID),
                      (dict(dtype=msm.MSM_BF16, logits=BUF + 1), INVALID), (dict(temperature=BUF + 2), INVALID),
                      (dict(top_k=BUF + 1), INVALID), (dict(top_p=BUF + 2), INVALID), (dict(min_p=BUF + 2), INVALID),
                      (dict(random=BUF + 2), INVALID), (dict(tokens=BUF + 2), INVALID), (dict(probs=BUF + 2), INVALID),
                      (dict(kept=BUF + 2), INVALID)):
        assert msm.msm_sample(msm.MsmSampling(**{**ok, **bad})) == want, bad
    assert msm.msm_sample(msm.MsmSampling(**{**ok, "n_rows": 0, "logits": None})) == msm.MSM_OK  # nothing to do


def test_the_torch_wrappers_check_what_torch_knows():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="CUDA"):
        msm.sample(torch.zeros(2, 5), torch.zeros(2))


def test_e4m3_of_the_reference():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, VALUES, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 9, 4000), VALUES[:127],
                        (VALUES[:126] + VALUES[1:127]) / 2, [0.0, -0.0, 2.0 ** -10, -2.0 ** -10]])
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(e4m3_codes(x.astype(np.float64)), want)
    assert list(e4m3_codes(np.array([1e9, -np.inf, 460.0]))) == [126, 254, 126]
    assert scale_for(448.0) == 1 and scale_for(448.1) == 2 and scale_for(1e-45) == 2.0 ** -126 and scale_for(0) == 0


def test_seen_and_draw_of_the_reference():
    assert seen(1, 6, 2, 1).tolist() == [[True, False, False, False, True, True]]
    assert seen(3, 2, 0, 0).tolist() == [[False, False], [True, False], [True, True]]
    x = np.log([0.1, 0.4, 0.4, 0.1])
    assert draw(x, 0.05)[:2] == (0, 4) and draw(x, 0.2)[0] == 1 and draw(x, 0.95)[0] == 3 and draw(x, 1.0)[0] == 3
    assert draw(x, 0.5, top_k=1)[:2] == (1, 1) and draw(x, 0.6, top_k=3)[:2] == (2, 3)
    assert draw(x, 0.9, top_p=0.5)[:2] == (2, 2) and draw(x, 0.0, min_p=0.5)[:2] == (1, 2)
    assert draw(x, 0.3, temperature=0)[:3] == (1, 1, 1.0) and draw([-np.inf, np.nan], 0.3)[0] == -1
    assert draw([0.0, np.inf, np.inf], 0.7)[:3] == (2, 2, 0.5) and draw(x, 1.5)[0] == -1
