"""The paged cache and the prompt attention without a GPU: every refusal that the header
names is found on the host, before the device is touched."""
import ctypes

import pytest

import moe_decode_megakernel_warp_gb300 as msm

INVALID, UNSUPPORTED = msm.MSM_ERR_INVALID_ARG, msm.MSM_ERR_UNSUPPORTED
BUF = 1 << 20  # an address that nothing follows: every call below is refused before a launch


def pages(**over):
    ptrs = over.pop("ptrs", [BUF, BUF])
    kp, ka = msm._ptr_array(ptrs)
    c = dict(device=0, dtype=msm.MSM_BF16, n_layers=len(ptrs), n_pages=8, page_rows=16, n_kv_heads=2, head_dim=64,
             n_seqs=3, max_pages=4, k_pages=kp, v_pages=kp, table=BUF, lens=BUF, refs=BUF, status=BUF, scratch=BUF)
    c.update(over)
    p = msm.MsmPages(**c)
    p.keep = ka
    return p


BAD_PAGES = [
    (dict(dtype=2), INVALID), (dict(n_layers=0), INVALID), (dict(n_pages=0), INVALID), (dict(page_rows=0), INVALID),
    (dict(n_kv_heads=-1), INVALID), (dict(n_seqs=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), INVALID),
    (dict(n_seqs=1 << 16, max_pages=1 << 16), UNSUPPORTED), (dict(max_pages=1 << 20, page_rows=1 << 11), UNSUPPORTED),
    (dict(n_kv_heads=1 << 16), UNSUPPORTED), (dict(n_pages=1 << 30), UNSUPPORTED),
    (dict(n_pages=1 << 29, page_rows=16), UNSUPPORTED),
    (dict(ptrs=[BUF, 0]), INVALID), (dict(ptrs=[BUF + 8, BUF]), INVALID), (dict(k_pages=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(refs=None), INVALID), (dict(status=None), INVALID),
    (dict(scratch=None), INVALID), (dict(table=BUF + 2), INVALID), (dict(lens=BUF + 1), INVALID),
]


@pytest.mark.parametrize("over,want", BAD_PAGES)
def test_every_call_refuses_a_bad_description(over, want):
    c = pages(**over)
    calls = [lambda: msm.msm_pages_resize(c, BUF), lambda: msm.msm_pages_fork(c, BUF),
             lambda: msm.msm_pages_compact(c), lambda: msm.msm_pages_sync(c),
             lambda: msm.msm_pages_write(c, 0, BUF, BUF, (128, 64), (128, 64), BUF, 1),
             lambda: msm.msm_paged_attention(c, 0, BUF, (128, 64), 2, 1.0, 0, BUF, (128, 64), BUF, 1 << 30)]
    for call in calls:
        assert call() == want
    assert msm.msm_paged_attention_workspace(c, 2) == 0


def test_null_descriptions():
    lib = msm.lib()
    assert lib.msm_pages_resize(None, None, None) == INVALID
    assert lib.msm_pages_fork(None, None, None) == INVALID
    assert lib.msm_pages_compact(None, None) == INVALID
    assert lib.msm_pages_sync(None, None) == INVALID
    assert lib.msm_pages_write(None, 0, None, None, 0, 0, 0, 0, None, 0, None) == INVALID
    assert lib.msm_paged_attention(None, 0, None, 0, 0, 0, 0.0, 0, None, 0, 0, None, 0, None) == INVALID
    assert lib.msm_prompt_attention(None, None) == INVALID
    assert msm.msm_pages_scratch_ints(0, 1) == 0 and msm.msm_pages_scratch_ints(1, -1) == 0
    assert msm.msm_pages_scratch_ints(100, 10) >= 200


def test_arguments_of_the_page_calls():
    c = pages()
    assert msm.msm_pages_resize(c, None) == INVALID and msm.msm_pages_resize(c, BUF + 2) == INVALID
    assert msm.msm_pages_fork(c, None) == INVALID and msm.msm_pages_fork(c, BUF + 1) == INVALID
    ok = dict(layer=0, k=BUF, v=BUF, k_strides=(128, 64), v_strides=(128, 64), starts=BUF, n_tokens=1)
    for bad in (dict(layer=2), dict(layer=-1), dict(k=None), dict(v=BUF + 8), dict(k_strides=(129, 64)),
                dict(v_strides=(128, -64)), dict(k_strides=(1 << 31, 64)), dict(starts=None), dict(starts=BUF + 2),
                dict(n_tokens=-1)):
        assert msm.msm_pages_write(c, **{**ok, **bad}) == INVALID, bad
    assert msm.msm_pages_write(c, **{**ok, "n_tokens": 0, "k": None}) == msm.MSM_OK  # nothing to do


def test_arguments_of_the_paged_attention():
    c = pages()
    ok = dict(layer=0, q=BUF, q_strides=(256, 64), n_q_heads=4, scale=0.125, window=0, out=BUF, out_strides=(256, 64),
              workspace=BUF, workspace_bytes=1 << 30)
    for bad, want in ((dict(layer=2), INVALID), (dict(q=None), INVALID), (dict(q=BUF + 2), INVALID),
                      (dict(out=None), INVALID), (dict(out=BUF + 8), INVALID), (dict(n_q_heads=0), INVALID),
                      (dict(n_q_heads=3), INVALID), (dict(n_q_heads=6), UNSUPPORTED),
                      (dict(n_q_heads=32), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
                      (dict(scale=float("inf")), INVALID), (dict(window=-1), INVALID),
                      (dict(q_strides=(250, 64)), INVALID), (dict(out_strides=(256, 0)), INVALID),
                      (dict(out_strides=(256, 32)), INVALID), (dict(workspace=None), INVALID),
                      (dict(workspace=BUF + 4), INVALID)):
        assert msm.msm_paged_attention(c, **{**ok, **bad}) == want, bad
    assert msm.msm_paged_attention_workspace(c, 5) == 0 and "multiple" in msm.msm_last_error()


def test_arguments_of_the_prompt_attention():
    ok = dict(device=0, dtype=msm.MSM_FP16, n_seqs=2, n_q=10, n_k=10, n_q_heads=4, n_kv_heads=2, head_dim=128, window=0,
              scale=0.1, q=BUF, k=BUF, v=BUF, out=BUF, q_token_stride=512, q_head_stride=128, k_token_stride=256,
              k_head_stride=128, v_token_stride=256, v_head_stride=128, out_token_stride=512, out_head_stride=128,
              q_starts=BUF, k_starts=BUF)
    bad = [(dict(dtype=-1), INVALID), (dict(n_seqs=0), INVALID), (dict(n_q=-1), INVALID), (dict(n_k=-1), INVALID),
           (dict(n_q_heads=0), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_q_heads=3), INVALID),
           (dict(n_q_heads=6), UNSUPPORTED), (dict(head_dim=80), UNSUPPORTED), (dict(n_q=1 << 27), UNSUPPORTED),
           (dict(n_k=1 << 27), UNSUPPORTED), (dict(window=-1), INVALID), (dict(scale=float("nan")), INVALID),
           (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
           (dict(q_starts=None), INVALID), (dict(k_starts=None), INVALID), (dict(q=BUF + 8), INVALID),
           (dict(k=BUF + 2), INVALID), (dict(out=BUF + 4), INVALID), (dict(q_starts=BUF + 2), INVALID)]
    for name in ("q_token_stride", "q_head_stride", "k_token_stride", "k_head_stride", "v_token_stride",
                 "v_head_stride", "out_token_stride", "out_head_stride"):
        bad += [(dict([(name, s)]), INVALID) for s in (0, 120, 132, -128, 1 << 31)]
    for over, want in bad:
        assert msm.msm_prompt_attention(msm.MsmPrompt(**{**ok, **over})) == want, over
    assert msm.msm_prompt_attention(msm.MsmPrompt(**{**ok, "n_q": 0, "q": None})) == msm.MSM_OK  # nothing to do


def test_status_and_flags_of_the_prompt_attention():
    ok = dict(device=0, dtype=msm.MSM_BF16, n_seqs=1, n_q=10, n_k=10, n_q_heads=2, n_kv_heads=2, head_dim=64, scale=0.1,
              q=BUF, k=BUF, v=BUF, out=BUF, q_token_stride=128, q_head_stride=64, k_token_stride=128, k_head_stride=64,
              v_token_stride=128, v_head_stride=64, out_token_stride=128, out_head_stride=64, q_starts=BUF, k_starts=BUF)
    for bad in (dict(status=BUF + 2), dict(flags=1), dict(flags=msm.MSM_FLAG_TEST_DROP_HANDOFF | 8)):
        assert msm.msm_prompt_attention(msm.MsmPrompt(**{**ok, **bad})) == INVALID, bad


def test_more_work_than_a_launch_of_the_prompt_attention_takes():
    ok = dict(device=0, dtype=msm.MSM_BF16, n_seqs=1 << 20, n_q=10, n_k=10, n_q_heads=4096, n_kv_heads=4096, head_dim=64,
              scale=0.1, q=BUF, k=BUF, v=BUF, out=BUF, q_token_stride=1 << 18, q_head_stride=64, k_token_stride=1 << 18,
              k_head_stride=64, v_token_stride=1 << 18, v_head_stride=64, out_token_stride=1 << 18, out_head_stride=64,
              q_starts=BUF, k_starts=BUF)
    assert msm.msm_prompt_attention(msm.MsmPrompt(**ok)) == UNSUPPORTED
    assert "too many sequences" in msm.msm_last_error()
    for more in (dict(n_seqs=(1 << 31) - 1, n_q_heads=1, n_kv_heads=1), dict(n_seqs=(1 << 31) - 1),
                 dict(n_seqs=1, n_q=(1 << 27) - 1, n_q_heads=65528, n_kv_heads=8191)):
        assert msm.msm_prompt_attention(msm.MsmPrompt(**{**ok, **more})) == UNSUPPORTED, more


def test_the_torch_wrappers_check_what_torch_knows():
    torch = pytest.importorskip("torch")
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    ints = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        msm.PagedCache([k], [k], ints.view(2, 2), ints[:2], ints)
    with pytest.raises(ValueError, match="per layer"):
        msm.PagedCache([], [], ints.view(2, 2), ints[:2], ints)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        msm.prompt_attention(x, x, x, ints[:2])


def test_integers_as_c_ints():
    from moe_decode_megakernel_warp_gb300.paged import _c_int
    top = 2 ** 31 - 1
    for x, want in ((0, 0), (5, 5), (top, top), (top + 1, top), (1 << 32, top), (2 ** 63 - 1, top), (-1, -1), (-7, -1),
                    (-(1 << 32), -1)):
        assert _c_int(x) == want
