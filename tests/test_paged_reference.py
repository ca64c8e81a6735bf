"""The paged cache's reference on the CPU: random calls keep its invariants and every
sequence's rows, and its attention equals an independent statement of the formula."""
import numpy as np
import pytest

from paged_reference import Pages, attend


@pytest.mark.parametrize("seed", range(6))
def test_random_calls_keep_the_rows_of_every_sequence(seed):
    rng = np.random.default_rng(seed)
    rows, n_seqs, max_pages, n_pages = int(rng.integers(1, 9)), 6, 7, 30
    pool = rng.standard_normal((n_pages, 2, rows, 4))
    c = Pages(n_pages, rows, n_seqs, max_pages, [pool])
    want = [np.zeros((0, 2, 4)) for _ in range(n_seqs)]
    for _ in range(60):
        op = rng.integers(0, 3)
        if op == 0:
            new = [int(rng.integers(-1, max_pages * rows + 1)) for _ in range(n_seqs)]
            old = c.lens.copy()
            if c.resize(new) is None:
                add = np.maximum(c.lens - old, 0)
                starts = np.concatenate([[0], np.cumsum(add)])
                new_rows = rng.standard_normal((starts[-1], 2, 4))
                c.write(pool, new_rows, starts)
                for s in range(n_seqs):
                    want[s] = np.concatenate([want[s][:c.lens[s]], new_rows[starts[s]:starts[s + 1]]])
        elif op == 1:
            parent = [-1] * n_seqs
            for s in range(n_seqs):
                if c.lens[s] == 0 and rng.random() < 0.5:
                    parent[s] = int(rng.integers(0, n_seqs))
            if c.fork(parent) is None:
                for s, p in enumerate(parent):
                    if p >= 0:
                        want[s] = want[p].copy()
        else:
            c.compact()
            n = int((c.refs > 0).sum())
            assert (c.refs[:n] > 0).all()
        c.check()
        for s in range(n_seqs):
            assert np.array_equal(c.gather(pool, s), want[s])


def test_resize_refuses_without_changing_anything():
    c = Pages(3, 4, 2, 3)
    assert c.resize([4, 9]) == "MSM_ERR_OOM"
    assert c.resize([-2, 1]) == c.resize([13, 0]) == "MSM_ERR_INVALID_ARG"
    assert (c.lens == 0).all() and (c.refs == 0).all() and (c.table == -1).all()


@pytest.mark.parametrize("shift,window", [(0, 0), (3, 0), (-2, 0), (5, 3), (0, 1)])
def test_attention_equals_the_masked_softmax(shift, window):
    rng = np.random.default_rng(7)
    nq, hq, hkv, hd = 5, 4, 2, 8
    nk = nq + shift
    q, k, v = (rng.standard_normal(s) for s in ((nq, hq, hd), (nk, hkv, hd), (nk, hkv, hd)))
    out, tol = attend(q, k, v, shift, window, 0.3, "bf16")
    s = np.einsum("ihd,jhd->hij", q, np.repeat(k, 2, 1)) * 0.3
    i, j = np.arange(nq)[:, None] + shift, np.arange(nk)[None]
    mask = (j <= i) & ((i - j < window) if window else True)
    s = np.where(mask, s, -np.inf)
    with np.errstate(invalid="ignore"):
        e = np.where(mask, np.exp(s - s.max(-1, keepdims=True)), 0)
    w = e / np.maximum(e.sum(-1, keepdims=True), 1e-300)
    assert np.allclose(out, np.einsum("hij,jhd->ihd", w, np.repeat(v, 2, 1)))
    assert (tol >= 0).all() and (out[~mask.any(1)] == 0).all()


@pytest.mark.parametrize("nq,nk,window,kind", [(40, 40, 0, "bf16"), (33, 90, 20, "fp16"), (50, 20, 0, "bf16"),
                                               (30, 10, 4, "fp16"), (5, 0, 0, "bf16"), (1, 200, 0, "fp16")])
def test_the_two_forms_of_the_attention_agree(nq, nk, window, kind):
    from paged_reference import attend_matrix
    rng = np.random.default_rng(nq)
    q, k, v = (rng.standard_normal((n, h, 16)) for n, h in ((nq, 4), (nk, 2), (nk, 2)))
    for scale in (0.25, -1.0, 0.0):
        a, b = (f(q, k, v, nk - nq, window, scale, kind) for f in (attend, attend_matrix))
        assert np.allclose(a[0], b[0], rtol=0, atol=1e-12) and np.allclose(a[1], b[1], rtol=1e-9, atol=1e-30)
