"""The paged KV cache, the attention over it and the prompt attention on the GPU, against the
64-bit reference in paged_reference.py."""
import numpy as np
import pytest

from paged_reference import Pages, attend, attend_matrix

pytestmark = pytest.mark.gpu


def _mods():
    import torch
    import moe_decode_megakernel_warp_gb300 as msm
    return torch, msm


def _dtype(kind):
    torch, _ = _mods()
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[kind]


def randn(kind, *shape, seed=0, std=1.0):
    torch, _ = _mods()
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * std).to(_dtype(kind))


def f64(t):
    return t.detach().cpu().double().numpy()


def ints(values):
    torch, _ = _mods()
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _dtype_tensor(kind, values):
    torch, _ = _mods()
    return torch.from_numpy(np.asarray(values)).to(_dtype(kind))


def starts_of(lens):
    return [int(x) for x in np.concatenate([[0], np.cumsum(lens)])]


def bits(t):
    torch, _ = _mods()
    return t.contiguous().view(torch.int16).cpu().numpy()


def assert_close(got, want, tol, what=""):
    got = f64(got)
    assert not np.isnan(got).any(), what
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound at %s" % (
        what, bad.sum(), bad.size, (np.abs(got - want) / tol).max(),
        np.unravel_index((np.abs(got - want) / tol).argmax(), got.shape))


# ------------------------------------------------------------------ page operations
class Both:
    """A cache on the GPU and its reference, called alike and compared after every call."""

    def __init__(self, rng, layers, n_pages, rows, heads, hd, n_seqs, max_pages, kind="bf16"):
        torch, msm = _mods()
        self.kind = kind
        shape = (n_pages, heads, rows, hd)
        k = [randn(kind, *shape, seed=int(rng.integers(1 << 30))) for _ in range(layers)]
        v = [randn(kind, *shape, seed=int(rng.integers(1 << 30))) for _ in range(layers)]
        self.gpu = msm.PagedCache([t.cuda() for t in k], [t.cuda() for t in v], ints([[-1] * max_pages] * n_seqs),
                                  ints([0] * n_seqs), ints([0] * n_pages))
        self.ref = Pages(n_pages, rows, n_seqs, max_pages, [bits(t).copy() for t in k + v])

    def same(self):
        g, r = self.gpu, self.ref
        assert np.array_equal(g.table.cpu().numpy(), r.table)
        assert np.array_equal(g.lens.cpu().numpy(), r.lens)
        assert np.array_equal(g.refs.cpu().numpy(), r.refs)
        for a, b in zip(g.k_pages + g.v_pages, r.pools):
            assert np.array_equal(bits(a), b)

    def call(self, name, arg=None):
        torch, msm = _mods()
        args = () if arg is None else (ints(arg),)
        getattr(self.gpu, name)(*args)
        err = getattr(self.ref, name)(*(() if arg is None else (arg,)))
        if err is None:
            self.gpu.sync()
        else:
            with pytest.raises(msm.MsmError, match=name) as e:
                self.gpu.sync()
            assert msm.STATUS_NAMES[e.value.code] == err
            self.gpu.sync()  # cleared
        self.same()
        return err

    def write(self, counts, seed):
        torch, _ = _mods()
        st = starts_of(counts)
        heads, hd = self.gpu.k_pages[0].shape[1], self.gpu.k_pages[0].shape[3]
        for layer in range(len(self.gpu.k_pages)):
            # both out of one packed tensor, and a row behind the last sequence
            kv = randn(self.kind, st[-1] + 1, 2 * heads, hd, seed=seed + layer).cuda()
            self.gpu.write(layer, kv[:, :heads], kv[:, heads:], ints(st))
            rows = bits(kv)
            self.ref.write(self.ref.pools[layer], rows[:, :heads], st)
            self.ref.write(self.ref.pools[len(self.gpu.k_pages) + layer], rows[:, heads:], st)
        self.gpu.sync()
        self.same()


@pytest.mark.parametrize("rows,heads,hd,kind", [(16, 2, 64, "bf16"), (1, 1, 128, "fp16"), (7, 3, 64, "fp16"),
                                                (64, 8, 128, "bf16"), (33, 1, 64, "bf16")])
def test_random_calls_equal_the_reference(rows, heads, hd, kind):
    rng = np.random.default_rng(rows)
    n_seqs, max_pages = 9, 6
    c = Both(rng, 2, 40, rows, heads, hd, n_seqs, max_pages, kind)
    for step in range(14):
        new = [-1 if rng.random() < 0.3 else int(rng.integers(0, max_pages * rows + 1)) for _ in range(n_seqs)]
        old = c.ref.lens.copy()
        if c.call("resize", new) is None:
            c.write(np.maximum(c.ref.lens - old, 0), 100 * step)
        if step % 2:
            parent = [-1] * n_seqs
            live = [s for s in range(n_seqs) if c.ref.lens[s] > 0]
            for s in range(n_seqs):
                if c.ref.lens[s] == 0 and live:
                    parent[s] = int(rng.choice(live))
            c.call("fork", parent)
        if step % 3 == 2:
            c.call("compact")
    c.ref.check()


def test_a_shared_last_page_is_copied_once_for_each_that_grows():
    rng = np.random.default_rng(3)
    c = Both(rng, 3, 12, 16, 2, 64, 4, 3)
    c.call("resize", [20, 0, 0, 0])
    c.write([20, 0, 0, 0], 1)
    c.call("fork", [-1, 0, 0, -1])
    assert list(c.ref.refs[:2]) == [3, 3]
    c.call("resize", [-1, 21, -1, -1])    # one child leaves the shared page
    c.write([0, 1, 0, 0], 2)
    c.call("resize", [21, 21, 22, -1])    # the parent and the other child both do
    c.write([1, 0, 2, 0], 3)
    c.call("resize", [5, 0, 17, -1])      # back into the shared first page
    c.call("resize", [6, -1, -1, -1])     # which the growth must leave
    c.write([1, 0, 0, 0], 4)
    c.ref.check()


@pytest.mark.parametrize("n_pages", [60000, 150001])
def test_a_pool_of_many_pages_and_sequences(n_pages):
    rng = np.random.default_rng(4)
    n_seqs, rows = 1500, 2
    c = Both(rng, 1, n_pages, rows, 1, 64, n_seqs, 40)
    if n_pages > 100000:  # the free pages begin far behind the front
        c.gpu.refs[:99990] = 1
        c.ref.refs[:99990] = 1
    for i in range(3):
        c.call("resize", [int(x) for x in rng.integers(0, 40 * rows + 1, n_seqs)])
    c.call("resize", [0 if s % 3 else -1 for s in range(n_seqs)])
    c.call("fork", [s - s % 3 if s % 3 else -1 for s in range(n_seqs)])
    if n_pages > 100000:
        c.gpu.refs[:99990] = 0
        c.ref.refs[:99990] = 0
    c.call("compact")
    c.call("resize", [int(n) + 1 if n < 80 else -1 for n in c.ref.lens])
    c.ref.check()


def test_more_layers_than_one_copy_launch_carries():
    rng = np.random.default_rng(5)
    c = Both(rng, 70, 9, 4, 1, 64, 3, 3)
    c.call("resize", [6, 5, 0])
    c.call("fork", [-1, -1, 0])
    c.call("resize", [7, 0, 8])
    c.call("compact")
    c.ref.check()


def test_refusals_on_the_device_change_nothing():
    rng = np.random.default_rng(6)
    c = Both(rng, 1, 6, 16, 1, 64, 4, 4)
    c.call("resize", [30, 10, 0, 0])
    assert c.call("resize", [-1, -1, 64, 1]) == "MSM_ERR_OOM"
    assert c.call("resize", [0, 0, 65, 0]) == "MSM_ERR_INVALID_ARG"
    assert c.call("resize", [-2, -1, -1, -1]) == "MSM_ERR_INVALID_ARG"
    for parent in ([-1, -1, 2, -1], [-1, -1, 4, -1], [-1, -1, -2, -1], [-1, 0, -1, -1], [-1, -1, 3, 0]):
        assert c.call("fork", parent) == "MSM_ERR_INVALID_ARG"
    # the OOM is about the pages free before the call: a second call has those that the first gave up
    assert c.call("resize", [0, -1, 64, -1]) == "MSM_ERR_OOM"
    assert c.call("resize", [0, -1, -1, -1]) is None
    assert c.call("resize", [-1, -1, 64, -1]) is None


def contents(c):
    return [t.clone() for t in [c.table, c.lens, c.refs] + c.k_pages + c.v_pages]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("what", ["oom", "length", "fork"])
def test_nothing_changes_between_a_refused_call_and_its_report(what, captured):
    """Full pages, held once: the rows of a write behind a resize that found no page would
    replace the last ones of the history."""
    torch, msm = _mods()
    c = Both(np.random.default_rng(30), 2, 5, 16, 2, 64, 4, 4)
    c.call("resize", [32, 16, 0, 0])
    g = c.gpu
    kv = randn("bf16", 5, 2, 64, seed=1).cuda()
    st = ints([0, 4, 5, 5, 5])
    bad, grow, shrink = ints({"length": [65, 17, -1, -1]}.get(what, [64, 17, -1, -1])), ints([36, 17, 0, 0]), ints([1, 0, 0, 0])
    parents, wrong = ints([-1, -1, 0, -1]), ints([-1, 0, -1, -1])

    def step():
        if what == "fork":
            g.fork(wrong)
        else:
            g.resize(bad)
        for layer in range(2):
            g.write(layer, kv, kv, st)
        g.fork(parents)
        g.write(0, kv, kv, st)
        g.resize(grow)
        g.resize(shrink)
        g.compact()
        g.write(0, kv[:1], kv[:1], ints_1)
    ints_1 = ints([0, 1, 1, 1, 1])
    # a hole in front of the pages in use, for compact
    c.call("resize", [-1, -1, 5, -1])
    c.call("resize", [16, -1, -1, -1])
    c.call("resize", [0, -1, -1, -1])
    c.call("resize", [16, 16, 0, -1])
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    before = contents(g)
    for _ in range(2):
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(before, contents(g)))
        q = randn("bf16", 4, 2, 64, seed=2).cuda()
        seen = g.attention(0, q)  # the sequences as they stand
        with pytest.raises(msm.MsmError, match="msm_pages_fork" if what == "fork" else "msm_pages_resize") as e:
            g.sync()
        assert msm.STATUS_NAMES[e.value.code] == ("MSM_ERR_OOM" if what == "oom" else "MSM_ERR_INVALID_ARG")
        assert np.array_equal(bits(seen), bits(g.attention(0, q)))
    # reported: the calls work again
    c.call("resize", [20, 17, -1, -1])
    c.write([4, 1, 0, 0], 5)
    c.call("fork", [-1, -1, 0, -1])
    c.call("compact")


def test_an_earlier_error_does_not_hide_a_refusal():
    """A write that left a token out stops nothing, but the refused resize behind it does."""
    torch, msm = _mods()
    c = Both(np.random.default_rng(31), 1, 3, 16, 2, 64, 2, 4)
    c.call("resize", [32, 3])
    g, kv = c.gpu, randn("bf16", 5, 2, 64, seed=1).cuda()
    g.write(0, kv, kv, ints([0, 0, 5]))   # two of the five tokens have no row
    g.write(0, kv, kv, ints([0, 1, 1]))   # stored
    torch.cuda.synchronize()
    c.ref.write(c.ref.pools[0], bits(kv)[2:], [0, 0, 3])
    c.ref.write(c.ref.pools[1], bits(kv)[2:], [0, 0, 3])
    c.ref.write(c.ref.pools[0], bits(kv), [0, 1, 1])
    c.ref.write(c.ref.pools[1], bits(kv), [0, 1, 1])
    c.same()
    g.resize(ints([36, -1]))
    g.write(0, kv, kv, ints([0, 4, 4]))
    with pytest.raises(msm.MsmError, match="msm_pages_write"):
        g.sync()
    c.same()
    g.sync()


def test_write_leaves_out_tokens_without_a_row_of_their_own():
    torch, msm = _mods()
    rng = np.random.default_rng(7)
    c = Both(rng, 1, 6, 16, 2, 64, 3, 2)
    c.call("resize", [20, 3, 0])
    c.call("fork", [-1, -1, 0])
    k = randn("bf16", 9, 2, 64).cuda()
    for st in ([0, 2, 2, 2],      # a shared page
               [0, 0, 4, 4],      # one row more than the sequence has: its first token has none
               [0, 0, 0, 1]):     # a shared page through the child
        before = [bits(t) for t in c.gpu.k_pages + c.gpu.v_pages]
        c.gpu.write(0, k, k, ints(st))
        with pytest.raises(msm.MsmError, match="msm_pages_write"):
            c.gpu.sync()
        if st == [0, 0, 4, 4]:
            c.ref.write(c.ref.pools[0], bits(k)[1:], [0, 0, 3, 3])
            c.ref.write(c.ref.pools[1], bits(k)[1:], [0, 0, 3, 3])
        else:
            assert all(np.array_equal(a, bits(b)) for a, b in zip(before, c.gpu.k_pages + c.gpu.v_pages))
        c.same()


def test_tables_that_name_pages_outside_the_pool():
    torch, msm = _mods()
    for bad in (-1, -5, 6, 1 << 30):
        c = Both(np.random.default_rng(8), 1, 6, 16, 1, 64, 2, 3)
        c.call("resize", [40, 10])
        c.gpu.table[0, 2] = bad
        for call in (lambda: c.gpu.resize(ints([1, -1])), lambda: c.gpu.resize(ints([41, -1])),
                     lambda: c.gpu.resize(ints([0, 0]))):
            call()
            with pytest.raises(msm.MsmError, match="msm_pages_resize"):
                c.gpu.sync()
        k = randn("bf16", 1, 1, 64).cuda()
        c.gpu.write(0, k, k, ints([0, 1, 1]))
        with pytest.raises(msm.MsmError, match="msm_pages_write"):
            c.gpu.sync()
        out = c.gpu.attention(0, randn("bf16", 2, 2, 64).cuda())
        with pytest.raises(msm.MsmError, match="msm_paged_attention"):
            c.gpu.sync()
        assert not torch.isnan(out).any()  # the rows on the other pages are there
        c.gpu.compact()
        c.gpu.sync()
        assert c.gpu.table[0, 2].item() == bad
        c.gpu.table[0, 2] = int(c.ref.table[0, 2])
        c.same()


# ------------------------------------------------------------------ paged attention
def filled(rng, kind, lens, rows, hkv, hd, extra=5, max_pages=None):
    """A cache of the given lengths on random pages; every row that no sequence holds is NaN."""
    torch, msm = _mods()
    per = [-(-n // rows) for n in lens]
    n_pages = sum(per) + extra
    order = rng.permutation(n_pages)
    width = max_pages or max(1, max(per))
    table, refs, at = np.full((len(lens), width), -7, np.int64), np.zeros(n_pages, np.int64), 0
    k = torch.full((n_pages, hkv, rows, hd), float("nan"), dtype=_dtype(kind))
    v = torch.full_like(k, float("nan"))
    rows_k, rows_v = [], []
    for s, n in enumerate(lens):
        kk = randn(kind, n, hkv, hd, seed=int(rng.integers(1 << 30)))
        vv = randn(kind, n, hkv, hd, seed=int(rng.integers(1 << 30)))
        for j in range(per[s]):
            p = int(order[at])
            at += 1
            table[s, j], refs[p] = p, 1
            part = slice(j * rows, min(n, (j + 1) * rows))
            cnt = part.stop - part.start
            k[p, :, :cnt] = kk[part].transpose(0, 1)
            v[p, :, :cnt] = vv[part].transpose(0, 1)
        rows_k.append(kk)
        rows_v.append(vv)
    c = msm.PagedCache([k.cuda()], [v.cuda()], ints(table.tolist()), ints(lens), ints(refs.tolist()))
    return c, rows_k, rows_v


def decode_want(q, rows_k, rows_v, window, scale, kind):
    outs, tols = [], []
    for s in range(len(rows_k)):
        n = rows_k[s].shape[0]
        o, t = attend(f64(q[s:s + 1]), f64(rows_k[s]), f64(rows_v[s]), n - 1, window, scale, kind)
        outs.append(o)
        tols.append(t)
    return np.concatenate(outs), np.concatenate(tols)


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 255, 300, 1000]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("hkv,group", [(1, 1), (2, 8), (8, 4), (3, 2)])
@pytest.mark.parametrize("rows", [16, 64, 1, 13])
def test_paged_attention_equals_the_formula(kind, hd, hkv, group, rows):
    rng = np.random.default_rng(hd + rows + group)
    c, rk, rv = filled(rng, kind, LENS, rows, hkv, hd)
    q = randn(kind, len(LENS), hkv * group, hd, seed=9).cuda()
    for window in (0, 1, 20, 128):
        got = c.attention(0, q, window=window)
        c.sync()
        want, tol = decode_want(q, rk, rv, window, hd ** -0.5, kind)
        assert_close(got, want, tol, "window %d" % window)


def test_paged_windows_longer_than_the_sequences():
    rng = np.random.default_rng(17)
    c, _, _ = filled(rng, "bf16", LENS, 16, 2, 64)
    q = randn("bf16", len(LENS), 4, 64, seed=9).cuda()
    want = bits(c.attention(0, q))
    for window in (1000, 1001, 2 ** 30, 2 ** 31 - 1):
        assert np.array_equal(bits(c.attention(0, q, window=window)), want)


@pytest.mark.parametrize("kind,lens,rows,window", [
    ("bf16", [40000], 64, 0), ("fp16", [33001, 7], 48, 0), ("bf16", [20000] * 3, 16, 5000),
    ("bf16", [1] * 700, 16, 0), ("fp16", [100 + 3 * i for i in range(300)], 32, 0), ("bf16", [39999, 0, 0, 1], 100, 0)])
def test_long_and_many_sequences(kind, lens, rows, window):
    rng = np.random.default_rng(len(lens))
    c, rk, rv = filled(rng, kind, lens, rows, 2, 128)
    q = randn(kind, len(lens), 4, 128, seed=2).cuda()
    got = c.attention(0, q, window=window)
    c.sync()
    want, tol = decode_want(q, rk, rv, window, 128 ** -0.5, kind)
    assert_close(got, want, tol)
    for _ in range(3):  # the split does not change a bit
        assert np.array_equal(bits(c.attention(0, q, window=window)), bits(got))


def test_scales_and_large_scores():
    rng = np.random.default_rng(11)
    lens = [50, 700, 16]
    for scale, std in ((1.0, 1.0), (-0.2, 1.0), (0.0, 1.0), (0.125, 8.0)):
        c, rk, rv = filled(rng, "bf16", lens, 16, 2, 64)
        q = randn("bf16", 3, 4, 64, seed=3, std=std).cuda()
        want, tol = decode_want(q, rk, rv, 0, scale, "bf16")
        assert_close(c.attention(0, q, scale=scale), want, tol, "scale %g" % scale)


def test_infinities_and_nan_reach_only_the_rows_that_see_them():
    torch, _ = _mods()
    rng = np.random.default_rng(12)
    c, rk, rv = filled(rng, "bf16", [100, 100, 100, 100], 16, 1, 64)
    at = lambda s, r: (int(c.table[s, r // 16]), 0, r % 16)
    c.k_pages[0][at(0, 10)] = float("nan")
    c.v_pages[0][at(1, 10)][3] = float("inf")
    c.k_pages[0][at(2, 99)] = float("inf")
    q = randn("bf16", 4, 2, 64, seed=1).cuda()
    seen = c.attention(0, q).cpu()
    assert torch.isnan(seen[0]).all()
    assert (seen[1, :, 3] == float("inf")).all() and torch.isfinite(seen[1, :, :3]).all()
    assert torch.isnan(seen[2]).any()
    want, tol = decode_want(q, rk, rv, 0, 0.125, "bf16")
    assert_close(seen[3:], want[3:], tol[3:])
    # behind a window the first two are clean
    want, tol = decode_want(q, rk, rv, 89, 0.125, "bf16")
    assert_close(c.attention(0, q, window=89)[:2], want[:2], tol[:2])
    # scores that are all -inf: 0 / 0, as the formula has it
    c.k_pages[0].fill_(float("-inf"))
    assert torch.isnan(c.attention(0, q.abs())).all()


def test_strided_queries_and_results():
    torch, _ = _mods()
    rng = np.random.default_rng(13)
    c, rk, rv = filled(rng, "fp16", [37, 200, 0], 16, 2, 64)
    qkv = randn("fp16", 3, 8 + 4, 64, seed=4).cuda()
    big = torch.full((3, 16, 3, 64), 7.0, dtype=torch.float16, device="cuda")
    out = big[:, ::2, 1]
    got = c.attention(0, qkv[:, :8], out=out)
    assert got is out
    want, tol = decode_want(qkv[:, :8], rk, rv, 0, 0.125, "fp16")
    assert_close(out, want, tol)
    big[:, ::2, 1] = 7.0
    assert (big == 7.0).all()


def test_lengths_beyond_the_table_are_cut_off():
    torch, _ = _mods()
    rng = np.random.default_rng(14)
    c, rk, rv = filled(rng, "bf16", [32, 20], 16, 1, 64)
    q = randn("bf16", 2, 1, 64).cuda()
    want = bits(c.attention(0, q))
    c.lens.copy_(ints([1 << 30, 20]))
    assert np.array_equal(bits(c.attention(0, q)), want)
    c.lens.copy_(ints([-3, 20]))
    got = c.attention(0, q)
    assert (got[0] == 0).all() and np.array_equal(bits(got[1:]), want[1:])


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("hd,group,rows", [(64, 4, 16), (128, 8, 64), (128, 1, 7)])
def test_weights_keep_more_than_16_bits(kind, hd, group, rows):
    """Random sequences; values that cancel, where equal weights all err the same way; and many
    small weights beside a large one: within the bound of weights in two terms."""
    torch, msm = _mods()
    rng = np.random.default_rng(19)
    c, rk, rv = filled(rng, kind, LENS + [5000, 5000, 40000], rows, 2, hd)
    n = len(LENS)
    q = randn(kind, n + 3, 2 * group, hd, seed=9)
    q[n:] = 0
    q[n:, :, 0] = 1

    def put(s, k0, v):   # keys (k0, 0, 0, ...), values v
        k = torch.zeros((len(k0), 2, hd), dtype=_dtype(kind))
        k[:, :, 0] = torch.from_numpy(k0).to(_dtype(kind))[:, None]
        v = torch.from_numpy(v).to(_dtype(kind))[:, None, None].expand(len(k0), 2, hd)
        rk[s], rv[s] = k, v
        for r0 in range(0, len(k0), rows):
            page = int(c.table[s, r0 // rows])
            c.k_pages[0][page, :, :len(k0) - r0] = k[r0:r0 + rows].transpose(0, 1).cuda()
            c.v_pages[0][page, :, :len(k0) - r0] = v[r0:r0 + rows].transpose(0, 1).cuda()
    # scores 0 with value 1, and a score whose weight is far from a 16-bit one with value -1,
    # as many as make the sum almost zero
    for s, score in ((n, -0.6875), (n + 1, -2.421875)):
        e = np.exp(score)
        one = int(5000 * e / (1 + e))
        put(s, np.where(np.arange(5000) < one, 0.0, score), np.where(np.arange(5000) < one, 1.0, -1.0))
    # 39,999 weights of e^-17.75 (2^-25.6) beside one of 1
    put(n + 2, np.where(np.arange(40000) == 7, 0.0, -17.75), np.where(np.arange(40000) == 7, 0.0, 1.0))
    q = q.cuda()
    for window, scale in ((0, hd ** -0.5), (0, 1.0), (300, 1.0)):
        got = c.attention(0, q, window=window, scale=scale)
        c.sync()
        for s in range(n + 3):
            want, tol = attend_matrix(f64(q[s:s + 1]), f64(rk[s]), f64(rv[s]), len(rk[s]) - 1, window, scale, kind, 2)
            assert_close(got[s:s + 1], want, tol, "sequence %d window %d scale %g" % (s, window, scale))


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_infinite_values_under_small_weights(kind):
    """Not NaN: every weight above 0 passes an infinite value on."""
    torch, msm = _mods()
    c, rk, rv = filled(np.random.default_rng(23), kind, [300], 16, 1, 64)
    q = torch.zeros((1, 8, 64), dtype=_dtype(kind), device="cuda")
    q[0, :, 0] = 1
    for r in (0, 150, 299):
        for score in (0.0, -0.5, -2.0, -5.5, -9.0, -13.0):
            k = torch.zeros((300, 64), dtype=_dtype(kind))
            k[r, 0] = score
            v = randn(kind, 300, 64, seed=1)
            v[r, 3], v[r, 4] = float("inf"), float("-inf")
            for j in range(0, 300, 16):
                page = int(c.table[0, j // 16])
                c.k_pages[0][page, 0, :len(k[j:j + 16])] = k[j:j + 16].cuda()
                c.v_pages[0][page, 0, :len(v[j:j + 16])] = v[j:j + 16].cuda()
            out = c.attention(0, q, scale=1.0)[0].cpu()
            assert (out[:, 3] == float("inf")).all() and (out[:, 4] == float("-inf")).all(), (r, score)
            assert torch.isfinite(out[:, 5:]).all()


@pytest.mark.parametrize("kind,hd", [("bf16", 64), ("fp16", 128)])
@pytest.mark.parametrize("group", [1, 4, 8])
def test_sequences_whose_rows_are_all_on_pages_outside_the_pool(kind, hd, group):
    """Zeros, as for a sequence without rows, in one block's work and in parts that are joined; one
    row left gives that row; scores that are all -inf stay NaN."""
    torch, msm = _mods()
    rng = np.random.default_rng(18)
    lens = [5, 100, 12000, 200, 40000, 12000, 90, 0]
    c, rk, rv = filled(rng, kind, lens, 16, 2, hd)
    q = randn(kind, len(lens), 2 * group, hd, seed=1).cuda().abs()
    c.table[0, 0] = -1
    c.table[2] = 1 << 30
    c.table[4] = -5
    c.table[5, :700] = c.table.shape[1] * 1000
    c.k_pages[0][c.table[6, :6].long()] = float("-inf")

    def lost():
        with pytest.raises(msm.MsmError, match="msm_paged_attention"):
            c.sync()
    out = c.attention(0, q)
    lost()
    assert all((out[s] == 0).all() for s in (0, 2, 4, 7))
    assert torch.isnan(out[6]).all()
    rest = [s for s in range(len(lens)) if s in (1, 3)]
    want, tol = decode_want(q[rest], [rk[s] for s in rest], [rv[s] for s in rest], 0, hd ** -0.5, kind)
    assert_close(out[rest], want, tol)
    want, tol = decode_want(q[5:6], [rk[5][11200:]], [rv[5][11200:]], 0, hd ** -0.5, kind)
    assert_close(out[5:6], want, tol)
    # a window that lies on such a page, and one that has one row more
    c.table[1, 6] = -2   # rows 96 .. 99
    out = c.attention(0, q, window=4)
    lost()
    assert all((out[s] == 0).all() for s in (0, 1, 2, 4, 7))
    out = c.attention(0, q, window=5)
    lost()
    assert np.array_equal(f64(out[1]), np.repeat(f64(rv[1][95]), group, axis=0))


@pytest.mark.parametrize("lens", [[0, 0, 0], [0] * 400, [0] * 150 + [77] + [0] * 300 + [200, 0, 1] + [0] * 90])
def test_batches_of_mostly_empty_slots(lens):
    rng = np.random.default_rng(16)
    c, rk, rv = filled(rng, "bf16", lens, 16, 2, 64)
    q = randn("bf16", len(lens), 8, 64, seed=6).cuda()
    want, tol = decode_want(q, rk, rv, 0, 0.125, "bf16")
    assert_close(c.attention(0, q), want, tol)
    c.sync()


def test_the_wrappers_refuse_what_does_not_fit():
    torch, msm = _mods()
    rng = np.random.default_rng(15)
    c, _, _ = filled(rng, "bf16", [32, 20], 16, 2, 64)
    q = randn("bf16", 2, 4, 64).cuda()
    for bad in (q[:1], q.half(), q.cpu(), q[:, :, :32], q.transpose(1, 2).contiguous().transpose(1, 2), q[0]):
        with pytest.raises(ValueError):
            c.attention(0, bad)
    with pytest.raises(ValueError):
        c.attention(0, q, out=q[:1])
    with pytest.raises(msm.MsmError):
        c.attention(1, q)
    with pytest.raises(msm.MsmError, match="1, 2, 4 or 8"):
        c.attention(0, randn("bf16", 2, 6, 64).cuda())
    with pytest.raises(ValueError):
        c.resize(ints([1]))
    with pytest.raises(ValueError):
        c.fork(torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        c.write(0, q, q, ints([0, 1, 2]))
    with pytest.raises(ValueError):
        msm.prompt_attention(q, q[:1], q, ints([0, 2]))
    with pytest.raises(ValueError):
        msm.prompt_attention(q.float(), q.float(), q.float(), ints([0, 2]))
    with pytest.raises(msm.MsmError, match="strides"):
        msm.prompt_attention(q, q[:1].expand(2, 4, 64), q, ints([0, 2]))
    c.sync()


def test_tables_of_more_than_2_to_the_30_pages():
    """The needs of sequences whose tables hold more pages than any pool (a 4.3 GB table): no
    page left, and nothing changed; ordinary lengths in such a table are served."""
    torch, msm = _mods()
    for n_seqs, width, new in ((1, (1 << 30) + 64, [(1 << 30) + 1]), (1, (1 << 30) + 64, [1 << 30]),
                               (2, (1 << 29) + 64, [(1 << 29) + 1, (1 << 29) + 7]), (1, (1 << 30) + 64, [9])):
        pool = torch.zeros((8, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
        table = torch.empty((n_seqs, width), dtype=torch.int32, device="cuda")
        c = msm.PagedCache([pool], [pool.clone()], table, ints([0] * n_seqs), ints([0] * 8))
        c.resize(ints([3] + [0] * (n_seqs - 1)))
        c.sync()
        kept = [c.lens.clone(), c.refs.clone(), table[:, :16].clone()]
        c.resize(ints(new))
        with pytest.raises(msm.MsmError, match="no free page"):
            c.sync()
        assert all(torch.equal(a, b) for a, b in zip(kept, (c.lens, c.refs, table[:, :16])))
        c.resize(ints([8] + [0] * (n_seqs - 1)))
        c.sync()
        assert table[0, :8].tolist() == list(range(8)) and (c.refs == 1).all()
        del pool, table, c


def test_integers_beyond_32_bits():
    """Windows that hide nothing; layers that are none; not their low 32 bits."""
    torch, msm = _mods()
    c, _, _ = filled(np.random.default_rng(25), "bf16", [300, 40], 16, 2, 64)
    q = randn("bf16", 2, 4, 64).cuda()
    kv = randn("bf16", 100, 2, 64, seed=1).cuda()
    qq, st = randn("bf16", 100, 4, 64, seed=2).cuda(), ints([0, 100])
    want, p_want = bits(c.attention(0, q)), bits(msm.prompt_attention(qq, kv, kv, st))
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1, 10 ** 30):
        assert np.array_equal(bits(c.attention(0, q, window=window)), want)
        assert np.array_equal(bits(msm.prompt_attention(qq, kv, kv, st, window=window)), p_want)
    for window in (-1, -2 ** 31, -2 ** 32, 5 - 2 ** 32):
        with pytest.raises(msm.MsmError, match="window"):
            c.attention(0, q, window=window)
        with pytest.raises(msm.MsmError, match="window"):
            msm.prompt_attention(qq, kv, kv, st, window=window)
    before = contents(c)
    for layer in (1, -1, 2 ** 32, -2 ** 32):
        with pytest.raises(msm.MsmError, match="layer"):
            c.attention(layer, q)
        with pytest.raises(msm.MsmError, match="layer"):
            c.write(layer, kv, kv, ints([0, 100, 100]))
    with pytest.raises(ValueError, match="tokens"):
        c.write(0, kv[:1].expand(2 ** 32 + 1, 2, 64), kv[:1].expand(2 ** 32 + 1, 2, 64), ints([0, 1, 1]))
    torch.cuda.synchronize()
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(before, contents(c)))


def test_pools_of_more_than_2_to_the_31_elements():
    """The last pages of a 4.6 GB pool: written, read, copied and moved."""
    torch, msm = _mods()
    n_pages, rows, hkv, hd = 4400, 1024, 8, 64
    c = msm.PagedCache.allocate(1, n_pages, rows, hkv, hd, 2, 3)
    assert c.k_pages[0].numel() > 1 << 31
    c.refs.fill_(1)
    c.refs[n_pages - 4:] = 0
    c.resize(ints([1100, 0]))
    kv = randn("bf16", 1100, 2 * hkv, hd, seed=1).cuda()
    c.write(0, kv[:, :hkv], kv[:, hkv:], ints([0, 1100, 1100]))
    c.sync()
    assert c.table[0].tolist() == [n_pages - 4, n_pages - 3, -1]
    assert torch.equal(c.k_pages[0][n_pages - 3, :, :76], kv[1024:, :hkv].transpose(0, 1))
    q = randn("bf16", 2, hkv, hd, seed=2).cuda()
    rows_k, rows_v = [kv[:, :hkv]] * 2, [kv[:, hkv:]] * 2
    c.fork(ints([-1, 0]))
    c.resize(ints([-1, 1101]))
    new = randn("bf16", 1, 2 * hkv, hd, seed=3).cuda()
    c.write(0, new[:, :hkv], new[:, hkv:], ints([0, 0, 1]))
    rows_k[1], rows_v[1] = torch.cat([rows_k[1], new[:, :hkv]]), torch.cat([rows_v[1], new[:, hkv:]])
    c.sync()
    assert c.table[1].tolist() == [n_pages - 4, n_pages - 2, -1]
    want, tol = decode_want(q, rows_k, rows_v, 0, 0.125, "bf16")
    assert_close(c.attention(0, q), want, tol)
    c.refs[:n_pages - 4] = 0
    c.compact()
    c.sync()
    assert c.table.tolist() == [[0, 1, -1], [0, 2, -1]]
    assert_close(c.attention(0, q), want, tol)


# ------------------------------------------------------------------ prompt attention
def prompt_want(q, k, v, qs, ks, window, scale, kind):
    out, tol = np.zeros(q.shape), np.full(q.shape, 1e-30)
    for s in range(len(qs) - 1):
        a, b = slice(qs[s], qs[s + 1]), slice(ks[s], ks[s + 1])
        o, t = attend(f64(q[a]), f64(k[b]), f64(v[b]), (b.stop - b.start) - (a.stop - a.start), window, scale, kind)
        out[a], tol[a] = o, t
    return out, tol


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("hkv,group", [(1, 1), (1, 8), (2, 4), (3, 2)])
def test_prompt_attention_equals_the_formula(kind, hd, hkv, group):
    _, msm = _mods()
    lens = [1, 0, 17, 64, 5, 130, 257, 31]
    st = starts_of(lens)
    qkv = randn(kind, st[-1], (group + 2) * hkv, hd, seed=hd + group).cuda()
    q, k, v = qkv[:, :hkv * group], qkv[:, hkv * group:hkv * (group + 1)], qkv[:, hkv * (group + 1):]
    for window in (0, 1, 40, 128):
        got = msm.prompt_attention(q, k, v, ints(st), window=window)
        want, tol = prompt_want(q, k, v, st, st, window, hd ** -0.5, kind)
        assert_close(got, want, tol, "window %d" % window)


@pytest.mark.parametrize("hd,group", [(64, 2), (128, 8)])
@pytest.mark.parametrize("qlens,klens", [([3, 40, 1], [300, 40, 129]), ([1, 1, 1], [1, 128, 513]),
                                         ([70, 20], [30, 0]), ([200], [500]), ([5, 5], [0, 5])])
def test_resumed_prompts_and_rows_without_keys(hd, group, qlens, klens):
    torch, msm = _mods()
    qs, ks = starts_of(qlens), starts_of(klens)
    q = randn("bf16", qs[-1], 2 * group, hd, seed=1).cuda()
    # the keys in a verify-step cache's order, NaN behind the last one
    kc = torch.full((2, ks[-1] + 9, hd), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    kc[:, :ks[-1]] = randn("bf16", 2, ks[-1], hd, seed=2).cuda()
    vc[:, :ks[-1]] = randn("bf16", 2, ks[-1], hd, seed=3).cuda()
    k, v = kc.transpose(0, 1), vc.transpose(0, 1)
    for window in (0, 33):
        got = msm.prompt_attention(q, k, v, ints(qs), ints(ks), window=window)
        want, tol = prompt_want(q, k[:ks[-1]], v[:ks[-1]], qs, ks, window, hd ** -0.5, "bf16")
        assert_close(got, want, tol, "window %d" % window)


@pytest.mark.parametrize("qlens,klens", [([70, 20], [30, 0]), ([20], [10]), ([300, 5], [40, 700]), ([40], [40])])
@pytest.mark.parametrize("window", [40, 45, 700, 740, 2 ** 30, 2 ** 31 - 1])
def test_windows_longer_than_the_keys(qlens, klens, window):
    """Up to the largest one, which callers pass for none; queries in front of the first key."""
    torch, msm = _mods()
    qs, ks = starts_of(qlens), starts_of(klens)
    q, k, v = (randn("bf16", n, h, 64, seed=h).cuda() for n, h in ((qs[-1], 4), (ks[-1], 2), (ks[-1], 1)))
    v = v.expand(-1, 2, 64).contiguous()
    got = msm.prompt_attention(q, k, v, ints(qs), ints(ks), window=window)
    want, tol = prompt_want(q, k, v, qs, ks, window, 0.125, "bf16")
    assert_close(got, want, tol)


@pytest.mark.parametrize("kind,n,hq,hkv,hd,window", [("bf16", 1500, 2, 1, 128, 0), ("fp16", 1100, 1, 1, 64, 0),
                                                     ("bf16", 1300, 4, 1, 64, 300), ("fp16", 900, 8, 1, 128, 257)])
def test_longer_prompts(kind, n, hq, hkv, hd, window):
    _, msm = _mods()
    q, k, v = (randn(kind, n, h, hd, seed=h + i).cuda() for i, h in enumerate((hq, hkv, hkv)))
    got = msm.prompt_attention(q, k, v, ints([0, n]), window=window)
    want, tol = prompt_want(q, k, v, [0, n], [0, n], window, hd ** -0.5, kind)
    assert_close(got, want, tol)
    for _ in range(3):
        assert np.array_equal(bits(msm.prompt_attention(q, k, v, ints([0, n]), window=window)), bits(got))


def test_prompt_scales_and_large_scores():
    _, msm = _mods()
    st = [0, 200, 333]
    for scale, std in ((1.0, 1.0), (-0.2, 1.0), (0.0, 1.0), (0.125, 8.0)):
        q, k, v = (randn("bf16", 333, 2, 64, seed=i, std=std if i == 0 else 1.0).cuda() for i in range(3))
        want, tol = prompt_want(q, k, v, st, st, 0, scale, "bf16")
        assert_close(msm.prompt_attention(q, k, v, ints(st), scale=scale), want, tol, "scale %g" % scale)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("place", ["last", "first", "middle"])
def test_many_small_weights_beside_a_large_one(kind, hd, place):
    """Keys of 2^-25.6 of the largest weight each, which together move the result; the largest one
    in the tile that is worked on first, last, or between."""
    _, msm = _mods()
    n, nq = 12000, 200
    at = dict(last=n - nq, first=3, middle=6000)[place]
    q, k, v = (randn(kind, m, h, hd, seed=h, std=0.0) for m, h in ((nq, 2), (n, 1), (n, 1)))
    q[:, :, 0] = 1
    k[:, :, 0] = -17.75
    k[at, :, 0] = 0
    v[:] = 1
    v[at] = 0
    got = msm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), ints([0, nq]), ints([0, n]), scale=1.0)
    # (fp16 weights are at least 2^3 where a score equals the maximum that a row works with)
    want, tol = attend_matrix(f64(q), f64(k), f64(v), n - nq, 0, 1.0, kind, 1, 2.0 ** -28)
    assert (want > 2e-4).all() and (tol < 0.25 * want).all()
    assert_close(got, want, tol)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("hd", [64, 128])
def test_growing_scores(kind, hd):
    """Maxima that grow from key tile to key tile, by less and by more than a row lets them grow."""
    _, msm = _mods()
    n = 900
    rng = np.random.default_rng(hd)
    q, k, v = (randn(kind, n, h, hd, seed=h) for h in (2, 1, 1))
    q[:, :, 0] = 1
    for steps in (3.0, 4.0, 8.0, 13.0):   # in powers of two, per tile from the last key to the first
        k[:, 0, 1:] *= 0.1
        k[:, 0, 0] = _dtype_tensor(kind, (n - np.arange(n)) / 128 * steps * np.log(2) + rng.standard_normal(n))
        got = msm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), ints([0, n]), scale=1.0)
        want, tol = attend_matrix(f64(q), f64(k), f64(v), 0, 0, 1.0, kind, 1, 2.0 ** -28)
        assert_close(got, want, tol, "%g" % steps)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("scale", [2.0 ** -123, -2.0 ** -123, 2.0 ** -124, 2.0 ** -140, 0.0])
def test_the_smallest_scales(hd, scale):
    """Scores near the largest 32-bit number, and a scale that makes ordinary ones of them."""
    _, msm = _mods()
    st = [0, 200, 333]
    q, k, v = (randn("bf16", 333, 2, hd, seed=i, std=2.0 ** 60 if i < 2 else 1.0) for i in range(3))
    got = msm.prompt_attention(q.cuda(), k.cuda(), v.cuda(), ints(st), scale=scale)
    want, tol = prompt_want(q, k, v, st, st, 0, scale, "bf16")
    assert_close(got, want, tol)
    c, rk, rv = filled(np.random.default_rng(24), "bf16", [200, 1, 33], 16, 2, hd)
    c.k_pages[0] *= 2.0 ** 60
    rk = [t * 2.0 ** 60 for t in rk]
    got = c.attention(0, q[:3].cuda(), scale=scale)
    want, tol = decode_want(q[:3], rk, rv, 0, scale, "bf16")
    assert_close(got, want, tol)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
def test_keys_that_a_query_does_not_see_have_no_part(hd, bad):
    """One row of K or V is not finite: the queries that see it follow the formula, every
    other one is as if the row were not there."""
    torch, msm = _mods()
    n, window = 400, 150
    st = [0, n, n + 30]
    for which in (1, 2):
        for row in (0, 131, 255, 399):
            x = [randn("bf16", n + 30, 2, hd, seed=i).cuda() for i in range(3)]
            clean = [t.clone() for t in x]
            x[which][row, 0, 5:9] = float(bad)
            for w in (0, window):
                got = msm.prompt_attention(*x, ints(st), window=w).cpu().double()
                want, tol = prompt_want(*clean, st, st, w, hd ** -0.5, "bf16")
                seen = torch.zeros(n + 30, 2, dtype=torch.bool)
                seen[row:(min(n, row + w) if w else n), 0] = True
                free = ~seen
                assert torch.isfinite(got[free]).all()
                assert (np.abs(got.numpy() - want)[free.numpy()] <= tol[free.numpy()]).all()
                if which == 2:  # V: those columns take the value, the others are untouched
                    hit = got[seen][:, 5:9]
                    assert torch.isnan(hit).all() if bad == "nan" else (hit == float(bad)).all()
                    rest = [c for c in range(hd) if c < 5 or c >= 9]
                    s = seen.numpy()
                    assert (np.abs(got.numpy()[s][:, rest] - want[s][:, rest]) <= tol[s][:, rest]).all()
                elif bad == "nan":
                    assert torch.isnan(got[seen]).all()


@pytest.mark.parametrize("window", [0, 300])
def test_values_that_are_not_finite_in_longer_prompts(window):
    """NaN rows of V and K throughout three packed prompts whose work the blocks share: only the
    queries that see one are touched."""
    torch, msm = _mods()
    lens = [1400, 700, 33]
    st = starts_of(lens)
    x = [randn("bf16", st[-1], h, 64, seed=i).cuda() for i, h in enumerate((8, 2, 2))]
    clean = [t.clone() for t in x]
    rows = [(1, 900), (2, 5), (2, 1399), (1, 1400), (2, 1700), (2, st[-1] - 1)]
    seen = np.zeros(st[-1], bool)
    for which, r in rows:
        x[which][r, :, 7] = float("nan")
        end = next(e for e in st if e > r)
        seen[r:min(end, r + window) if window else end] = True
    got = f64(msm.prompt_attention(*x, ints(st), window=window))
    base = f64(msm.prompt_attention(*clean, ints(st), window=window))
    assert np.array_equal(got[~seen], base[~seen])
    assert np.isnan(got[seen][:, :, 7]).all()


@pytest.mark.parametrize("n_seqs,most", [(700, 3), (150, 40)])
def test_many_short_prompts(n_seqs, most):
    _, msm = _mods()
    rng = np.random.default_rng(n_seqs)
    st = starts_of(rng.integers(0, most + 1, n_seqs))
    q, k, v = (randn("fp16", st[-1], h, 64, seed=h).cuda() for h in (4, 2, 2))
    want, tol = prompt_want(q, k, v, st, st, 0, 0.125, "fp16")
    assert_close(msm.prompt_attention(q, k, v, ints(st)), want, tol)


@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("window", [0, 100, 5000])
def test_work_of_many_resumed_prompts(window, group):
    """Prompts of unlike lengths and cached rows, keys missing in some, more than one look at the
    list of sequences takes in, one look with a single prompt: every row is worked on once."""
    torch, msm = _mods()
    rng = np.random.default_rng(window + group)
    ql = np.concatenate([rng.integers(0, 600, 32), [0] * 7, [333], [0] * 24, rng.integers(0, 90, 9)])
    kl = np.maximum(0, ql + rng.integers(-40, 700, len(ql)) * rng.integers(0, 2, len(ql)))
    qs, ks = starts_of(ql), starts_of(kl)
    q = randn("bf16", qs[-1], group, 64, seed=1).cuda()
    k, v = (randn("bf16", ks[-1], 1, 64, seed=i).cuda() for i in (2, 3))
    out = torch.full_like(q, float("nan"))
    msm.prompt_attention(q, k, v, ints(qs), ints(ks), window=window, out=out)
    want, tol = prompt_want(q, k, v, qs, ks, window, 0.125, "bf16")
    assert_close(out, want, tol)


@pytest.mark.parametrize("kind,hd", [("bf16", 128), ("fp16", 128), ("bf16", 64)])
@pytest.mark.parametrize("window", [0, 300])
def test_blocks_with_several_pieces_of_work(kind, hd, window):
    """Far more pieces of work than blocks, pieces of two tiles (more than 128 rows) and of one by
    turns, both with several key tiles: what a block's pieces hand on to one another (the ring's
    last values, Q, the results in tensor memory) has to be through when the next one takes it."""
    torch, msm = _mods()
    rng = np.random.default_rng(hd + window)
    hkv, group = 8, 4
    # a block takes 64 tokens: every other prompt's last piece has at most 32
    ql = [int(64 * rng.integers(0, 3) + rng.integers(1, 33) + (32 if i % 2 else 0)) for i in range(40)]
    kl = [n + int(rng.integers(0, 500)) for n in ql]
    qs, ks = starts_of(ql), starts_of(kl)
    q = randn(kind, qs[-1], hkv * group, hd, seed=1).cuda()
    k, v = (randn(kind, ks[-1], hkv, hd, seed=i).cuda() for i in (2, 3))
    pieces = hkv * sum(-(-n // 64) for n in ql)
    assert pieces > 3 * torch.cuda.get_device_properties(0).multi_processor_count
    out = torch.full_like(q, float("nan"))
    msm.prompt_attention(q, k, v, ints(qs), ints(ks), window=window, out=out)
    for s in range(len(ql)):
        a, b = slice(qs[s], qs[s + 1]), slice(ks[s], ks[s + 1])
        want, tol = attend_matrix(f64(q[a]), f64(k[b]), f64(v[b]), kl[s] - ql[s], window, hd ** -0.5, kind)
        assert_close(out[a], want, tol, "sequence %d" % s)
    for _ in range(20):
        assert np.array_equal(bits(msm.prompt_attention(q, k, v, ints(qs), ints(ks), window=window)), bits(out))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("window", [0, 50])
def test_a_batch_of_caches_with_rows_to_spare(hd, window):
    """Contiguous caches side by side, filled in part (NaN behind), each with a turn that continues it: the
    spare rows as sequences without queries."""
    torch, msm = _mods()
    room, have, new = 300, [120, 300, 0, 7, 299], [33, 5, 0, 7, 130]
    k, v = (randn("bf16", 2, room * len(have), hd, seed=i).cuda() for i in (1, 2))
    qs, ks, at = [0], [0], 0
    for s, (h, n) in enumerate(zip(have, new)):
        at += n
        qs += [at, at]
        ks += [room * s + h, room * (s + 1)]
        k[:, room * s + h:room * (s + 1)] = float("nan")
        v[:, room * s + h:room * (s + 1)] = float("nan")
    k, v = k.transpose(0, 1), v.transpose(0, 1)
    q = randn("bf16", at, 8, hd, seed=3).cuda()
    got = msm.prompt_attention(q, k, v, ints(qs), ints(ks), window=window)
    for s, (h, n) in enumerate(zip(have, new)):
        a, b = slice(qs[2 * s], qs[2 * s] + n), slice(room * s, room * s + h)
        want, tol = attend_matrix(f64(q[a]), f64(k[b]), f64(v[b]), h - n, window, hd ** -0.5, "bf16")
        assert_close(got[a], want, tol, "cache %d" % s)


def test_prompts_on_two_streams_at_once():
    torch, msm = _mods()
    n = 3000
    x = [[randn("bf16", n, h, 128, seed=s + h).cuda() for h in (8, 2, 2)] for s in range(2)]
    x = [[q, k, v] for q, k, v in x]
    st = ints([0, n])
    want = [bits(msm.prompt_attention(*y, st)) for y in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(msm.prompt_attention(*x[i], st))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert np.array_equal(bits(o), want[i])


def test_a_wait_that_runs_out_is_reported():
    """Through the test hook that leaves the loads out (2 s): the launch ends, its rows are NaN, the
    status says why, and the calls behind it are what they were."""
    torch, msm = _mods()
    x = [randn("bf16", 400, 4, 64, seed=i).cuda() for i in range(3)]
    st, status = ints([0, 300, 400]), ints([0])
    want = bits(msm.prompt_attention(*x, st, status=status))
    assert status.item() == 0
    out = torch.zeros_like(x[0])
    p = msm.MsmPrompt(0, msm.MSM_BF16, 2, 400, 400, 4, 4, 64, 0, 0.125, *(t.data_ptr() for t in x), out.data_ptr(),
                      *([256, 64] * 4), st.data_ptr(), st.data_ptr(), status.data_ptr(), msm.MSM_FLAG_TEST_DROP_HANDOFF)
    assert msm.msm_prompt_attention(p, torch.cuda.current_stream().cuda_stream) == msm.MSM_OK
    torch.cuda.synchronize()
    assert torch.isnan(out).all() and status.item() == msm.MSM_ERR_DEVICE_TIMEOUT
    status.zero_()
    for _ in range(3):
        assert np.array_equal(bits(msm.prompt_attention(*x, st, status=status)), want)
    assert status.item() == 0
    p.status = None
    p.flags = 0
    assert msm.msm_prompt_attention(p, torch.cuda.current_stream().cuda_stream) == msm.MSM_OK
    assert np.array_equal(bits(out), want)
    with pytest.raises(ValueError, match="status"):
        msm.prompt_attention(*x, st, status=status.cpu())


def test_prompt_leaves_what_is_not_its_own():
    torch, msm = _mods()
    x = [randn("bf16", 100, 4, 64, seed=i).cuda() for i in range(3)]
    big = torch.full((120, 2, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out = big[10:110, 1]
    st = [0, 20, 81]
    assert msm.prompt_attention(*x, ints(st), out=out) is out
    want, tol = prompt_want(*x, st, st, 0, 0.125, "bf16")
    assert_close(out[:81], want[:81], tol[:81])
    out[:81] = 3.0
    assert (big == 3.0).all()


def test_rows_more_than_2_to_the_32_elements_apart():
    torch, msm = _mods()
    n, stride = 70, 1 << 26
    big = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda")  # 9.4 GB
    views = [big.as_strided((n, 2, 64), (stride, 64, 1), i * 4096) for i in range(4)]
    for i in range(3):
        views[i].copy_(randn("bf16", n, 2, 64, seed=i))
    got = msm.prompt_attention(*views[:3], ints([0, 30, n]), out=views[3])
    want, tol = prompt_want(*views[:3], [0, 30, n], [0, 30, n], 0, 0.125, "bf16")
    assert_close(got, want, tol)


def test_starts_out_of_range_are_cut_off():
    torch, msm = _mods()
    x = [randn("bf16", 50, 2, 64, seed=i).cuda() for i in range(3)]
    for st in ([0, 50, 1 << 30], [-5, 50, 50], [0, 50, 20]):
        got = msm.prompt_attention(*x, ints(st))
        want, tol = prompt_want(*x, [0, 50], [0, 50], 0, 0.125, "bf16")
        assert_close(got, want, tol, str(st))


def test_empty_prompts():
    torch, msm = _mods()
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert msm.prompt_attention(e, e, e, ints([0, 0])).shape == (0, 2, 64)
    q = randn("bf16", 3, 2, 64).cuda()
    assert (msm.prompt_attention(q, e, e, ints([0, 3]), ints([0, 0])) == 0).all()


# ------------------------------------------------------------------ together
def test_a_prompt_a_search_and_single_tokens():
    """Two prompts through the prompt attention into pages, one of them forked, every branch
    continued token by token, the others freed, the pool compacted: at each step the paged
    attention equals the formula over the rows that the sequence was given."""
    torch, msm = _mods()
    rng = np.random.default_rng(20)
    hq, hkv, hd, slots = 8, 2, 64, 5
    cache = msm.PagedCache.allocate(2, 40, 16, hkv, hd, slots, 12, dtype=torch.bfloat16)
    hist = [[torch.empty((0, hkv, hd), dtype=torch.bfloat16)] * 2 for _ in range(slots)]  # per sequence: K, V
    prompts = [70, 33, 0, 0, 0]
    st = starts_of(prompts)
    x = randn("bf16", st[-1], hq + 2 * hkv, hd, seed=1).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    cache.resize(ints(prompts))
    cache.write(1, k, v, ints(st))
    got = msm.prompt_attention(q, k, v, ints(st))
    want, tol = prompt_want(q, k, v, st, st, 0, hd ** -0.5, "bf16")
    assert_close(got, want, tol)
    for s in range(slots):
        hist[s] = [k[st[s]:st[s + 1]].cpu(), v[st[s]:st[s + 1]].cpu()]
    cache.fork(ints([-1, -1, 0, 0, 1]))
    for s, p in ((2, 0), (3, 0), (4, 1)):
        hist[s] = list(hist[p])
    active = list(range(slots))
    for step in range(8):
        n = [hist[s][0].shape[0] + 1 if s in active else 0 for s in range(slots)]
        cache.resize(ints(n))
        cnt = starts_of([int(s in active) for s in range(slots)])
        y = randn("bf16", cnt[-1], 2 * hkv, hd, seed=50 + step).cuda()
        cache.write(1, y[:, :hkv], y[:, hkv:], ints(cnt))
        for i, s in enumerate(active):
            hist[s] = [torch.cat([hist[s][0], y[i:i + 1, :hkv].cpu()]), torch.cat([hist[s][1], y[i:i + 1, hkv:].cpu()])]
        qq = randn("bf16", slots, hq, hd, seed=70 + step).cuda()
        got = cache.attention(1, qq)
        cache.sync()
        for s in range(slots):
            if s in active:
                nk = hist[s][0].shape[0]
                want, tol = attend(f64(qq[s:s + 1]), f64(hist[s][0]), f64(hist[s][1]), nk - 1, 0, hd ** -0.5, "bf16")
                assert_close(got[s:s + 1], want, tol, "step %d sequence %d" % (step, s))
            else:
                assert (got[s] == 0).all()
        if step == 3:
            active = [0, 3, 4]
        if step == 5:
            cache.resize(ints([-1 if s in active else 0 for s in range(slots)]))
            cache.compact()
            used = int((cache.refs > 0).sum())
            assert (cache.refs[:used] > 0).all()


def test_pages_are_caches_of_the_verify_step():
    """With page_rows = max_ctx a page is what msm_verify_step takes: histories that
    msm_pages_write stored give the step's results bit for bit, and its new rows are in the
    sequence's page."""
    torch, msm = _mods()
    import synth
    from gpu_cases import make_case
    case = make_case("cfg1_stack")
    cfg, dev = case.cfg, torch.device("cuda", 0)
    model = msm.Model(cfg, [synth.to_torch(w, dev) for w in case.layers], synth.to_torch(case.final, dev), device=0)
    try:
        hid = torch.from_numpy(case.hidden.view(np.int16)).to(dev)

        def step(kc, vc):
            logits = torch.empty((16, cfg.vocab), dtype=torch.float32, device=dev)
            model.verify_step(hid, case.parent, case.pos0, kc, vc, logits_out=logits)
            assert model.sync() == msm.MSM_OK
            return logits
        as_bf16 = lambda a: torch.from_numpy(a.view(np.int16)).to(dev).view(torch.bfloat16)
        kc, vc = [as_bf16(k) for k, _ in case.kv], [as_bf16(v) for _, v in case.kv]
        cache = msm.PagedCache.allocate(cfg.n_layers, 3, cfg.max_ctx, cfg.hkv, cfg.hd, 2, 1)
        cache.resize(ints([5, case.pos0]))
        for l in range(cfg.n_layers):
            cache.write(l, kc[l][:, :case.pos0].transpose(0, 1), vc[l][:, :case.pos0].transpose(0, 1),
                        ints([0, 0, case.pos0]))
        cache.resize(ints([-1, case.pos0 + 16]))
        cache.sync()
        page = int(cache.table[1, 0])
        got = step([t[page] for t in cache.k_pages], [t[page] for t in cache.v_pages])
        want = step(kc, vc)
        assert torch.equal(got, want)
        for l in range(cfg.n_layers):
            rows = slice(0, case.pos0 + 16)
            assert np.array_equal(bits(cache.k_pages[l][page][:, rows]), bits(kc[l][:, rows]))
            assert np.array_equal(bits(cache.v_pages[l][page][:, rows]), bits(vc[l][:, rows]))
    finally:
        model.close()


def test_captured_and_replayed_with_other_lengths():
    torch, msm = _mods()
    rng = np.random.default_rng(21)
    c, rk, rv = filled(rng, "bf16", [60, 200, 33], 16, 2, 64, extra=20, max_pages=16)
    q = randn("bf16", 3, 4, 64, seed=5).cuda()
    new = ints([61, 201, 34])
    st = ints([0, 1, 2, 3])
    kv = randn("bf16", 3, 4, 64, seed=6).cuda()
    c.attention(0, q)
    c.table[c.table < 0] = -1
    saved = [t.clone() for t in (c.table, c.lens, c.refs)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.resize(new)
        c.write(0, kv[:, :2], kv[:, 2:], st)
        out = c.attention(0, q)
        p_out = msm.prompt_attention(kv, kv[:, :2], kv[:, 2:], st)
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other, stream=side):
        out2 = c.attention(0, q, window=20)
    for lens in ([61, 201, 34], [100, 0, 250], [0, 17, 16]):
        for t, x in zip((c.table, c.lens, c.refs), saved):
            t.copy_(x)
        # rows that a sequence gains beyond those it had are whatever its pages held: zeros
        c.k_pages[0].nan_to_num_(0.0)
        c.v_pages[0].nan_to_num_(0.0)
        new.copy_(ints(lens))
        st.copy_(ints(starts_of([int(n > 0) for n in lens])))
        g.replay()
        other.replay()
        c.sync()
        ref_k, ref_v = [], []
        table, kp, vp = c.table.cpu().numpy(), c.k_pages[0].cpu(), c.v_pages[0].cpu()
        for s, n in enumerate(lens):
            ids = [int(table[s, r // 16]) for r in range(n)]
            ref_k.append(torch.stack([kp[p, :, r % 16] for r, p in enumerate(ids)]) if n else kp[0, :, :0].transpose(0, 1))
            ref_v.append(torch.stack([vp[p, :, r % 16] for r, p in enumerate(ids)]) if n else vp[0, :, :0].transpose(0, 1))
        want, tol = decode_want(q, ref_k, ref_v, 0, 0.125, "bf16")
        assert_close(out, want, tol, str(lens))
        want, tol = decode_want(q, ref_k, ref_v, 20, 0.125, "bf16")
        assert_close(out2, want, tol, str(lens))
        n = sum(int(x > 0) for x in lens)
        assert np.array_equal(f64(p_out[:n]), f64(kv[:n, [2, 2, 3, 3]]))  # one key each: its v


def test_two_streams_at_once():
    """Attention calls of one cache on two streams, each with its own workspace."""
    torch, msm = _mods()
    rng = np.random.default_rng(22)
    c, rk, rv = filled(rng, "bf16", [9000, 500, 3000], 64, 2, 128)
    qs = [randn("bf16", 3, 8, 128, seed=i).cuda() for i in range(2)]
    want = [bits(c.attention(0, q)) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(c.attention(0, qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert np.array_equal(bits(o), want[i])
