"""The cache in 8 bits, attention with sinks and sampling on the GPU, against the 64-bit references in
stream_reference.py."""
import numpy as np
import pytest

from stream_reference import VALUES, QPages, attend_seen, draw, seen
from test_gpu_paged import _dtype, _mods, assert_close, bits, f64, ints, randn, starts_of

pytestmark = pytest.mark.gpu
NAN = float("nan")
INF = float("inf")


def codes(t):
    torch, _ = _mods()
    return t.view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------ the cache in 8 bits
class Both:
    """A cache in 8 bits on the GPU and its reference, called alike and compared after every call."""

    def __init__(self, rng, layers, n_pages, rows, block, heads, hd, n_seqs, max_pages, kind="bf16"):
        torch, msm = _mods()
        self.kind, self.layers = kind, layers
        shape, blocks = (n_pages, heads, rows, hd), -(-rows // block)
        pools = [rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2 * layers)]
        scales = [(2.0 ** rng.integers(-6, 3, (n_pages, heads, blocks))).astype(np.float32) for _ in pools]
        gpu = [torch.from_numpy(p).cuda().view(torch.float8_e4m3fn) for p in pools]
        sc = [torch.from_numpy(s).cuda() for s in scales]
        self.gpu = msm.PagedCache(gpu[:layers], gpu[layers:], ints([[-1] * max_pages] * n_seqs), ints([0] * n_seqs),
                                  ints([0] * n_pages), k_scales=sc[:layers], v_scales=sc[layers:], block_rows=block)
        self.ref = QPages(n_pages, rows, n_seqs, max_pages, [p.copy() for p in pools], block_rows=block,
                          scales=[s.astype(np.float64) for s in scales])

    def same(self):
        g, r = self.gpu, self.ref
        assert np.array_equal(g.table.cpu().numpy(), r.table)
        assert np.array_equal(g.lens.cpu().numpy(), r.lens)
        assert np.array_equal(g.refs.cpu().numpy(), r.refs)
        for a, b in zip(g.k_scales + g.v_scales, r.scales):
            assert np.array_equal(f64(a), b)
        for a, b in zip(g.k_pages + g.v_pages, r.pools):
            a = codes(a)
            nan = (a & 127 == 127) & (b & 127 == 127)  # (a NaN's sign says nothing)
            assert np.array_equal(np.where(nan, 0, a), np.where(nan, 0, b))

    def call(self, name, arg=None):
        torch, msm = _mods()
        args = () if arg is None else (ints(arg),)
        getattr(self.gpu, name)(*args)
        err = getattr(self.ref, name)(*(() if arg is None else (arg,)))
        if err is None:
            self.gpu.sync()
        else:
            with pytest.raises(msm.MsmError, match="msm_qpages_" + name) as e:
                self.gpu.sync()
            assert msm.STATUS_NAMES[e.value.code] == err
        self.same()
        return err

    def write(self, counts, seed, sizes=1.0, change=None):
        torch, _ = _mods()
        st = starts_of(counts)
        heads, hd = self.gpu.k_pages[0].shape[1], self.gpu.k_pages[0].shape[3]
        for layer in range(self.layers):
            # both out of one packed tensor, and a row behind the last sequence
            kv = randn(self.kind, st[-1] + 1, 2 * heads, hd, seed=seed + layer)
            kv = (kv.float() * sizes).to(kv.dtype)
            if change:
                change(kv)
            kv = kv.cuda()
            self.gpu.write(layer, kv[:, :heads], kv[:, heads:], ints(st))
            rows = f64(kv)
            self.ref.write(layer, rows[:, :heads], st)
            self.ref.write(self.layers + layer, rows[:, heads:], st)
        self.gpu.sync()
        self.same()


@pytest.mark.parametrize("rows,block,heads,hd,kind", [
    (16, 16, 2, 64, "bf16"), (1, 1, 1, 128, "fp16"), (7, 3, 3, 64, "fp16"), (64, 16, 4, 128, "bf16"),
    (33, 32, 1, 64, "bf16"), (40, 17, 2, 128, "fp16"), (64, 64, 1, 128, "bf16"), (70, 70, 2, 64, "bf16")])
def test_random_calls_equal_the_reference(rows, block, heads, hd, kind):
    """Writes of prompts and of single tokens, of sizes that make scales grow and stay."""
    rng = np.random.default_rng(rows * 100 + block)
    n_seqs, max_pages = 9, 6
    c = Both(rng, 2, 40, rows, block, heads, hd, n_seqs, max_pages, kind)
    for step in range(14):
        old = c.ref.lens.copy()
        if step % 3 == 1:  # a few more for everybody
            new = [min(int(n) + int(rng.integers(0, 4)), max_pages * rows) for n in old]
        else:
            new = [-1 if rng.random() < 0.3 else int(rng.integers(0, max_pages * rows + 1)) for _ in range(n_seqs)]
        if c.call("resize", new) is None:
            c.write(np.maximum(c.ref.lens - old, 0), 100 * step, sizes=float(2.0 ** rng.uniform(-4, 5)))
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


@pytest.mark.parametrize("rows,block,hd,n_seqs", [(300, 300, 128, 3), (200, 190, 64, 3), (130, 128, 128, 2), (16, 5, 64, 70),
                                                  (8, 8, 128, 31), (8, 3, 128, 32), (40, 40, 64, 33)])
def test_long_blocks_and_many_sequences(rows, block, hd, n_seqs):
    """Blocks of more rows than registers hold; searches of one step and of more."""
    rng = np.random.default_rng(rows + n_seqs)
    c = Both(rng, 1, 4 * n_seqs, rows, block, 2, hd, n_seqs, 3)
    for step in range(5):
        old = c.ref.lens.copy()
        grow = rng.integers(0, [3 * rows, 3, rows, 2, 40][step] + 1, n_seqs)
        assert c.call("resize", [int(min(n + g, 3 * rows)) for n, g in zip(old, grow)]) is None
        c.write(c.ref.lens - old, step, sizes=float(2.0 ** rng.uniform(-3, 4)))
        if step == 1:
            c.call("resize", [int(n) // 2 if s % 2 else -1 for s, n in enumerate(c.ref.lens)])
    c.ref.check()


@pytest.mark.parametrize("block", [5, 64, 200])
def test_one_token_at_a_time_through_growing_sizes(block):
    c = Both(np.random.default_rng(7), 1, 6, 200, block, 2, 64, 2, 3)
    for i in range(23):
        c.call("resize", [i + 1, 2 * i + 2])
        c.write([1, 2], i, sizes=float(1.3 ** i))


@pytest.mark.parametrize("kind,sizes", [("bf16", 2.0 ** -130), ("bf16", 2.0 ** 120), ("fp16", 2.0 ** -20),
                                        ("fp16", 2.0 ** 13), ("bf16", 0.0)])
def test_the_smallest_and_largest_rows(kind, sizes):
    c = Both(np.random.default_rng(8), 1, 8, 16, 8, 2, 128, 3, 4, kind)
    c.call("resize", [16, 5, 40])
    c.write([16, 5, 40], 1, sizes=sizes)
    c.call("resize", [17, 6, 41])
    c.write([1, 1, 1], 2, sizes=1.0)
    c.call("resize", [18, 7, 42])
    c.write([1, 1, 1], 3, sizes=sizes)


def test_rows_that_are_not_finite():
    def change(kv):
        kv[0, :, 3] = INF
        kv[1, :, 5] = -INF
        kv[2, 0] = NAN
        kv[9] = INF
        kv[10:18] = NAN
    c = Both(np.random.default_rng(9), 1, 8, 16, 8, 2, 64, 2, 4)
    c.call("resize", [20, 9])
    c.write([20, 9], 1, change=change)
    c.call("resize", [21, 10])
    c.write([1, 1], 2, sizes=50.0)


def test_tokens_without_a_row_are_left_out():
    torch, msm = _mods()
    c = Both(np.random.default_rng(10), 1, 6, 8, 4, 1, 64, 3, 2)
    c.call("resize", [8, 5, 3])
    c.call("resize", [3, 5, 0])
    kv = randn("bf16", 20, 1, 64, seed=1).cuda()
    before = [codes(t).copy() for t in c.gpu.k_pages], c.gpu.lens.clone()
    # sequence 0: two tokens more than rows; 1: fine; 2: none of its tokens has a row
    st = [0, 5, 7, 9]
    c.gpu.write(0, kv, kv, ints(st))
    with pytest.raises(msm.MsmError, match="msm_qpages_write") as e:
        c.gpu.sync()
    assert e.value.code == msm.MSM_ERR_INVALID_ARG
    rows = f64(kv)
    for i in (0, 1):
        c.ref.lens[2] = 0
        c.ref.write(i, np.concatenate([rows[2:7]]), [0, 3, 5, 5])
    c.same()
    # a shared page takes no rows
    c.call("fork", [-1, -1, 1])
    c.gpu.write(0, kv[:1], kv[:1], ints([0, 0, 1, 1]))
    with pytest.raises(msm.MsmError, match="msm_qpages_write"):
        c.gpu.sync()
    c.same()
    # nothing changes behind a refused resize
    c.gpu.resize(ints([99, 0, 0]))
    c.gpu.write(0, kv[:1], kv[:1], ints([0, 1, 1, 1]))
    c.gpu.compact()
    with pytest.raises(msm.MsmError, match="msm_qpages_resize"):
        c.gpu.sync()
    c.same()


def test_starts_that_make_no_sense_stay_in_bounds():
    torch, msm = _mods()
    c = Both(np.random.default_rng(11), 1, 6, 8, 4, 1, 64, 3, 2)
    c.call("resize", [8, 5, 3])
    kv = randn("bf16", 6, 1, 64, seed=1).cuda()
    for st in ([5, 0, 3, 6], [0, 100, 100, 100], [-5, -3, 2, 6], [0, 6, 2, 4], [3, 3, 3, -1]):
        c.gpu.write(0, kv, kv, ints(st))
        torch.cuda.synchronize()
        try:
            c.gpu.sync()
        except msm.MsmError as e:
            assert e.code == msm.MSM_ERR_INVALID_ARG


def test_more_layers_than_one_copy_launch_carries():
    c = Both(np.random.default_rng(5), 70, 9, 4, 3, 1, 64, 3, 3)
    c.call("resize", [6, 5, 0])
    c.call("fork", [-1, -1, 0])
    c.call("resize", [7, 0, 8])
    c.call("compact")
    c.ref.check()


# ------------------------------------------------------------------ decoding
def decode_case(kind, hq, hkv, hd, rows, lens, block=None, seed=0, q_std=1.0, spread=3):
    """A filled cache (16 bits, or 8 with a block), q, and the sequences' K and V as 64-bit rows."""
    torch, msm = _mods()
    rng = np.random.default_rng(seed)
    n_pages = sum(-(-n // rows) for n in lens) + 2
    order = rng.permutation(n_pages)
    table, refs, at = np.full((len(lens), max(1, max(-(-n // rows) for n in lens))), -1), np.zeros(n_pages), 0
    for s, n in enumerate(lens):
        m = -(-n // rows)
        table[s, :m] = order[at:at + m]
        at += m
    refs[order[:at]] = 1
    shape, more, scales = (n_pages, hkv, rows, hd), {}, [None, None]
    if block:
        held = [rng.normal(size=shape) * 40 for _ in range(2)]
        pools = [torch.from_numpy(x).to(torch.float8_e4m3fn).cuda() for x in held]
        scales = [2.0 ** rng.integers(-5 - spread, -4, (n_pages, hkv, -(-rows // block))) for _ in range(2)]
        more = dict(k_scales=[torch.from_numpy(scales[0]).float().cuda()],
                    v_scales=[torch.from_numpy(scales[1]).float().cuda()], block_rows=block)
    else:
        pools = [randn(kind, *shape, seed=seed + 1 + i).cuda() for i in range(2)]
    cache = msm.PagedCache(pools[:1], pools[1:], ints(table.tolist()), ints(lens), ints(refs.astype(int).tolist()), **more)
    q = randn(kind, len(lens), hq, hd, seed=seed + 9, std=q_std).cuda()
    return cache, q, table


def rows_of(cache, table, s, n, rows, which):
    """[n][heads][hd] of sequence s, and the scales of its rows."""
    pool = f64((cache.k_pages, cache.v_pages)[which][0].float())
    r = np.arange(n)
    x = pool[table[s, r // rows], :, r % rows] if n else pool[:0, :, 0]
    if not getattr(cache, "k_scales", None):
        return x, None
    sc = f64((cache.k_scales, cache.v_scales)[which][0])
    f = sc[table[s, r // rows], :, r % rows // cache.block_rows] if n else sc[:0, :, 0]
    return x * f[..., None], f


def check_decode(cache, q, table, lens, rows, kind, window, sinks, got, scale=None):
    hd = q.shape[2]
    for s, n in enumerate(lens):
        k, _ = rows_of(cache, table, s, n, rows, 0)
        v, f = rows_of(cache, table, s, n, rows, 1)
        see = seen(1, n, window, sinks)
        # a weight is two 16-bit terms: off by at most 3 u^2 of itself (8 bits: fp16's u) and, in fp16, by
        # 2^-39 of the largest; the products' scores are also scaled in 32 bits (far inside 2 hd 2^-23 B)
        u = 2.0 ** -11 if f is not None or kind == "fp16" else 2.0 ** -8
        least = 2.0 ** -39 if f is not None or kind == "fp16" else 0.0
        want, tol = attend_seen(f64(q)[s:s + 1], k, v, see, scale or hd ** -0.5, kind, weight=3 * u * u, least=least, big=f)
        assert_close(got[s:s + 1], want, tol, "sequence %d of %d rows" % (s, n))


LAYOUTS = [("bf16", 8, 2, 64, 16), ("fp16", 8, 8, 128, 7), ("bf16", 16, 2, 128, 64), ("fp16", 4, 2, 64, 33),
           ("bf16", 3, 3, 128, 1)]


@pytest.mark.parametrize("window,sinks", [(1, 1), (5, 3), (64, 4), (100, 64), (33, 65), (128, 130), (500, 100), (7, 10 ** 9),
                                          (2 ** 31, 4), (10, 0)])
@pytest.mark.parametrize("kind,hq,hkv,hd,rows", LAYOUTS)
def test_decode_with_sinks(kind, hq, hkv, hd, rows, window, sinks):
    lens = [0, 1, 2, 7, 64, 65, 129, 300, 1000, 1]
    cache, q, table = decode_case(kind, hq, hkv, hd, rows, lens, seed=rows)
    got = cache.attention(0, q, window=window, sinks=sinks)
    cache.sync()
    check_decode(cache, q, table, lens, rows, kind, window, sinks, got)
    if sinks == 0:
        assert np.array_equal(bits(got), bits(cache.attention(0, q, window=window)))


def test_rows_between_the_sinks_and_the_window_are_not_read():
    """Their pages may be gone, and what they hold is of no interest."""
    torch, msm = _mods()
    lens, rows, window, sinks = [700, 40, 500], 16, 100, 20
    for block in (None, 8):
        cache, q, table = decode_case("bf16", 8, 2, 128, rows, lens, block=block, seed=3)
        want = cache.attention(0, q, window=window, sinks=sinks).clone()
        for s, n in enumerate(lens):
            for r in range(sinks, n - window):
                p = int(table[s, r // rows])
                cache.k_pages[0].view(torch.uint8)[p, :, r % rows] = 0x7F
                cache.v_pages[0].view(torch.uint8)[p, :, r % rows] = 0x7F
            cache.table[s, -(-sinks // rows):(max(0, n - window)) // rows] = 10 ** 6
        got = cache.attention(0, q, window=window, sinks=sinks)
        cache.sync()
        assert np.array_equal(bits(got), bits(want))


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 5), (1, 0), (64, 4), (100, 70), (33, 200)])
@pytest.mark.parametrize("kind,hq,hkv,hd,rows,block", [
    ("bf16", 8, 2, 64, 16, 16), ("fp16", 8, 8, 128, 7, 3), ("bf16", 16, 2, 128, 64, 16), ("fp16", 4, 2, 64, 33, 32),
    ("bf16", 3, 3, 128, 1, 1), ("fp16", 8, 1, 64, 256, 100), ("bf16", 2, 1, 128, 40, 40)])
def test_decode_over_8_bits(kind, hq, hkv, hd, rows, block, window, sinks):
    lens = [0, 1, 2, 7, 64, 65, 129, 300, 1000, 1, 33]
    cache, q, table = decode_case(kind, hq, hkv, hd, rows, lens, block=block, seed=rows + block)
    got = cache.attention(0, q, window=window, sinks=sinks)
    cache.sync()
    check_decode(cache, q, table, lens, rows, kind, window, sinks, got)


@pytest.mark.parametrize("block", [None, 4])
def test_many_short_sequences(block):
    """More sequences than a block has threads, most of them of a tile or none."""
    rng = np.random.default_rng(12)
    lens = [int(n) for n in rng.integers(0, 60, 300)] + [900]
    cache, q, table = decode_case("fp16", 4, 2, 64, 8, lens, block=block, seed=12)
    got = cache.attention(0, q, window=40, sinks=2)
    cache.sync()
    check_decode(cache, q, table, lens, 8, "fp16", 40, 2, got)


@pytest.mark.parametrize("kind,hd,window,sinks", [("bf16", 64, 0, 0), ("fp16", 128, 70, 30)])
def test_a_batch_of_more_items_than_blocks(kind, hd, window, sinks):
    """Items of one to three tiles that a warp does alone, between longer ones."""
    rng = np.random.default_rng(13)
    lens = [int(n) for n in rng.integers(0, 230, 640)]
    lens[100], lens[400] = 1500, 700
    cache, q, table = decode_case(kind, 8, 4, hd, 16, lens, block=16, seed=13)
    got = cache.attention(0, q, window=window, sinks=sinks)
    cache.sync()
    check_decode(cache, q, table, lens, 16, kind, window, sinks, got)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_long_and_ragged_batches_over_8_bits(kind):
    """More parts of an item than are joined at once, and scales far apart within a sequence."""
    for lens, spread in (([40000], 0), ([9000, 1, 0, 333, 20000], 20)):
        cache, q, table = decode_case(kind, 8, 2, 128, 64, lens, block=16, seed=4, spread=spread)
        got = cache.attention(0, q)
        cache.sync()
        check_decode(cache, q, table, lens, 64, kind, 0, 0, got)


@pytest.mark.parametrize("kind,std", [("bf16", 2.0 ** 60), ("bf16", 2.0 ** -60), ("fp16", 2.0 ** -12), ("bf16", 2.0 ** -129)])
def test_small_and_large_queries_over_8_bits(kind, std):
    lens = [5, 200]
    cache, q, table = decode_case(kind, 8, 2, 64, 16, lens, block=16, seed=5, q_std=std)
    scale = min(0.1 / std, 2.0 ** 110)
    got = cache.attention(0, q, scale=scale)
    # (q of 2^-129 is below 2^-98: exact to 2^-24 x 2^-112 only, 2^-7 of its size; its scores are below
    # 2^-129 x 2^110 x 64 x 448 x 2^-4, so all weights are equal to 2^-8 and that part moves them by 2^-15)
    check_decode(cache, q, table, lens, 16, kind, 0, 0, got, scale)


def test_special_values_over_8_bits():
    torch, msm = _mods()
    lens = [40, 40, 40, 40, 40, 3]
    cache, q, table = decode_case("bf16", 4, 2, 64, 8, lens, block=4, seed=6)
    k, v, ks, vs = cache.k_pages[0].view(torch.uint8), cache.v_pages[0].view(torch.uint8), cache.k_scales[0], cache.v_scales[0]
    # sequence 0: all of V's blocks 0; 1: one block of K and one of V 0; 2: a NaN key; 3: a NaN value;
    # 4: V's scales over the whole range, down to subnormal ones; 5: V's scales large
    vs[cache.table[0, :5].long()] = 0
    ks[int(table[1, 0])] = 0
    vs[int(table[1, 1]), :, 1] = 0
    k[int(table[2, 3]), 1, 2, 5] = 0x7F
    v[int(table[3, 2]), 0, 1, 7] = 0xFF
    vs[int(table[4, 0])] = 2.0 ** -140
    vs[int(table[4, 1])] = 2.0 ** -126
    vs[int(table[4, 2])] = 3 * 2.0 ** 100
    vs[int(table[4, 3])] = 1.7
    vs[int(table[5, 0])] = 2.0 ** 110
    got = f64(cache.attention(0, q))
    assert (got[0] == 0).all()
    assert np.isnan(got[2, 2:]).all() and not np.isnan(got[2, :2]).any()
    assert np.isnan(got[3, :2, 7]).all() and np.isnan(got[3]).sum() == 2
    for s in (1, 4, 5):
        check_decode(cache, q[s:s + 1], table[s:s + 1], lens[s:s + 1], 8, "bf16", 0, 0, torch.from_numpy(got[s:s + 1]))


def test_strides_and_other_outputs_over_8_bits():
    torch, msm = _mods()
    lens = [3, 100]
    cache, q, table = decode_case("fp16", 4, 2, 64, 16, lens, block=16, seed=7)
    want = cache.attention(0, q)
    wide = torch.zeros(2, 6, 3, 64, dtype=torch.float16, device="cuda")
    wide[:, 1:5, 1] = q
    out = torch.full((2, 9, 64), 7.0, dtype=torch.float16, device="cuda")
    cache.attention(0, wide[:, 1:5, 1], out=out[:, 2:6])
    assert torch.equal(out[:, 2:6], want) and (out[:, :2] == 7).all() and (out[:, 6:] == 7).all()
    both = cache.attention(0, q.bfloat16())  # q and out of either type over the same cache
    assert both.dtype == torch.bfloat16
    with pytest.raises(ValueError):
        cache.attention(0, q.float())
    with pytest.raises(ValueError):
        cache.write(0, q.float()[:, :2], q.float()[:, :2], ints([0, 1, 2]))
    with pytest.raises(ValueError, match="scales"):
        msm.PagedCache(cache.k_pages, cache.v_pages, cache.table, cache.lens, cache.refs)
    with pytest.raises(ValueError, match="scales"):
        msm.PagedCache([wide], [wide], cache.table, cache.lens, cache.refs, k_scales=cache.k_scales,
                       v_scales=cache.v_scales)
    with pytest.raises(ValueError, match="float32"):
        msm.PagedCache(cache.k_pages, cache.v_pages, cache.table, cache.lens, cache.refs, k_scales=cache.k_scales,
                       v_scales=[t[:, :1] for t in cache.v_scales], block_rows=16)


def test_pages_outside_the_pool_over_8_bits():
    torch, msm = _mods()
    lens = [40, 20]
    cache, q, table = decode_case("bf16", 4, 2, 64, 8, lens, block=8, seed=8)
    cache.table[0, 1] = 10 ** 8
    cache.table[1, :3] = -5
    got = cache.attention(0, q, window=30, sinks=3)
    with pytest.raises(msm.MsmError, match="msm_qpages_attention"):
        cache.sync()
    assert (got[1] == 0).all() and not got.isnan().any()


# ------------------------------------------------------------------ prompts with sinks
def prompt_case(kind, hq, hkv, hd, q_lens, k_lens, seed=0):
    q = randn(kind, max(1, sum(q_lens)), hq, hd, seed=seed).cuda()
    k = randn(kind, max(1, sum(k_lens)), hkv, hd, seed=seed + 1).cuda()
    v = randn(kind, max(1, sum(k_lens)), hkv, hd, seed=seed + 2).cuda()
    return q, k, v, starts_of(q_lens), starts_of(k_lens)


def check_prompt(q, k, v, qs, ks, window, sinks, kind, got):
    for s in range(len(qs) - 1):
        a, b, c, d = qs[s], qs[s + 1], ks[s], ks[s + 1]
        # one 16-bit term for a weight; fp16: a largest weight of 8 at least 2^-12 of the row's scale, so that half of
        # its smallest step is 2^-16 of the largest... 2^-28 + 12 of it at worst, as paged_reference has it
        want, tol = attend_seen(f64(q[a:b]), f64(k[c:d]), f64(v[c:d]), seen(b - a, d - c, window, sinks), q.shape[2] ** -0.5,
                                kind, least=2.0 ** -25 if kind == "fp16" else 0.0)
        assert_close(got[a:b], want, tol, "sequence %d" % s)


@pytest.mark.parametrize("window,sinks", [(1, 1), (100, 3), (128, 128), (64, 200), (300, 129), (1000, 5), (50, 10 ** 9), (7, 0)])
@pytest.mark.parametrize("kind,hq,hkv,hd", [("bf16", 8, 2, 64), ("fp16", 8, 8, 128), ("bf16", 8, 1, 128), ("fp16", 4, 2, 64)])
def test_prompts_with_sinks(kind, hq, hkv, hd, window, sinks):
    q_lens, k_lens = [1, 130, 0, 700, 5, 64, 20], [1, 130, 9, 700, 900, 10, 400]
    q, k, v, qs, ks = prompt_case(kind, hq, hkv, hd, q_lens, k_lens, seed=window)
    _, msm = _mods()
    got = msm.prompt_attention(q, k, v, ints(qs), ints(ks), window=window, sinks=sinks)
    check_prompt(q, k, v, qs, ks, window, sinks, kind, got)
    if sinks == 0:
        assert np.array_equal(bits(got), bits(msm.prompt_attention(q, k, v, ints(qs), ints(ks), window=window)))


@pytest.mark.parametrize("sinks", [5, 40, 130])
def test_prompts_with_sinks_out_of_a_cache(sinks):
    """K and V in the layout of the contiguous caches, with rows to spare behind each sequence."""
    torch, msm = _mods()
    q_lens, k_lens, spare, window = [200, 33], [600, 450], 30, 100
    ks = [0, 600, 630, 1080, 1110]           # a sequence without queries stands for the spare rows
    qs = [0, 200, 200, 233, 233]
    q = randn("bf16", 233, 8, 128, seed=1).cuda()
    k, v = (randn("bf16", 2, 1110, 128, seed=i).cuda().transpose(0, 1) for i in (2, 3))
    k[600:630], v[600:630], k[1080:], v[1080:] = NAN, NAN, NAN, NAN
    out = torch.full((240, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    msm.prompt_attention(q, k, v, ints(qs), ints(ks), window=window, sinks=sinks, out=out[:233])
    assert (out[233:] == 7).all()
    for a, b, c, d in ((0, 200, 0, 600), (200, 233, 630, 1080)):
        want, tol = attend_seen(f64(q[a:b]), f64(k[c:d]), f64(v[c:d]), seen(b - a, d - c, window, sinks), 128 ** -0.5, "bf16")
        assert_close(out[a:b], want, tol)


def test_waits_of_the_prompt_kernel_with_sinks_end():
    """No key is loaded (the test hook): every wait runs out, the rows are NaN and the status says so."""
    import ctypes
    torch, msm = _mods()
    q, k, v, qs, ks = prompt_case("bf16", 4, 2, 64, [300], [300])
    out, status, st = torch.zeros_like(q), ints([0]), ints(qs)
    p = msm.MsmPrompt(device=0, dtype=msm.MSM_BF16, n_seqs=1, n_q=300, n_k=300, n_q_heads=4, n_kv_heads=2, head_dim=64,
                      window=50, scale=0.1, q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), out=out.data_ptr(),
                      q_token_stride=256, q_head_stride=64, k_token_stride=128, k_head_stride=64, v_token_stride=128,
                      v_head_stride=64, out_token_stride=256, out_head_stride=64, q_starts=st.data_ptr(),
                      k_starts=st.data_ptr(), status=status.data_ptr(), flags=msm.MSM_FLAG_TEST_DROP_HANDOFF)
    assert msm.msm_prompt_attention_sinks(p, 3, torch.cuda.current_stream().cuda_stream) == msm.MSM_OK
    torch.cuda.synchronize()
    assert int(status) == msm.MSM_ERR_DEVICE_TIMEOUT and out.isnan().all()
    p.flags = 0
    assert msm.msm_prompt_attention_sinks(p, 3, torch.cuda.current_stream().cuda_stream) == msm.MSM_OK
    want, tol = attend_seen(f64(q), f64(k), f64(v), seen(300, 300, 50, 3), 0.1, "bf16")
    assert_close(out, want, tol)


def test_a_window_of_all_keys_makes_sinks_meaningless():
    _, msm = _mods()
    q, k, v, qs, ks = prompt_case("bf16", 8, 2, 64, [300], [300])
    want = msm.prompt_attention(q, k, v, ints(qs))
    for window, sinks in ((0, 5), (300, 4), (1 << 40, 7), (10, 300), (10, 1 << 40)):
        got = msm.prompt_attention(q, k, v, ints(qs), window=window, sinks=sinks)
        assert np.array_equal(bits(got), bits(want)), (window, sinks)


def test_keys_between_the_sinks_and_the_window_have_no_part():
    """Infinities and NaN there, and at keys that only some rows of a tile see."""
    torch, msm = _mods()
    n, window, sinks = 900, 150, 70
    for kind in ("bf16", "fp16"):
        q, k, v, qs, ks = prompt_case(kind, 4, 2, 128, [n], [n], seed=2)
        want = msm.prompt_attention(q, k, v, ints(qs), window=window, sinks=sinks)
        k[200], k[300], v[200], v[300], v[301] = NAN, INF, NAN, INF, -INF
        got = msm.prompt_attention(q, k, v, ints(qs), window=window, sinks=sinks)
        away = np.array([i for i in range(n) if not any(0 <= i - j < window for j in (200, 300, 301))])
        assert np.array_equal(bits(got[away]), bits(want[away]))
        assert got[301].isnan().all()
    # an infinite value at a sink: every row that sees it
    q, k, v, qs, ks = prompt_case("bf16", 4, 2, 64, [n], [n], seed=3)
    v[5, 0, 9] = INF
    got = f64(msm.prompt_attention(q, k, v, ints(qs), window=window, sinks=sinks))
    assert np.isfinite(got[:5]).all() and (got[5:, :2, 9] == INF).all() and np.isfinite(got[5:, 2:]).all()
    got = f64(msm.prompt_attention(q, k, v, ints(qs), window=window, sinks=5))
    assert (got[5:155, :2, 9] == INF).all() and np.isfinite(got[155:]).all()


def test_a_long_prompt_with_sinks_and_a_resumed_one_agree():
    """The rows of a prompt in one call, and in pieces that continue it."""
    torch, msm = _mods()
    n, window, sinks = 5000, 512, 4
    q, k, v, qs, ks = prompt_case("bf16", 8, 2, 128, [n], [n], seed=4)
    whole = msm.prompt_attention(q, k, v, ints(qs), window=window, sinks=sinks)
    some = [0, 1, 600, 601, 4999]
    for i in some:
        want, tol = attend_seen(f64(q[i:i + 1]), f64(k[:i + 1]), f64(v[:i + 1]), seen(1, i + 1, window, sinks), 128 ** -0.5, "bf16")
        assert_close(whole[i:i + 1], want, tol, "row %d" % i)
    for a, b in ((0, 1000), (1000, 1001), (1001, 5000)):
        part = msm.prompt_attention(q[a:b], k[:b], v[:b], ints([0, b - a]), ints([0, b]), window=window, sinks=sinks)
        for i in (0, (b - a) // 2, b - a - 1):
            want, tol = attend_seen(f64(q[a + i:a + i + 1]), f64(k[:a + i + 1]), f64(v[:a + i + 1]),
                                    seen(1, a + i + 1, window, sinks), 128 ** -0.5, "bf16")
            assert_close(part[i:i + 1], want, tol)


# ------------------------------------------------------------------ sampling
FREE = 2.0 ** -34  # sums are off by at most vocab x 2^-43 of the largest weight: 2^-23 of it for 2^20 logits, 2^-34 for 512;
#                    weights round to either side, so that borders further than this from the target decide alike


def check_draw(x, u, got, temperature=None, top_k=None, top_p=None, min_p=None):
    """got: tokens, probs, kept."""
    tokens, probs, kept = (t.cpu().numpy() for t in got)
    free = max(FREE, x.shape[1] * 2.0 ** -43)
    close = 0
    for i in range(len(x)):
        par = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
        par = {n: float(v[i]) if n != "top_k" else int(v[i]) for n, v in par.items() if v is not None}
        token, n, p, room, near = draw(x[i], float(u[i]), **par)
        if room < free or near < free:
            close += 1
            continue
        assert (tokens[i], kept[i]) == (token, n), (i, par, room, near, tokens[i], token, kept[i], n)
        assert abs(probs[i] - p) <= 2.0 ** -20 * p + 2.0 ** -40, (i, probs[i], p)
    return close


def run_draw(x, u, dtype="fp32", **par):
    torch, msm = _mods()
    n = len(x)
    kept, probs = torch.full((n,), -7, dtype=torch.int32, device="cuda"), torch.full((n,), NAN, device="cuda")
    dev = {k: torch.tensor(np.asarray(v), dtype=torch.int32 if k == "top_k" else torch.float32).cuda()
           for k, v in par.items()}
    got = msm.sample(x, torch.as_tensor(u, dtype=torch.float32).cuda(), probs=probs, kept=kept, **dev)
    host = {k: v.cpu().double().numpy() for k, v in dev.items()}
    return check_draw(f64(x), torch.as_tensor(u, dtype=torch.float32).double().numpy(), (got, probs, kept), **host)


def logits(n, vocab, dtype, seed, std=2.5):
    torch, _ = _mods()
    gen = torch.Generator().manual_seed(seed)
    t = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    return (torch.randn((n, vocab), generator=gen) * std).to(t).cuda(), np.random.default_rng(seed).random(n)


SETTINGS = [{}, dict(top_k=1), dict(top_k=40), dict(top_k=3000), dict(top_p=0.0), dict(top_p=0.5), dict(top_p=0.97),
            dict(min_p=0.05), dict(min_p=1.0), dict(top_k=50, top_p=0.9), dict(top_k=5000, top_p=0.6),
            dict(top_k=2000, top_p=0.99, min_p=0.001), dict(temperature=0.3, top_p=0.9), dict(temperature=30.0, top_p=0.7),
            dict(temperature=30.0, top_k=2500), dict(temperature=0.0)]


@pytest.mark.parametrize("par", SETTINGS, ids=lambda p: "-".join("%s%s" % i for i in p.items()) or "plain")
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_draws_equal_the_reference(dtype, par):
    close = rows = 0
    for vocab, n in ((1, 3), (2, 5), (31, 40), (1000, 30), (4097, 20), (50021, 6), (131072, 3)):
        x, u = logits(n, vocab, dtype, vocab)
        close += run_draw(x, u, **{k: [v] * n for k, v in par.items()})
        rows += n
    assert close <= 2  # (expected: rows x 2 x borders x 2^-34 and less)


def test_large_vocabularies():
    for vocab, dtype in ((262144, "fp32"), (409601, "bf16"), (1 << 20, "fp32")):
        x, u = logits(2, vocab, dtype, vocab)
        for par in ({}, dict(top_k=[7, 4000]), dict(top_p=[0.9, 0.3])):
            assert run_draw(x, u, **par) <= 1


def edges(t, top, grid):
    """Logits of the grid whose class (16 of 2^-10 of log2 of the weight) depends on whether the product with
    log2(e) / t is rounded before the sum that rounds it to 2^-10."""
    c = np.float32(1.44269502162933349609375) / np.float32(t)
    d = (np.float32(top) - grid).astype(np.float32)
    apart = ((d * c).astype(np.float32) + np.float32(12288)).astype(np.float32).view(np.int32) >> 4
    at_once = (d.astype(np.float64) * np.float64(c) + 12288).astype(np.float32).view(np.int32) >> 4
    return grid[(apart != at_once) & (d * c < 15)]


def test_logits_on_the_edges_of_classes():
    """Every step of a draw has to give a logit the same class: the border lies among logits on an edge."""
    torch, _ = _mods()
    rng = np.random.default_rng(21)
    grid = np.arange(-4000, 4000).astype(np.float32) / 512     # exact in fp16 and fp32
    rows, temps, ps = [], [], []
    while len(rows) < 150:
        t = np.float32(rng.uniform(0.4, 3.0))
        for x in edges(t, 8.0, grid)[:3]:
            row = np.full(3000, -6.0, np.float32)
            at = rng.permutation(np.arange(8, 3000))
            n = int(rng.choice([100, 900]))                    # in front: with and without them in the list
            row[7], row[at[:120]], row[at[120:120 + n]] = 8.0, x, min(8.0, x + 0.5)
            w = np.exp((row.astype(np.float64) - 8) / t)
            rows.append(row)
            temps.append(float(t))
            ps.append(float((w[row > x].sum() + 0.4 * w[row == x].sum()) / w.sum()))
    x, u = torch.from_numpy(np.stack(rows)).cuda(), rng.random(len(rows))
    # The target is the sum that ends with the 48th of the 120, up to top_p's rounding to fp32, and so within 3000 x 2^-43
    # of a border for sum(3000 x 2^-43 / (half a step of top_p)) = 2.3 of the rows on average, by the inputs alone: the
    # number follows Poisson's law, and exceeds 8 once in 2,000 times.
    for dtype in (torch.float32, torch.float16):
        assert run_draw(x.to(dtype), u, temperature=temps, top_p=ps) <= 8
        k = [int((r > 0).sum()) + 9 for r in rows]
        assert run_draw(x.to(dtype), u, temperature=temps, top_k=k, top_p=[0.95] * len(k)) <= 2


def test_borders_far_below_the_largest_logit():
    """One logit far above a broad body: the border lies where the first histogram has its last class."""
    for vocab, dtype, spike in ((3000, "fp32", 22.0), (60000, "fp32", 26.0), (131072, "bf16", 24.0), (40000, "fp32", 60.0)):
        x, u = logits(4, vocab, dtype, 5, std=1.0)
        x[:, 77] = spike
        u = 1 - u * 2.0 ** -24
        for par in (dict(top_p=[0.9999, 0.99999, 0.999999, 0.5]), dict(top_k=[2500, 700, 2, 1]),
                    dict(top_k=[2900, 1300, 600, 9], top_p=[0.99999] * 4), dict(min_p=[1e-11, 1e-9, 1e-8, 0.1]), {}):
            run_draw(x, u, **par)


def test_logits_past_two_to_the_31_elements():
    torch, msm = _mods()
    stride, vocab = (1 << 30) + 3, 40000
    room = torch.empty(2 * stride + vocab, dtype=torch.bfloat16, device="cuda")
    x = room.as_strided((3, vocab), (stride, 1))
    y, u = logits(3, vocab, "bf16", 9)
    x.copy_(y)
    ud = torch.from_numpy(u).float().cuda()
    for par in ({}, dict(top_p=torch.full((3,), 0.8, device="cuda")), dict(top_k=ints([50, 5, 5000]))):
        assert torch.equal(msm.sample(x, ud, **par), msm.sample(y, ud, **par))


def test_a_batch_with_settings_of_its_own():
    rng = np.random.default_rng(3)
    for n, vocab, dtype in ((300, 3001, "fp32"), (700, 50, "fp16"), (160, 20001, "bf16")):
        x, u = logits(n, vocab, dtype, n)
        close = run_draw(x, u, temperature=rng.choice([0.0, 0.5, 1.0, 2.0], n), top_k=rng.choice([0, -1, 5, 100, vocab + 9], n),
                         top_p=rng.choice([0.1, 0.9, 1.0], n), min_p=rng.choice([0.0, 0.02, 0.5], n))
        assert close <= 2


@pytest.mark.parametrize("vocab", [40, 2500, 33000])
def test_equal_logits_are_taken_from_the_lowest_index_on(vocab):
    torch, _ = _mods()
    rng = np.random.default_rng(vocab)
    n = 12
    few = torch.from_numpy(rng.choice([0.0, -0.0, 1.0, 1.5, -20.0], (n, vocab))).float().cuda()
    same = torch.full((n, vocab), 3.25, device="cuda")
    zero = torch.where(torch.rand(n, vocab, device="cuda") < 0.5, 0.0, -0.0)
    for x in (few, same, zero, few.bfloat16()):
        for par in (dict(top_k=[max(1, vocab // 3)] * n), dict(top_p=[0.37] * n), dict(temperature=[0.0] * n),
                    dict(top_k=[max(1, vocab // 2)] * n, top_p=[0.31] * n), dict(min_p=[1.0] * n), {}):
            run_draw(x, (rng.integers(0, 1000, n) + 0.377) / 1000, **par)


def test_rows_without_a_choice_and_masked_rows():
    torch, msm = _mods()
    x, u = logits(10, 5000, "fp32", 1)
    x[0] = -INF
    x[1] = NAN
    x[2, :] = -INF
    x[2, 4321] = -3.0
    x[3, ::2] = NAN
    x[4, 1:] = torch.finfo(torch.float32).min   # masks of the type's lowest value
    x[5] = torch.finfo(torch.float32).min
    x[6, 17], x[6, 99] = INF, INF
    x[7, 5] = torch.finfo(torch.float32).max
    x[8, 100:] = -INF
    for par in ({}, dict(top_k=[50] * 10), dict(top_p=[0.8] * 10), dict(temperature=[0.0] * 10), dict(min_p=[0.1] * 10),
                dict(top_k=[4999] * 10, top_p=[0.999] * 10), dict(temperature=[1e-38] * 10), dict(temperature=[1e-45] * 10),
                dict(temperature=[3e38] * 10, top_p=[0.5] * 10), dict(top_k=[2 ** 31 - 1] * 10), dict(top_k=[-2 ** 31] * 10)):
        run_draw(x, u, **par)
        run_draw(x.bfloat16(), u, **par)


def test_random_numbers_at_the_ends():
    x, _ = logits(6, 3000, "fp32", 2)
    for u in (0.0, 1.0, 1 - 2.0 ** -24, 2.0 ** -149):
        for par in ({}, dict(top_k=[9] * 6), dict(top_p=[0.5] * 6)):
            torch, msm = _mods()
            dev = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32).cuda() for k, v in par.items()}
            kept = torch.empty(6, dtype=torch.int32, device="cuda")
            got = msm.sample(x, torch.full((6,), u, device="cuda"), kept=kept, **dev).cpu().numpy()
            for i in range(6):
                host = {k: v[i] for k, v in par.items()}
                assert got[i] == draw(f64(x[i]), u, **host)[0], (u, par, i)


def test_numbers_out_of_range_give_no_token():
    torch, msm = _mods()
    x, u = logits(12, 100, "fp32", 4)
    t, p, m, u = [1.0] * 12, [0.9] * 12, [0.1] * 12, list(u)
    t[0], t[1], t[2] = -1.0, NAN, INF
    p[3], p[4], p[5] = -0.1, 1.5, NAN
    m[6], m[7] = 1.1, NAN
    u[8], u[9], u[10] = -0.5, 1.5, NAN
    probs, kept = torch.full((12,), 3.0, device="cuda"), torch.full((12,), 3, dtype=torch.int32, device="cuda")
    par = [torch.tensor(v, dtype=torch.float32, device="cuda") for v in (u, t, p, m)]
    got = msm.sample(x, par[0], temperature=par[1], top_p=par[2], min_p=par[3], probs=probs, kept=kept)
    assert (got[:11] == -1).all() and got[11] >= 0
    assert (probs[:11] == 0).all() and (kept[:11] == 0).all() and kept[11] > 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_at_any_address(dtype):
    torch, msm = _mods()
    x, u = logits(5, 2011, dtype, 6)
    ud = torch.from_numpy(u).float().cuda()
    want = msm.sample(x, ud)
    for off, stride in ((1, 2013), (3, 2011), (5, 4096), (7, 2019)):
        room = torch.full((off + 5 * stride + 8,), NAN, dtype=x.dtype, device="cuda")
        y = room[off:off + 5 * stride].view(5, stride)[:, :2011]
        y.copy_(x)
        assert torch.equal(msm.sample(y, ud), want)
    out = torch.empty(5, dtype=torch.int32, device="cuda")
    assert msm.sample(x, ud, out=out) is out and torch.equal(out, want)
    assert msm.sample(x[:0], ud[:0]).numel() == 0
    for bad in (dict(random=ud[:4]), dict(random=ud.double()), dict(random=None)):
        with pytest.raises(ValueError):
            msm.sample(x, **bad)
    with pytest.raises(ValueError):
        msm.sample(x.t(), ud)
    with pytest.raises(ValueError):
        msm.sample(x, ud, top_k=ud)


def test_the_same_draw_every_time_and_the_right_shares():
    torch, msm = _mods()
    x, _ = logits(1, 50000, "fp32", 8)
    u = torch.rand(64, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    row = x.expand(64, 50000)
    par = dict(top_p=torch.full((64,), 0.95, device="cuda"))
    first = msm.sample(row, u, **par)
    for _ in range(5):
        assert torch.equal(msm.sample(row, u, **par), first)
    # evenly spread numbers: each token is drawn as often as its weight says, to one
    y = torch.tensor([0.0, 1.0, -1.0, 2.0, -INF, 0.5], device="cuda")
    n = 20000
    got = msm.sample(y.expand(n, 6), (torch.arange(n, device="cuda") + 0.5) / n)
    share = torch.softmax(y.double(), 0) * n
    assert ((torch.bincount(got, minlength=6) - share).abs() <= 1.01).all()


# ------------------------------------------------------------------ streams, graphs, a whole step
def test_other_streams_and_a_captured_step():
    """Write, attention and sampling of a few steps, eagerly on a side stream and as one graph replayed,
    against the reference of each operator."""
    torch, msm = _mods()
    n, hq, hkv, hd, vocab, window, sinks = 3, 4, 2, 64, 1500, 24, 3
    gen = torch.Generator("cuda").manual_seed(0)
    table = torch.randn((vocab, (hq + 2 * hkv) * hd), generator=gen, device="cuda", dtype=torch.bfloat16)
    head = torch.randn((hq * hd, vocab), generator=gen, device="cuda", dtype=torch.bfloat16) * 0.3
    state = {}

    def setup():
        c = msm.PagedCache.allocate(1, 40, 8, hkv, hd, n, 12, dtype=torch.float8_e4m3fn, block_rows=4)
        state.update(c=c, tokens=torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda"),
                     target=torch.zeros(n, dtype=torch.int32, device="cuda"),
                     u=torch.zeros(n, device="cuda"), top_p=torch.full((n,), 0.9, device="cuda"),
                     starts=ints([0, 1, 2, 3]), kept=torch.zeros(n, dtype=torch.int32, device="cuda"))

    def step():
        s = state
        s["target"] += 1
        s["c"].resize(s["target"])
        x = table[s["tokens"].long()].view(n, hq + 2 * hkv, hd)
        s["c"].write(0, x[:, hq:hq + hkv], x[:, hq + hkv:], s["starts"])
        s["o"] = s["c"].attention(0, x[:, :hq], window=window, sinks=sinks)
        s["logits"] = s["o"].view(n, -1) @ head
        msm.sample(s["logits"], s["u"], top_p=s["top_p"], out=s["tokens"], kept=s["kept"])

    us = torch.rand((60, n), generator=gen, device="cuda")
    side = torch.cuda.Stream()
    setup()
    eager = []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(60):
            state["u"].copy_(us[i])
            x_before = state["tokens"].clone()
            step()
            eager.append((state["tokens"].clone(), state["o"].clone(), state["logits"].clone(), x_before))
    side.synchronize()
    state["c"].sync()
    # the last step against the references
    tokens, o, lg, fed = eager[-1]
    hist = torch.stack([e[3] for e in eager], 1).long()  # [n, 60] tokens that were fed
    ref = QPages(40, 8, n, 12, [np.zeros((40, hkv, 8, hd), np.uint8) for _ in range(2)], block_rows=4,
                 scales=[np.zeros((40, hkv, 2)) for _ in range(2)])
    x = f64(table[hist].view(n, 60, hq + 2 * hkv, hd))
    for i in range(60):
        assert ref.resize([i + 1] * n) is None
        ref.write(0, x[:, i, hq:hq + hkv], [0, 1, 2, 3])
        ref.write(1, x[:, i, hq + hkv:], [0, 1, 2, 3])
    assert np.array_equal(codes(state["c"].k_pages[0]), ref.pools[0]) and np.array_equal(codes(state["c"].v_pages[0]), ref.pools[1])
    check_decode(state["c"], table[hist[:, -1]].view(n, -1, hd)[:, :hq], ref.table, [60] * n, 8, "bf16", window, sinks, o)
    for i in range(n):
        t, _, _, room, near = draw(f64(lg[i]), float(us[-1][i].double()), top_p=float(state["top_p"][i].double()))
        assert t == int(tokens[i]) or min(room, near) < FREE
    # the same as a graph, twice from the beginning (the tables go back; pages and scales keep what they hold)
    setup()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        state["c"].resize(torch.zeros(n, dtype=torch.int32, device="cuda"))
        state["target"].zero_()
        state["tokens"].copy_(torch.tensor([5, 6, 7], dtype=torch.int32))
        for i in range(60):
            state["u"].copy_(us[i])
            graph.replay()
            assert torch.equal(state["tokens"], eager[i][0]) and torch.equal(state["o"], eager[i][1]), i
    state["c"].sync()


def test_two_graphs_and_an_eager_call_at_once():
    """Calls that a graph records take workspaces of their own."""
    torch, msm = _mods()
    lens = [3000, 1, 700]
    cache, q, table = decode_case("bf16", 8, 2, 128, 64, lens, block=16, seed=9)
    q2 = q.flip(0).contiguous()
    want = [cache.attention(0, x, window=500, sinks=4).clone() for x in (q, q2)]
    outs, graphs = [], []
    for x in (q, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cache.attention(0, x, window=500, sinks=4))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        mine = cache.attention(0, q, window=500, sinks=4)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(mine, want[0])


def test_rows_past_two_to_the_31_bytes():
    """A pool of 8 bits and its scales where offsets leave 32 bits."""
    torch, msm = _mods()
    n_pages, hkv, rows, hd = 70000, 8, 64, 128  # 4.6 GB a pool
    c = msm.PagedCache.allocate(1, n_pages, rows, hkv, hd, 2, 4, dtype=torch.float8_e4m3fn, block_rows=16)
    c.refs[:n_pages - 6] = 1
    c.resize(ints([130, 200 - 64]))
    kv = randn("bf16", 266, 2 * hkv, hd, seed=1).cuda()
    c.write(0, kv[:, :hkv], kv[:, hkv:], ints([0, 130, 266]))
    q = randn("bf16", 2, 16, hd, seed=2).cuda()
    got = c.attention(0, q)
    c.sync()
    small = msm.PagedCache.allocate(1, 6, rows, hkv, hd, 2, 4, dtype=torch.float8_e4m3fn, block_rows=16)
    small.resize(ints([130, 136]))
    small.write(0, kv[:, :hkv], kv[:, hkv:], ints([0, 130, 266]))
    assert torch.equal(small.attention(0, q), got)
    assert torch.equal(c.k_pages[0][-6:].view(torch.uint8), small.k_pages[0].view(torch.uint8))
    c.refs[:n_pages - 6] = 0
    c.compact()
    assert torch.equal(c.attention(0, q), got)
    c.sync()
