"""Measured cases of decoding streams from a cache held in 8 bits.

Five operators, each in the form a serving loop calls it:

  prompt   causal attention of packed prompts on a sliding window with sinks: the first tokens
           of a sequence stay visible behind the window
  decode   attention of one new token per sequence over the paged cache, window and sinks
  q_decode the same over a cache held in 8 bits (e4m3), a scale for each block of tokens and head
  q_write  reserving the pages of new tokens and storing their K/V rows in 8 bits
  sample   drawing the next tokens from logits with temperature, top-k, top-p and min-p, one given
           random number per row

``own`` selects the framework's calls; without it ``run`` computes the same results with
elementary torch operations in 32 bits (sampling, and what decides between two tokens, in 64).
"""
import math
import random

import torch

own = False

BF16, FP16, FP32 = "bf16", "fp16", "fp32"
_DTYPES = {BF16: torch.bfloat16, FP16: torch.float16, FP32: torch.float32}
_E4M3 = torch.float8_e4m3fn
_TOP = 448.0  # the largest e4m3 value


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a batch of turns that continue streams whose first rows stay in contiguous caches
        dict(name="prompt_turns", op="prompt", dtype=FP16, hq=32, hkv=8, hd=128, seqs=12, shortest=1, longest=1500,
             lens=1, prefix=2500, window=1024, sinks=4, in_cache=True),
        # one long document on a sliding-window layer
        dict(name="prompt_document", op="prompt", dtype=BF16, hq=32, hkv=8, hd=128, seqs=1, shortest=32768,
             longest=32768, lens=2, prefix=0, window=2048, sinks=4, in_cache=False),
        # one user's stream on the smallest head layout: latency
        dict(name="decode_stream", op="decode", dtype=BF16, hq=8, hkv=2, hd=64, seqs=1, shortest=3001, longest=3001,
             lens=3, page=16, window=128, sinks=4),
        # a batch of streams, most of them longer than the window
        dict(name="decode_streams", op="decode", dtype=FP16, hq=32, hkv=8, hd=128, seqs=128, shortest=700,
             longest=8192, lens=4, page=64, window=2048, sinks=64),
        # one user, a short history: latency
        dict(name="q_decode_one", op="q_decode", dtype=BF16, hq=8, hkv=2, hd=64, seqs=1, shortest=200, longest=200,
             lens=5, page=16, block=16, window=0, sinks=0),
        # a batch of ragged conversations on a global layer
        dict(name="q_decode_batch", op="q_decode", dtype=FP16, hq=32, hkv=8, hd=128, seqs=64, shortest=1,
             longest=8192, lens=6, page=64, block=16, window=0, sinks=0),
        # one long document on a global layer
        dict(name="q_decode_long", op="q_decode", dtype=BF16, hq=32, hkv=8, hd=128, seqs=1, shortest=131071,
             longest=131071, lens=7, page=256, block=64, window=0, sinks=0),
        # one step of a batch: one token per sequence behind its history
        dict(name="q_write_step", op="q_write", dtype=BF16, hkv=8, hd=128, seqs=32, shortest=20, longest=4000, lens=8,
             page=64, block=16, new=1),
        # whole prompts of a batch
        dict(name="q_write_prompt", op="q_write", dtype=BF16, hkv=8, hd=128, seqs=8, shortest=6250, longest=6250,
             lens=9, page=64, block=16, new=0),
        # one user's next token: latency
        dict(name="sample_one", op="sample", dtype=FP32, rows=1, vocab=32003, temperature=0.8, top_k=50, top_p=0.95,
             min_p=0.0, per_row=False, params=10),
        # a batch of users, each with settings of their own
        dict(name="sample_batch", op="sample", dtype=FP32, rows=64, vocab=131072, temperature=1.0, top_k=200,
             top_p=0.9, min_p=0.02, per_row=True, params=11),
        # many rows of 16-bit logits, the nucleus alone
        dict(name="sample_wide", op="sample", dtype=BF16, rows=500, vocab=50021, temperature=1.0, top_k=0, top_p=0.95,
             min_p=0.0, per_row=False, params=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "decode", "q_decode", "q_write", "sample"])
    lens = rng.randrange(1 << 20)
    if op == "sample":
        vocab = _log(rng, 50, 262144)
        return dict(op=op, dtype=rng.choice([FP32, BF16, FP16]), rows=_log(rng, 1, max(1, min(512, (1 << 23) // vocab))),
                    vocab=vocab, temperature=round(math.exp(rng.uniform(math.log(0.2), math.log(3))), 3),
                    top_k=rng.choice([0, 0, _log(rng, 1, 5000)]), top_p=rng.choice([1.0, round(rng.uniform(0.1, 0.99), 3)]),
                    min_p=rng.choice([0.0, 0.0, round(rng.uniform(0.001, 0.3), 4)]), per_row=rng.random() < 0.5,
                    params=lens)
    dtype, hd = rng.choice([BF16, FP16]), rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    if op == "prompt":
        longest = _log(rng, 1, 8192)
        return dict(op=op, dtype=dtype, hq=hq, hkv=hkv, hd=hd, seqs=_log(rng, 1, max(1, min(32, 16384 // longest))),
                    shortest=rng.randint(1, longest), longest=longest, lens=lens,
                    prefix=rng.choice([0, _log(rng, 1, 4096)]), window=_log(rng, 1, 4096), sinks=_log(rng, 1, 300),
                    in_cache=rng.random() < 0.5)
    page = _log(rng, 4, 256)
    block = rng.randint(1, page) if rng.random() < 0.5 else page
    if op == "q_write":
        longest = _log(rng, 1, 8192)
        return dict(op=op, dtype=dtype, hkv=hkv, hd=hd, seqs=_log(rng, 1, max(1, min(128, 65536 // longest))),
                    shortest=rng.randint(1, longest), longest=longest, lens=lens, page=page, block=block,
                    new=rng.choice([0, 1, rng.randint(1, 64)]))
    longest = _log(rng, 1, 65536)
    case = dict(op=op, dtype=dtype, hq=hq, hkv=hkv, hd=hd, seqs=_log(rng, 1, max(1, min(256, 131072 // longest))),
                shortest=rng.randint(0, longest), longest=longest, lens=lens, page=page)
    if op == "q_decode":
        case["block"] = block
    streams = op == "decode" or rng.random() < 0.5
    case.update(window=_log(rng, 1, 4096) if streams else 0, sinks=_log(rng, 1, 300) if streams else 0)
    return case


def _lengths(case):
    """The sequences' lengths: the longest and the shortest first, the rest spread over the
    logarithm of the range between them."""
    rng = random.Random(case["lens"])
    lo, hi = case["shortest"], case["longest"]
    out = [hi, lo] + [_log(rng, max(lo, 1), max(hi, 1)) for _ in range(case["seqs"])]
    return out[:case["seqs"]]


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype):
    """N(0, 1) values, drawn in 32 bits a slice at a time."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 27
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device="cuda")
    return out


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _tables(state, rng, lens, max_pages, n_pages, page):
    """A table of the pages of `lens` (taken from the pool in a random order), its lengths and
    the pages' reference counts, in one buffer."""
    order = list(range(n_pages))
    rng.shuffle(order)
    table = [[-1] * max_pages for _ in lens]
    refs = [0] * n_pages
    at = 0
    for s, n in enumerate(lens):
        for j in range(_ceil(n, page)):
            table[s][j] = order[at]
            refs[order[at]] = 1
            at += 1
    slots = len(lens)
    state["meta"] = _ints([p for row in table for p in row] + list(lens) + refs)
    state["saved"] = state["meta"].clone()
    a, b = slots * max_pages, slots * max_pages + slots
    state["table"] = state["meta"][:a].view(slots, max_pages)
    state["lens"] = state["meta"][a:b]
    state["refs"] = state["meta"][b:]


def _quantised_pool(case, gen, n_pages):
    """A pool in 8 bits with its scales; the heads differ in size, as keys and values do."""
    hkv, page, hd, block = case["hkv"], case["page"], case["hd"], case["block"]
    nb = _ceil(page, block)
    pool = torch.empty((n_pages, hkv, page, hd), dtype=_E4M3, device="cuda")
    scales = torch.empty((n_pages, hkv, nb), dtype=torch.float32, device="cuda")
    size = torch.exp(torch.randn((1, hkv, 1, 1), generator=gen, device="cuda"))
    step = max(1, (1 << 25) // (hkv * page * hd))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        x = torch.zeros((n, hkv, nb * block, hd), device="cuda")
        x[:, :, :page] = torch.randn((n, hkv, page, hd), generator=gen, device="cuda") * size
        x = x.view(n, hkv, nb, block, hd)
        s = _power(x.abs().amax((-1, -2)))
        scales[i:i + n] = s
        pool[i:i + n] = (x / s[..., None, None]).view(n, hkv, nb * block, hd)[:, :, :page].to(_E4M3)
    return pool, scales


def _power(amax):
    """The least power of two that amax / 448 does not exceed (at least 2^-126), 0 for 0."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _handle(state):
    """The cache object a user's program keeps."""
    if own:
        from moe_decode_megakernel_warp_gb300 import PagedCache
        if "ks" in state:
            state["cache"] = PagedCache(state["k"], state["v"], state["table"], state["lens"], state["refs"],
                                        k_scales=state["ks"], v_scales=state["vs"], block_rows=state["case"]["block"])
        else:
            state["cache"] = PagedCache(state["k"], state["v"], state["table"], state["lens"], state["refs"])


def _logits(case, gen):
    """Rows of a language model's kind: a broad body, in every other row a few likely tokens on top,
    in every fourth one half of the vocabulary ruled out."""
    rows, vocab = case["rows"], case["vocab"]
    x = torch.randn((rows, vocab), generator=gen, device="cuda") * 2.5
    at = torch.randint(0, vocab, (rows, 8), generator=gen, device="cuda")
    up = torch.rand((rows, 8), generator=gen, device="cuda") * 14
    x[::2].scatter_add_(1, at[::2], up[::2])
    ruled = torch.rand((len(x[3::4]), vocab), generator=gen, device="cuda") < 0.5
    x[3::4] = x[3::4].masked_fill(ruled, float("-inf"))
    return x.to(_DTYPES[case["dtype"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    op, t = case["op"], _DTYPES[case["dtype"]]
    state = dict(case=case)
    if op == "sample":
        rows = case["rows"]
        state["logits"] = _logits(case, gen)
        state["random"] = torch.rand(rows, generator=gen, device="cuda")
        temperature, top_k, top_p, min_p = ([case[n]] * rows for n in ("temperature", "top_k", "top_p", "min_p"))
        if case["per_row"]:  # every user's own; some want the most likely token
            pick = random.Random(case["params"])
            temperature = [pick.choice([0.0, v, v * pick.uniform(0.3, 1.5), v * pick.uniform(0.3, 1.5)]) for v in temperature]
            top_k = [pick.choice([0, v, _log(pick, 1, v)]) if v else 0 for v in top_k]
            top_p = [pick.choice([1.0, v, v * pick.uniform(0.5, 1.0)]) if v < 1 else 1.0 for v in top_p]
            min_p = [pick.choice([0.0, v, v * pick.uniform(0.5, 1.5)]) if v else 0.0 for v in min_p]
        state["top_k"] = _ints(top_k) if case["top_k"] else None
        for name, v, given in (("temperature", temperature, True), ("top_p", top_p, case["top_p"] < 1),
                               ("min_p", min_p, case["min_p"] > 0)):
            state[name] = torch.tensor(v, dtype=torch.float32, device="cuda") if given else None
        # the buffers that a serving loop keeps
        state["tokens"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        state["kept"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        state["probs"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        return state
    lens = _lengths(case)
    if op == "prompt":
        hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
        cu_q, cu_k = _cu(lens), _cu([n + case["prefix"] for n in lens])
        state.update(cu_q=cu_q, cu_k=cu_k, q_starts=_ints(cu_q), k_starts=_ints(cu_k))
        if case["prefix"] == 0 and not case["in_cache"]:
            # the packed output of the QKV projection
            qkv = _normal(gen, (cu_q[-1], hq + 2 * hkv, hd), t)
            state.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
        else:
            state["q"] = _normal(gen, (cu_q[-1], hq, hd), t)
            if case["in_cache"]:  # [kv heads][rows][head dim]
                state["k"] = _normal(gen, (hkv, cu_k[-1], hd), t).transpose(0, 1)
                state["v"] = _normal(gen, (hkv, cu_k[-1], hd), t).transpose(0, 1)
            else:
                state["k"] = _normal(gen, (cu_k[-1], hkv, hd), t)
                state["v"] = _normal(gen, (cu_k[-1], hkv, hd), t)
        return state
    page = case["page"]
    if op == "q_write":
        # `new` tokens behind each history, or the whole prompts
        news = [case["new"] or n for n in lens]
        base = [n if case["new"] else 0 for n in lens]
        after = [b + n for b, n in zip(base, news)]
        n_pages = sum(_ceil(n, page) for n in after) + 8
        _tables(state, rng, base, max(_ceil(n, page) for n in after), n_pages, page)
        cu = _cu(news)
        state.update(starts=_ints(cu), cu=cu, target=_ints(after))
        kv = _normal(gen, (cu[-1], 2 * case["hkv"], case["hd"]), t)
        state.update(new_k=kv[:, :case["hkv"]], new_v=kv[:, case["hkv"]:])
    else:
        pages = [_ceil(n, page) for n in lens]
        n_pages = max(1, sum(pages) + max(1, sum(pages) // 16))
        _tables(state, rng, lens, max(1, max(pages)), n_pages, page)
        state["host_lens"] = lens
        state["q"] = _normal(gen, (len(lens), case["hq"], case["hd"]), t)
    if op == "decode":
        shape = (n_pages, case["hkv"], page, case["hd"])
        state["k"], state["v"] = [_normal(gen, shape, t)], [_normal(gen, shape, t)]
    else:
        k, ks = _quantised_pool(case, gen, n_pages)
        v, vs = _quantised_pool(case, gen, n_pages)
        state.update(k=[k], v=[v], ks=[ks], vs=[vs])
    _handle(state)
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_prompt(s):
    from moe_decode_megakernel_warp_gb300 import prompt_attention
    c = s["case"]
    return prompt_attention(s["q"], s["k"], s["v"], s["q_starts"], s["k_starts"], window=c["window"], sinks=c["sinks"])


def _own_decode(s):
    return s["cache"].attention(0, s["q"], window=s["case"]["window"], sinks=s["case"]["sinks"])


# Each pass begins from the same tables, as a program that goes back to a saved point does, so that every
# pass does the same work.  (The rows and scales of a pass that is repeated are those it left before.)
def _own_q_write(s):
    s["meta"].copy_(s["saved"])
    s["cache"].resize(s["target"])
    s["cache"].write(0, s["new_k"], s["new_v"], s["starts"])
    return [s["table"], s["lens"], s["refs"], s["k"][0], s["v"][0], s["ks"][0], s["vs"][0]]


def _own_sample(s):
    from moe_decode_megakernel_warp_gb300 import sample
    sample(s["logits"], s["random"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
           min_p=s["min_p"], out=s["tokens"], probs=s["probs"], kept=s["kept"])
    return [s["tokens"], s["kept"], s["probs"]]


_OWN = dict(prompt=_own_prompt, decode=_own_decode, q_decode=_own_decode, q_write=_own_q_write, sample=_own_sample)


# ------------------------------------------------------------------ plain forms
def _softmax_times(scores, seen, v):
    """softmax over the seen keys times v, a row that sees no key giving zeros."""
    scores = scores.masked_fill(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, torch.ones_like(total), total)


def _plain_prompt(s):
    c = s["case"]
    hq, hkv, hd, window, sinks = c["hq"], c["hkv"], c["hd"], c["window"], c["sinks"]
    group = hq // hkv
    out = torch.empty((s["cu_q"][-1], hq, hd), dtype=s["q"].dtype, device="cuda")
    for b in range(c["seqs"]):
        q0, q1, k0, k1 = s["cu_q"][b], s["cu_q"][b + 1], s["cu_k"][b], s["cu_k"][b + 1]
        nq, nk = q1 - q0, k1 - k0
        shift = nk - nq
        for i0 in range(0, nq, 512):
            i1 = min(nq, i0 + 512)
            hi = max(0, i1 + shift)
            lo = max(0, i0 + shift - window + 1) if window else 0
            first = min(sinks, lo)
            j = torch.cat([torch.arange(first, device="cuda"), torch.arange(lo, hi, device="cuda")])
            q = s["q"][q0 + i0:q0 + i1].float().view(i1 - i0, hkv, group, hd).permute(1, 2, 0, 3)
            k = s["k"][k0 + j].float().transpose(0, 1).unsqueeze(1)
            v = s["v"][k0 + j].float().transpose(0, 1).unsqueeze(1)
            scores = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(hd))
            i = torch.arange(i0, i1, device="cuda").unsqueeze(1) + shift
            j = j.unsqueeze(0)
            seen = (j <= i) & ((i - j < window) | (j < sinks)) if window else j <= i
            o = _softmax_times(scores, seen, v)
            out[q0 + i0:q0 + i1] = o.permute(2, 0, 1, 3).reshape(i1 - i0, hq, hd).to(out.dtype)
    return out


def _seen_rows(n, window, sinks):
    """The rows that the newest token of n sees."""
    first = max(0, n - window) if window else 0
    return torch.cat([torch.arange(min(sinks, first), device="cuda"), torch.arange(first, n, device="cuda")])


def _rows_of(s, name, b, r):
    """Rows r of sequence b as [kv heads][rows][head dim] in 32 bits."""
    page = s["case"]["page"]
    ids, at = s["table"][b].long()[r // page], r % page
    pool = s[name][0]
    if pool.dtype != _E4M3:
        return pool[ids, :, at].float().transpose(0, 1)
    rows = pool.view(torch.uint8)[ids, :, at].view(_E4M3).float()
    return (rows * s[name + "s"][0][ids, :, at // s["case"]["block"]].unsqueeze(-1)).transpose(0, 1)


def _plain_decode(s):
    c = s["case"]
    hq, hkv, hd = c["hq"], c["hkv"], c["hd"]
    out = torch.zeros_like(s["q"])
    for b, n in enumerate(s["host_lens"]):
        if n == 0:
            continue
        r = _seen_rows(n, c["window"], c["sinks"])
        k, v = _rows_of(s, "k", b, r), _rows_of(s, "v", b, r)
        q = s["q"][b].float().view(hkv, hq // hkv, hd)
        scores = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(hd))
        out[b] = _softmax_times(scores, torch.ones_like(scores, dtype=torch.bool), v).view(hq, hd).to(out.dtype)
    return out


def _plain_resize(s):
    """Lengths grow; no page is shared."""
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["case"]["page"]
    old, new = lens.long(), s["target"].long()
    n_old, n_new = (old + page - 1) // page, (new + page - 1) // page
    j = torch.arange(table.shape[1], device="cuda").unsqueeze(0)
    want = (j >= n_old.unsqueeze(1)) & (j < n_new.unsqueeze(1))
    index = torch.arange(refs.numel(), device="cuda")
    free = torch.sort(torch.where(refs == 0, index, index + refs.numel())).values
    rank = (torch.cumsum(want.reshape(-1).long(), 0) - 1).clamp(min=0).view_as(want)
    taken = free[rank] % refs.numel()
    refs.index_add_(0, taken.reshape(-1), want.reshape(-1).int())
    table.copy_(torch.where(want, taken.int(), table))
    lens.copy_(new.int())


def _plain_store(pool, scales, x, ids, row, block):
    """Rows x [tokens][heads][head dim] into rows `row` of pages `ids`."""
    page = pool.shape[2]
    held = pool.view(torch.uint8)
    nb = scales.shape[2]
    blocks, of = torch.unique(ids * nb + row // block, return_inverse=True)
    p, b = blocks // nb, blocks % nb
    x = x.float()
    amax = torch.zeros((len(blocks), x.shape[1]), device="cuda").index_reduce_(0, of, x.abs().amax(-1), "amax")
    older = torch.full((len(blocks),), block, device="cuda").index_reduce_(0, of, row % block, "amin")
    had = scales[p, :, b] * (older > 0).unsqueeze(1)
    now = torch.maximum(_power(amax), had)
    # the rows that the blocks held before, on the new scales
    i = torch.arange(block, device="cuda").unsqueeze(0)
    at = b.unsqueeze(1) * block + i
    n, k = torch.nonzero((i < older.unsqueeze(1)) & (at < page), as_tuple=True)
    pn, rn = p[n], at[n, k]
    ratio = torch.where(now > 0, had / torch.where(now > 0, now, 1.0), 0.0)
    held[pn, :, rn] = (held[pn, :, rn].view(_E4M3).float() * ratio[n].unsqueeze(-1)).to(_E4M3).view(torch.uint8)
    inverse = torch.where(now > 0, 1.0 / torch.where(now > 0, now, 1.0), 0.0)
    held[ids, :, row] = (x * inverse[of].unsqueeze(-1)).to(_E4M3).view(torch.uint8)
    scales[p, :, b] = now


def _plain_q_write(s):
    s["meta"].copy_(s["saved"])
    _plain_resize(s)
    cu, page, block = s["cu"], s["case"]["page"], s["case"]["block"]
    counts = s["starts"].diff().long()
    seq = torch.repeat_interleave(torch.arange(len(cu) - 1, device="cuda"), counts, output_size=cu[-1])
    pos = torch.arange(cu[-1], device="cuda") - s["starts"].long()[seq] + (s["lens"].long() - counts)[seq]
    ids = s["table"][seq, pos // page].long()
    # (a page's blocks begin anew with the page)
    row = pos % page
    for name in ("k", "v"):
        _plain_store(s[name][0], s[name + "s"][0], s["new_" + name], ids, row, block)
    return [s["table"], s["lens"], s["refs"], s["k"][0], s["v"][0], s["ks"][0], s["vs"][0]]


def _plain_sample(s):
    x = s["logits"].double()
    rows, vocab = x.shape
    none = torch.zeros(rows, device="cuda")
    t = (s["temperature"] if s["temperature"] is not None else none + 1).double().unsqueeze(1)
    top_k = (s["top_k"] if s["top_k"] is not None else none).long().unsqueeze(1)
    top_p = (s["top_p"] if s["top_p"] is not None else none + 1).double().unsqueeze(1)
    min_p = (s["min_p"] if s["min_p"] is not None else none).double().unsqueeze(1)
    ordered, order = torch.sort(x, dim=1, descending=True, stable=True)  # equal logits: the lower index first
    top = ordered[:, :1]
    rank = torch.arange(vocab, device="cuda").unsqueeze(0)
    weight = torch.where(t > 0, torch.exp((ordered - top) / torch.where(t > 0, t, 1.0)), (rank == 0).double())
    weight = torch.where(ordered == float("-inf"), 0.0, weight)
    valid = (ordered > float("-inf")).sum(1, keepdim=True)
    n = torch.where(top_k > 0, torch.minimum(top_k, valid), valid)
    sums = weight.cumsum(1)
    whole = sums.gather(1, n - 1)
    n_p = (sums < top_p * whole).sum(1, keepdim=True) + 1
    n = torch.where(top_p < 1, torch.minimum(n, n_p), n)
    n_m = (weight >= min_p).sum(1, keepdim=True)
    n = torch.where(min_p > 0, torch.minimum(n, n_m), n)
    n = torch.where(t > 0, n, torch.ones_like(n))
    kept = torch.zeros_like(weight).scatter_(1, order, torch.where(rank < n, weight, 0.0))
    sums = kept.cumsum(1)
    token = (sums <= s["random"].double().unsqueeze(1) * sums[:, -1:]).sum(1, keepdim=True).clamp(max=vocab - 1)
    probs = kept.gather(1, token) / sums[:, -1:]
    return [token.squeeze(1).int(), n.squeeze(1).int(), probs.squeeze(1).float()]


_PLAIN = dict(prompt=_plain_prompt, decode=_plain_decode, q_decode=_plain_decode, q_write=_plain_q_write,
              sample=_plain_sample)


# ------------------------------------------------------------------ work
def _seen(position, window, sinks):
    """How many keys the query at a position sees."""
    n = position + 1
    return n if not window or n <= window else window + min(sinks, n - window)


def work(case):
    op = case["op"]
    if op == "sample":
        size = 4 if case["dtype"] == FP32 else 2
        return dict(bytes=case["rows"] * (case["vocab"] * size + 28), flops=0)
    lens, hd = _lengths(case), case["hd"]
    if op == "prompt":
        hq, hkv, w, prefix = case["hq"], case["hkv"], case["window"], case["prefix"]
        pairs = sum(_seen(prefix + i, w, case["sinks"]) for n in lens for i in range(n))
        keys = sum(min(n + prefix, n + w - 1 + case["sinks"]) for n in lens)
        return dict(bytes=2 * hd * (2 * hq * sum(lens) + 2 * hkv * keys), flops=4 * hq * hd * pairs)
    page, hkv = case["page"], case["hkv"]
    if op in ("decode", "q_decode"):
        keys = sum(_seen(n - 1, case["window"], case["sinks"]) if n else 0 for n in lens)
        size = 2 * hkv * hd * (2 if op == "decode" else 1)
        if op == "q_decode":
            size += 2 * hkv * 4 / case["block"]
        entries = sum(_ceil(n, page) if not case["window"] else
                      min(_ceil(n, page), _ceil(case["window"], page) + _ceil(case["sinks"], page)) for n in lens)
        return dict(bytes=2 * hd * 2 * case["hq"] * len(lens) + size * keys + 4 * entries,
                    flops=4 * case["hq"] * hd * keys)
    news = [case["new"] or n for n in lens]
    base = [n if case["new"] else 0 for n in lens]
    fresh = sum(_ceil(b + n, page) - _ceil(b, page) for b, n in zip(base, news))
    blocks = sum(_ceil(n, case["block"]) for n in news)
    return dict(bytes=2 * hkv * hd * (2 + 1) * sum(news) + 2 * hkv * 4 * blocks + 4 * (2 * fresh + 2 * len(lens)), flops=0)


# ------------------------------------------------------------------ 64-bit definition
def exact(case, seed):
    op = case["op"]
    if op == "sample":
        return _exact_sample(case, seed)
    if op == "q_write":
        return _exact_write(case, seed)
    lens = _lengths(case)
    hq, hkv, hd, window, sinks = case["hq"], case["hkv"], case["hd"], case["window"], case["sinks"]
    group = hq // hkv
    if op == "prompt":
        pairs = sum(n * min(n + case["prefix"], 1024 + window + sinks if window else n + case["prefix"]) for n in lens)
        if 8 * pairs * hq * hd > 8e12:
            return None
    state = prepare(dict(case), seed)
    if op != "prompt":
        out = torch.zeros((len(lens), hq, hd), dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            kk = torch.empty((n, hkv, hd), dtype=torch.float64, device="cuda")
            vv = torch.empty_like(kk)
            for j in range(_ceil(n, case["page"])):
                p, at = int(state["table"][b, j]), j * case["page"]
                m = min(case["page"], n - at)
                for to, name in ((kk, "k"), (vv, "v")):
                    page = state[name][0][p, :, :m].double()
                    if op == "q_decode":
                        every = state[name + "s"][0][p].double().repeat_interleave(case["block"], 1)[:, :m]
                        page = page * every.unsqueeze(-1)
                    to[at:at + m] = page.transpose(0, 1)
            pos = torch.arange(n, device="cuda")
            hidden = (n - 1 - pos >= window) & (pos >= sinks) if window else pos < 0
            for h in range(hq):
                if n:
                    a = torch.mv(kk[:, h // group], state["q"][b, h].double()) / math.sqrt(hd)
                    a[hidden] = -math.inf
                    a = torch.exp(a - a.max())
                    out[b, h] = torch.mv(vv[:, h // group].T, a) / a.sum()
        return out
    out = torch.zeros((sum(lens), hq, hd), dtype=torch.float64, device="cuda")
    row = at = 0
    for n in lens:
        nk = n + case["prefix"]
        kk, vv = state["k"][at:at + nk], state["v"][at:at + nk]
        at += nk
        for i0 in range(0, n, 1024):
            i1 = min(n, i0 + 1024)
            qpos = torch.arange(i0, i1, device="cuda") + (nk - n)
            end = i1 + nk - n
            kpos = torch.arange(end, device="cuda")
            if window:  # those that some query of the slice sees
                kpos = kpos[(kpos < sinks) | (kpos > int(qpos[0]) - window)]
            gap = qpos[:, None] - kpos[None, :]
            hidden = gap < 0
            if window:
                hidden |= (gap >= window) & (kpos >= sinks)[None, :]
            for h in range(hq):
                weight = torch.einsum("id,jd->ij", state["q"][row + i0:row + i1, h].double(),
                                      kk[kpos, h // group].double()) / math.sqrt(hd)
                weight[hidden] = -math.inf
                weight = torch.softmax(weight, 1)
                out[row + i0:row + i1, h] = torch.einsum("ij,jd->id", weight, vv[kpos, h // group].double())
        row += n
    return out


def _exact_e4m3(v):
    """The nearest e4m3 value, ties to an even last bit: steps of 2^(e - 3), e >= -6."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _exact_write(case, seed):
    """A block of rows at a time: the values held, and their scales."""
    lens = _lengths(case)
    if sum(case["new"] or n for n in lens) > 20000:
        return None
    state = prepare(dict(case), seed)
    page, block, hkv = case["page"], case["block"], case["hkv"]
    news = [case["new"] or n for n in lens]
    base = [n if case["new"] else 0 for n in lens]
    table, refs = state["table"].tolist(), state["refs"].tolist()
    free = [p for p, r in enumerate(refs) if r == 0]
    held = [state["k"][0].double(), state["v"][0].double()]
    scales = [state["ks"][0].double(), state["vs"][0].double()]
    given = [state["new_k"].double(), state["new_v"].double()]
    at = 0
    for s, (b, n) in enumerate(zip(base, news)):
        for j in range(_ceil(b, page), _ceil(b + n, page)):
            table[s][j] = free.pop(0)
        pos = b
        while pos < b + n:
            r = pos % page
            first = r - r % block                              # the block's first row
            last = min(r + b + n - pos, first + block, page)   # and the end of its new ones
            p = table[s][pos // page]
            for pool, sc, new in zip(held, scales, given):
                x = new[at:at + last - r].transpose(0, 1)
                most = x.abs().amax((1, 2))
                need = torch.exp2(torch.ceil(torch.log2(most / _TOP)).clamp(min=-126.0))
                was = sc[p, :, first // block] if r > first else torch.zeros_like(need)
                now = torch.maximum(torch.where(most > 0, need, 0.0), was)
                some = torch.where(now > 0, now, 1.0).view(hkv, 1, 1)
                if r > first:
                    pool[p, :, first:r] = _exact_e4m3(pool[p, :, first:r] * (was.view(hkv, 1, 1) / some))
                pool[p, :, r:last] = _exact_e4m3(x / some)
                sc[p, :, first // block] = now
            at += last - r
            pos += last - r
    return [None, None, None, held[0], held[1], scales[0], scales[1]]


def _exact_sample(case, seed):
    """A row at a time: the tokens in their order, added up until each limit is met."""
    state = prepare(dict(case), seed)
    tokens, counts, probs = [], [], []
    for i in range(case["rows"]):
        x = state["logits"][i].double()
        t = float(state["temperature"][i])
        k = int(state["top_k"][i]) if state["top_k"] is not None else 0
        p = float(state["top_p"][i]) if state["top_p"] is not None else 1.0
        m = float(state["min_p"][i]) if state["min_p"] is not None else 0.0
        order = torch.argsort(-x, stable=True)
        order = order[x[order] > -math.inf]
        if t <= 0:
            order = order[:1]
        if k > 0:
            order = order[:k]
        weight = torch.exp((x[order] - x[order[0]]) / (t if t > 0 else 1.0))
        n = len(order)
        if p < 1:
            run_ = torch.cumsum(weight, 0)
            n = min(n, 1 + int(torch.searchsorted(run_, p * run_[-1], right=False)))
        if m > 0:
            n = min(n, int(torch.count_nonzero(weight >= m)))
        mine, order_ = torch.sort(order[:n])
        share = weight[:n][order_] / weight[:n].sum()
        at = int(torch.searchsorted(torch.cumsum(share, 0), float(state["random"][i]), right=True))
        at = min(at, n - 1)
        tokens.append(int(mine[at]))
        counts.append(n)
        probs.append(float(share[at]))
    return [torch.tensor(tokens, dtype=torch.int32), torch.tensor(counts, dtype=torch.int32),
            torch.tensor(probs, dtype=torch.float64)]
