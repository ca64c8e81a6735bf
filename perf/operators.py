"""Measured cases of the paged KV cache and of the attention that reads it.

Five operators, each in the form a serving loop calls it:

  prompt   causal attention of whole prompts, packed, grouped heads, optional window
  decode   attention of one new token per sequence over the paged cache
  write    reserving the pages of new tokens and storing their K/V rows
  fork     giving sequences the pages of others, then one more token each (the last,
           partly filled page is copied because it is shared)
  compact  moving the pages in use to the front of the pool

``own`` selects the framework's calls; without it ``run`` computes the same results with
elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

BF16, FP16 = "bf16", "fp16"
_DTYPES = {BF16: torch.bfloat16, FP16: torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a first, short chat turn on the smallest head layout: latency
        dict(name="prompt_short", op="prompt", dtype=BF16, hq=8, hkv=2, hd=64, seqs=1, shortest=17, longest=17,
             lens=1, prefix=0, window=128, in_cache=False),
        # a batch of turns that continue conversations whose K/V rows stand in contiguous caches,
        # on a sliding-window layer
        dict(name="prompt_resume", op="prompt", dtype=FP16, hq=32, hkv=8, hd=128, seqs=12, shortest=3, longest=1500,
             lens=2, prefix=2500, window=2048, in_cache=True),
        # one long document on a global layer
        dict(name="prompt_long", op="prompt", dtype=BF16, hq=32, hkv=8, hd=128, seqs=1, shortest=16384, longest=16384,
             lens=3, prefix=0, window=0, in_cache=False),
        # one user, a short history: latency
        dict(name="decode_one", op="decode", dtype=BF16, hq=8, hkv=2, hd=64, seqs=1, shortest=200, longest=200, lens=4,
             page=16, window=0),
        # a batch of ragged conversations on a global layer
        dict(name="decode_batch", op="decode", dtype=BF16, hq=32, hkv=8, hd=128, seqs=64, shortest=1, longest=8192,
             lens=5, page=64, window=0),
        # one very long context: the split over its length carries the work
        dict(name="decode_long", op="decode", dtype=FP16, hq=32, hkv=8, hd=128, seqs=1, shortest=131071,
             longest=131071, lens=6, page=48, window=0),
        # one 16-token tree per sequence, on rows that the last step's tree had
        dict(name="write_step", op="write", dtype=BF16, hkv=8, hd=128, seqs=32, shortest=100, longest=8000, lens=7,
             page=64, new=16),
        # the K/V rows of a packed batch of prompts
        dict(name="write_prompt", op="write", dtype=BF16, hkv=8, hd=128, seqs=16, shortest=1, longest=8192, lens=8,
             page=64, new=0),
        # one prompt continued four ways
        dict(name="fork_beam", op="fork", dtype=BF16, hkv=8, hd=128, seqs=1, copies=3, shortest=1234, longest=1234,
             lens=9, page=16, layers=5),
        # a batch of prompts sampled four times each
        dict(name="fork_batch", op="fork", dtype=BF16, hkv=8, hd=128, seqs=64, copies=3, shortest=20, longest=4000,
             lens=10, page=64, layers=8),
        # a small pool after a few sequences ended
        dict(name="compact_small", op="compact", dtype=BF16, hkv=2, hd=64, seqs=8, shortest=10, longest=300, lens=11,
             page=16, layers=4, ended=2),
        # a large pool of which half the sequences ended
        dict(name="compact_large", op="compact", dtype=BF16, hkv=8, hd=128, seqs=48, shortest=50, longest=4096,
             lens=12, page=64, layers=6, ended=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "write", "fork", "compact"])
    dtype = rng.choice([BF16, FP16])
    hd = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 16, 32, 64, 128, rng.randint(1, 200)])
    lens = rng.randrange(1 << 30)
    if op == "prompt":
        longest = _log(rng, 1, 8192)
        seqs = _log(rng, 1, max(1, min(64, 16384 // longest)))
        return dict(op=op, dtype=dtype, hq=hq, hkv=hkv, hd=hd, seqs=seqs, shortest=rng.randint(1, longest),
                    longest=longest, lens=lens, prefix=rng.choice([0, 0, _log(rng, 1, 4000)]),
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), in_cache=rng.random() < 0.3)
    if op == "decode":
        longest = _log(rng, 1, 65536)
        seqs = _log(rng, 1, max(1, min(256, 262144 // longest)))
        return dict(op=op, dtype=dtype, hq=hq, hkv=hkv, hd=hd, seqs=seqs, shortest=rng.randint(0, longest),
                    longest=longest, lens=lens, page=page, window=rng.choice([0, 0, _log(rng, 1, 4096)]))
    page = max(page, 4)
    if op == "write":
        longest = _log(rng, 1, 8192)
        new = rng.choice([0, 1, rng.randint(1, 64)])
        return dict(op=op, dtype=dtype, hkv=hkv, hd=hd, seqs=_log(rng, 1, max(1, min(128, 65536 // longest))),
                    shortest=rng.randint(1, longest), longest=longest, lens=lens, page=page, new=new)
    longest = _log(rng, 10, 4096)
    seqs = _log(rng, 2, max(2, min(64, 65536 // longest)))
    case = dict(op=op, dtype=dtype, hkv=hkv, hd=hd, seqs=seqs, shortest=rng.randint(1, longest), longest=longest,
                lens=lens, page=page, layers=rng.randint(1, 6))
    if op == "fork":
        case["copies"] = rng.randint(1, 4)
    else:
        case["ended"] = rng.randint(2, 4)
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


def _pool(case, gen, layers, n_pages):
    shape = (n_pages, case["hkv"], case["page"], case["hd"])
    t = _DTYPES[case["dtype"]]
    return [_normal(gen, shape, t) for _ in range(layers)], [_normal(gen, shape, t) for _ in range(layers)]


def _tables(state, rng, lens, slots, max_pages, n_pages, page):
    """A table of the pages of `lens` (taken from the pool in a random order), its lengths and
    the pages' reference counts, in one buffer."""
    order = list(range(n_pages))
    rng.shuffle(order)
    table = [[-1] * max_pages for _ in range(slots)]
    refs = [0] * n_pages
    full = list(lens) + [0] * (slots - len(lens))
    at = 0
    for s, n in enumerate(full):
        for j in range(_ceil(n, page)):
            table[s][j] = order[at]
            refs[order[at]] = 1
            at += 1
    _set_tables(state, table, full, refs)
    return table, full, refs


def _set_tables(state, table, lens, refs):
    slots, max_pages = len(table), len(table[0])
    flat = [p for row in table for p in row] + lens + refs
    state["meta"] = _ints(flat)
    state["saved"] = state["meta"].clone()
    a, b = slots * max_pages, slots * max_pages + slots
    state["table"] = state["meta"][:a].view(slots, max_pages)
    state["lens"] = state["meta"][a:b]
    state["refs"] = state["meta"][b:]


def _handle(state):
    """The cache object a user's program keeps."""
    if own:
        from moe_decode_megakernel_warp_gb300 import PagedCache
        state["cache"] = PagedCache(state["k"], state["v"], state["table"], state["lens"], state["refs"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    t = _DTYPES[case["dtype"]]
    lens = _lengths(case)
    state = dict(case=case)
    op = case["op"]
    if op == "prompt":
        hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
        klens = [n + case["prefix"] for n in lens]
        cu_q, cu_k = _cu(lens), _cu(klens)
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
    pages = [_ceil(n, page) for n in lens]
    if op == "decode":
        n_pages = max(1, sum(pages) + max(1, sum(pages) // 16))
        state["k"], state["v"] = _pool(case, gen, 1, n_pages)
        _tables(state, rng, lens, len(lens), max(1, max(pages)), n_pages, page)
        state["host_lens"] = lens
        state["q"] = _normal(gen, (len(lens), case["hq"], case["hd"]), t)
    elif op == "write":
        # `new` tokens behind each history, or the whole prompts
        news = [case["new"] or n for n in lens]
        base = [n if case["new"] else 0 for n in lens]
        after = [b + n for b, n in zip(base, news)]
        n_pages = sum(_ceil(n, page) for n in after) + 8
        state["k"], state["v"] = _pool(case, gen, 1, n_pages)
        _tables(state, rng, base, len(lens), max(_ceil(n, page) for n in after), n_pages, page)
        cu = _cu(news)
        state.update(starts=_ints(cu), cu=cu, target=_ints(after), host_after=after)
        kv = _normal(gen, (cu[-1], 2 * case["hkv"], case["hd"]), t)
        state.update(new_k=kv[:, :case["hkv"]], new_v=kv[:, case["hkv"]:])
    elif op == "fork":
        n, copies = len(lens), case["copies"]
        slots = n * (1 + copies)
        n_pages = sum(pages) + slots + 8
        state["k"], state["v"] = _pool(case, gen, case["layers"], n_pages)
        _tables(state, rng, lens, slots, max(_ceil(x + 1, page) for x in lens), n_pages, page)
        state["parent"] = _ints([-1] * n + [s % n for s in range(n * copies)])
        state["target"] = _ints([lens[s % n] + 1 for s in range(slots)])
    else:
        n_pages = sum(pages) + 8
        state["k"], state["v"] = _pool(case, gen, case["layers"], n_pages)
        table, full, refs = _tables(state, rng, lens, len(lens), max(pages), n_pages, page)
        for s in range(len(lens)):
            if s % case["ended"] == 0:
                for j in range(pages[s]):
                    refs[table[s][j]] = 0
                    table[s][j] = -1
                full[s] = 0
        _set_tables(state, table, full, refs)
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
    return prompt_attention(s["q"], s["k"], s["v"], s["q_starts"], s["k_starts"], window=s["case"]["window"])


def _own_decode(s):
    return s["cache"].attention(0, s["q"], window=s["case"]["window"])


# The calls below change the tables.  Each pass begins from the same ones, as a program that
# goes back to a saved point does, so that every pass does the same work.
def _own_write(s):
    s["meta"].copy_(s["saved"])
    s["cache"].resize(s["target"])
    s["cache"].write(0, s["new_k"], s["new_v"], s["starts"])
    return [s["table"], s["lens"], s["refs"], s["k"][0], s["v"][0]]


def _own_fork(s):
    s["meta"].copy_(s["saved"])
    s["cache"].fork(s["parent"])
    s["cache"].resize(s["target"])
    return [s["table"], s["lens"], s["refs"]] + s["k"] + s["v"]


def _own_compact(s):
    s["meta"].copy_(s["saved"])
    s["cache"].compact()
    return [s["table"], s["lens"], s["refs"]] + s["k"] + s["v"]


_OWN = dict(prompt=_own_prompt, decode=_own_decode, write=_own_write, fork=_own_fork, compact=_own_compact)


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
    hq, hkv, hd, window = c["hq"], c["hkv"], c["hd"], c["window"]
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
            q = s["q"][q0 + i0:q0 + i1].float().view(i1 - i0, hkv, group, hd).permute(1, 2, 0, 3)
            k = s["k"][k0 + lo:k0 + hi].float().transpose(0, 1).unsqueeze(1)
            v = s["v"][k0 + lo:k0 + hi].float().transpose(0, 1).unsqueeze(1)
            scores = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(hd))
            i = torch.arange(i0, i1, device="cuda").unsqueeze(1) + shift
            j = torch.arange(lo, hi, device="cuda").unsqueeze(0)
            seen = (j <= i) & (i - j < window) if window else j <= i
            o = _softmax_times(scores, seen, v)
            out[q0 + i0:q0 + i1] = o.permute(2, 0, 1, 3).reshape(i1 - i0, hq, hd).to(out.dtype)
    return out


def _plain_decode(s):
    c = s["case"]
    hq, hkv, hd, page, window = c["hq"], c["hkv"], c["hd"], c["page"], c["window"]
    out = torch.zeros_like(s["q"])
    for b, n in enumerate(s["host_lens"]):
        if n == 0:
            continue
        first = max(0, n - window) if window else 0
        p0, p1 = first // page, _ceil(n, page)
        ids = s["table"][b, p0:p1].long()
        k = s["k"][0][ids].transpose(0, 1).reshape(hkv, -1, hd)[:, first - p0 * page:n - p0 * page].float()
        v = s["v"][0][ids].transpose(0, 1).reshape(hkv, -1, hd)[:, first - p0 * page:n - p0 * page].float()
        q = s["q"][b].float().view(hkv, hq // hkv, hd)
        scores = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(hd))
        out[b] = _softmax_times(scores, torch.ones_like(scores, dtype=torch.bool), v).view(hq, hd).to(out.dtype)
    return out


def _plain_resize(s, target):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["case"]["page"]
    old = lens.long()
    new = torch.where(target < 0, old, target.long())
    n_old, n_new = (old + page - 1) // page, (new + page - 1) // page
    j = torch.arange(table.shape[1], device="cuda").unsqueeze(0)
    last = (old // page).clamp(max=table.shape[1] - 1).unsqueeze(1)
    shared = refs[table.gather(1, last).squeeze(1).clamp(min=0).long()] > 1
    cow = (new > old) & (old % page != 0) & shared
    want = ((j >= n_old.unsqueeze(1)) & (j < n_new.unsqueeze(1))) | (cow.unsqueeze(1) & (j == last))
    drop = ((j >= n_new.unsqueeze(1)) & (j < n_old.unsqueeze(1))) | (cow.unsqueeze(1) & (j == last))
    index = torch.arange(refs.numel(), device="cuda")
    free = torch.sort(torch.where(refs == 0, index, index + refs.numel())).values
    rank = (torch.cumsum(want.reshape(-1).long(), 0) - 1).clamp(min=0).view_as(want)
    taken = free[rank] % refs.numel()
    src = table.gather(1, last).squeeze(1)[cow].long()
    dst = taken.gather(1, last).squeeze(1)[cow]
    rows = (old % page)[cow]
    refs.index_add_(0, table.clamp(min=0).reshape(-1).long(), -drop.reshape(-1).int())
    refs.index_add_(0, taken.reshape(-1), want.reshape(-1).int())
    keep = torch.where(j < n_new.unsqueeze(1), table, torch.full_like(table, -1))
    table.copy_(torch.where(want, taken.int(), keep))
    lens.copy_(new.int())
    r = torch.arange(page, device="cuda").view(1, 1, page, 1) < rows.view(-1, 1, 1, 1)
    for pool in s["k"] + s["v"]:
        pool[dst] = torch.where(r, pool[src], pool[dst])


def _plain_write(s):
    s["meta"].copy_(s["saved"])
    _plain_resize(s, s["target"])
    cu, page = s["cu"], s["case"]["page"]
    counts = s["starts"].diff().long()
    seq = torch.repeat_interleave(torch.arange(len(cu) - 1, device="cuda"), counts, output_size=cu[-1])
    pos = torch.arange(cu[-1], device="cuda") - s["starts"].long()[seq] + (s["lens"].long() - counts)[seq]
    ids = s["table"][seq, pos // page].long()
    s["k"][0][ids, :, pos % page] = s["new_k"]
    s["v"][0][ids, :, pos % page] = s["new_v"]
    return [s["table"], s["lens"], s["refs"], s["k"][0], s["v"][0]]


def _plain_fork(s):
    s["meta"].copy_(s["saved"])
    table, lens, refs = s["table"], s["lens"], s["refs"]
    has = s["parent"] >= 0
    p = s["parent"].clamp(min=0).long()
    table.copy_(torch.where(has.unsqueeze(1), table[p], table))
    lens.copy_(torch.where(has, lens[p], lens))
    used = has.unsqueeze(1) & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).reshape(-1).long(), used.reshape(-1).int())
    _plain_resize(s, s["target"])
    return [table, lens, refs] + s["k"] + s["v"]


def _plain_compact(s):
    s["meta"].copy_(s["saved"])
    table, refs = s["table"], s["refs"]
    live = refs > 0
    index = torch.arange(refs.numel(), device="cuda")
    front = index < live.sum()
    src, dst = index[live & ~front], index[~live & front]
    to = index.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    refs[dst] = refs[src]
    refs[src] = 0
    for pool in s["k"] + s["v"]:
        pool[dst] = pool[src]
    return [table, s["lens"], refs] + s["k"] + s["v"]


_PLAIN = dict(prompt=_plain_prompt, decode=_plain_decode, write=_plain_write, fork=_plain_fork,
              compact=_plain_compact)


# ------------------------------------------------------------------ work
def _seen_pairs(nq, nk, window):
    """Query-key pairs of one sequence under the causal mask and the window."""
    shift = nk - nq
    total = 0
    for a, b in ((0, 0), (window, 1)) if window else ((0, 0),):
        # sum over i of max(0, i + shift + 1 - a): all keys up to i, less those before the window
        lo = max(0, a - shift)
        n = max(0, nq - lo)
        s = n * (shift + 1 - a) + (lo + nq - 1) * n // 2
        total += -s if b else s
    return total


def work(case):
    lens, el = _lengths(case), 2
    op, hd = case["op"], case["hd"]
    if op == "prompt":
        hq, hkv = case["hq"], case["hkv"]
        pairs = sum(_seen_pairs(n, n + case["prefix"], case["window"]) for n in lens)
        keys = sum(min(n + case["prefix"], n + case["window"] - 1) if case["window"] else n + case["prefix"]
                   for n in lens)
        return dict(bytes=el * hd * (2 * hq * sum(lens) + 2 * hkv * keys), flops=4 * hq * hd * pairs)
    page = case["page"]
    if op == "decode":
        keys = sum(min(n, case["window"]) if case["window"] else n for n in lens)
        entries = sum(_ceil(n, page) for n in lens)
        return dict(bytes=el * hd * (2 * case["hq"] * len(lens) + 2 * case["hkv"] * keys) + 4 * entries,
                    flops=4 * case["hq"] * hd * keys)
    row = 2 * case["hkv"] * hd * el  # K and V of one token and layer
    if op == "write":
        news = [case["new"] or n for n in lens]
        base = [n if case["new"] else 0 for n in lens]
        fresh = sum(_ceil(b + n, page) - _ceil(b, page) for b, n in zip(base, news))
        return dict(bytes=2 * row * sum(news) + 4 * (2 * fresh + 2 * len(lens)), flops=0)
    if op == "fork":
        group = 1 + case["copies"]
        # each of a group that ends inside its shared page gets a copy of the rows there
        rows = sum(n % page for n in lens)
        entries = sum(_ceil(n, page) for n in lens)
        return dict(bytes=(1 + group) * row * case["layers"] * rows + 4 * (2 + case["copies"]) * 2 * entries, flops=0)
    # which pages move depends on their order in the pool: of the pages in use, the share that
    # stands behind the front, on average that of the free pages
    pages = [_ceil(n, page) for n in lens]
    used = sum(p for s, p in enumerate(pages) if s % case["ended"])
    total = sum(pages) + 8
    moved = used * (total - used) // total
    return dict(bytes=2 * row * case["layers"] * page * moved + 4 * 2 * (total + used), flops=0)


# ------------------------------------------------------------------ 64-bit definition
def exact(case, seed):
    if case["op"] not in ("prompt", "decode"):
        return None
    lens = _lengths(case)
    hq, hkv, hd, window = case["hq"], case["hkv"], case["hd"], case["window"]
    prefix = case.get("prefix", 0)
    pairs = sum(_seen_pairs(n, n + prefix, 0) for n in lens) if case["op"] == "prompt" else sum(lens)
    if 8 * pairs * hq * hd > 8e12:
        return None
    state = prepare(dict(case), seed)
    group = hq // hkv
    out = torch.zeros((sum(lens) if case["op"] == "prompt" else len(lens), hq, hd), dtype=torch.float64, device="cuda")
    row = at = 0
    for b, n in enumerate(lens):
        if case["op"] == "prompt":
            nk, queries = n + prefix, n
            kk, vv = state["k"][at:at + nk], state["v"][at:at + nk]
            at += nk
        else:
            nk, queries = n, 1
            pos = torch.arange(n, device="cuda")
            ids = state["table"][b].long()[pos // case["page"]]
            kk = state["k"][0][ids, :, pos % case["page"]]
            vv = state["v"][0][ids, :, pos % case["page"]]
        for i0 in range(0, queries, 1024):
            i1 = min(queries, i0 + 1024)
            qpos = torch.arange(i0, i1, device="cuda") + (nk - queries)
            end = max(0, i1 + nk - queries)
            for h in range(hq):
                scores = torch.einsum("id,jd->ij", state["q"][row + i0:row + i1, h].double(),
                                      kk[:end, h // group].double()) / math.sqrt(hd)
                kpos = torch.arange(end, device="cuda")
                gap = qpos[:, None] - kpos[None, :]
                hidden = gap < 0
                if window:
                    hidden |= gap >= window
                weight = torch.exp(scores - torch.max(scores.masked_fill(hidden, -1e30), 1, keepdim=True).values
                                   if end else scores)
                weight[hidden] = 0
                norm = weight.sum(1, keepdim=True)
                norm[norm == 0] = 1
                out[row + i0:row + i1, h] = torch.einsum("ij,jd->id", weight / norm, vv[:end, h // group].double())
        row += queries
    return out
