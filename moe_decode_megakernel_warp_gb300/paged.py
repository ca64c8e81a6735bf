"""Torch-facing wrappers of the paged KV cache and of the prompt attention (msm.h).

Argument marshalling only, like ``Model``: the work runs in the kernels of ``libmsm.so``.
The calls run on torch's current stream of the tensors' device, so ``torch.cuda.stream``
and graph capture apply to them.  What torch can tell about a tensor (its type, shape,
device, memory order) is checked here and raises ``ValueError``; everything else is checked
by the library and raises ``MsmError``.
"""
from __future__ import annotations

import ctypes
import math

from . import MSM_BF16, MSM_FP16, MsmPages, MsmPrompt, _check, _ptr_array, lib

_DTYPES = None


def _torch():
    global _DTYPES
    import torch
    if _DTYPES is None:
        _DTYPES = {torch.bfloat16: MSM_BF16, torch.float16: MSM_FP16}
    return torch


def _need(ok, msg):
    if not ok:
        raise ValueError(msg)


def _dtype(t):
    _torch()
    _need(t.dtype in _DTYPES, "expected bfloat16 or float16, got %s" % t.dtype)
    return _DTYPES[t.dtype]


def _rows(t, name, heads, head_dim, like):
    """(first, second) strides of a [n][heads][head_dim] tensor; a dimension of one element
    has no stride of its own."""
    _need(t.dim() == 3 and (heads is None or t.shape[1] == heads) and t.shape[2] == head_dim,
          "%s must be [n, %s, %d], got %s" % (name, "heads" if heads is None else heads, head_dim, tuple(t.shape)))
    _need(t.dtype == like.dtype and t.device == like.device, "%s must have the type and device of the others" % name)
    _need(t.stride(2) == 1, "%s: the elements of a row must be consecutive" % name)
    n0, n1, _ = t.shape
    return (t.stride(0) if n0 > 1 else n1 * head_dim), (t.stride(1) if n1 > 1 else head_dim)


def _int32(t, name, n, device):
    torch = _torch()
    _need(t.dtype == torch.int32 and t.is_contiguous() and t.device == device and (n is None or t.numel() == n),
          "%s must be a contiguous int32 tensor%s on %s" % (name, "" if n is None else " of %d entries" % n, device))
    return t.data_ptr()


def _stream(device):
    return _torch().cuda.current_stream(device).cuda_stream


class PagedCache:
    """A paged KV cache over the caller's tensors: ``k_pages`` and ``v_pages`` are lists of one
    [n_pages, n_kv_heads, page_rows, head_dim] tensor per layer (bfloat16 or float16),
    ``table`` int32 [n_seqs, max_pages] (-1 behind a sequence's last page), ``lens`` int32
    [n_seqs], ``refs`` int32 [n_pages].  ``PagedCache.allocate`` makes an empty one.

    ``resize``, ``fork``, ``compact`` and ``write`` change these tensors on the device, in
    stream order and without a host round trip; ``sync`` waits and raises what they met."""

    def __init__(self, k_pages, v_pages, table, lens, refs):
        torch = _torch()
        k_pages, v_pages = list(k_pages), list(v_pages)
        _need(len(k_pages) == len(v_pages) and k_pages, "one K and one V pool per layer")
        first = k_pages[0]
        _need(first.is_cuda, "the pools must be CUDA tensors")
        _need(first.dim() == 4, "a pool is [n_pages, n_kv_heads, page_rows, head_dim]")
        for t in k_pages + v_pages:
            _need(t.shape == first.shape and t.dtype == first.dtype and t.device == first.device and t.is_contiguous(),
                  "the pools must be contiguous and alike in shape, type and device")
        _need(table.dim() == 2, "table is [n_seqs, max_pages]")
        n_pages, n_kv_heads, page_rows, head_dim = first.shape
        n_seqs, max_pages = table.shape
        dev = first.device
        self.k_pages, self.v_pages, self.table, self.lens, self.refs = k_pages, v_pages, table, lens, refs
        self.device = dev
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.scratch = torch.empty(max(1, lib().msm_pages_scratch_ints(n_pages, n_seqs)), dtype=torch.int32,
                                   device=dev)
        kp, self._k_ptrs = _ptr_array([t.data_ptr() for t in k_pages])
        vp, self._v_ptrs = _ptr_array([t.data_ptr() for t in v_pages])
        self._c = MsmPages(dev.index, _dtype(first), len(k_pages), n_pages, page_rows, n_kv_heads, head_dim, n_seqs,
                           max_pages, kp, vp, _int32(table, "table", None, dev), _int32(lens, "lens", n_seqs, dev),
                           _int32(refs, "refs", n_pages, dev), self.status.data_ptr(), self.scratch.data_ptr())
        self._ref = ctypes.byref(self._c)
        self._workspace = {}  # bytes by number of query heads

    @classmethod
    def allocate(cls, n_layers, n_pages, page_rows, n_kv_heads, head_dim, n_seqs, max_pages, dtype=None, device=None):
        """An empty cache (bfloat16 by default)."""
        torch = _torch()
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)

        def pools():
            return [torch.zeros((n_pages, n_kv_heads, page_rows, head_dim), dtype=dtype or torch.bfloat16, device=dev)
                    for _ in range(n_layers)]

        def ints(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=dev)
        return cls(pools(), pools(), ints(n_seqs, max_pages).fill_(-1), ints(n_seqs), ints(n_pages))

    def resize(self, new_lens):
        """msm_pages_resize: int32 [n_seqs] on the device, -1 = leave as it is."""
        _check(lib().msm_pages_resize(self._ref, _int32(new_lens, "new_lens", self._c.n_seqs, self.device),
                                      _stream(self.device)))

    def fork(self, parent):
        """msm_pages_fork: int32 [n_seqs] on the device, -1 = none."""
        _check(lib().msm_pages_fork(self._ref, _int32(parent, "parent", self._c.n_seqs, self.device),
                                    _stream(self.device)))

    def compact(self):
        """msm_pages_compact."""
        _check(lib().msm_pages_compact(self._ref, _stream(self.device)))

    def write(self, layer, k, v, starts):
        """msm_pages_write: k, v [n_tokens, n_kv_heads, head_dim], starts int32 [n_seqs + 1]."""
        c, like = self._c, self.k_pages[0]
        kt, kh = _rows(k, "k", c.n_kv_heads, c.head_dim, like)
        vt, vh = _rows(v, "v", c.n_kv_heads, c.head_dim, like)
        _need(k.shape[0] == v.shape[0], "k and v must have as many tokens")
        _check(lib().msm_pages_write(self._ref, layer, k.data_ptr(), v.data_ptr(), kt, kh, vt, vh,
                                     _int32(starts, "starts", c.n_seqs + 1, self.device), k.shape[0],
                                     _stream(self.device)))

    def attention(self, layer, q, window=0, scale=None, out=None):
        """msm_paged_attention: q [n_seqs, n_q_heads, head_dim]; scale defaults to
        1 / sqrt(head_dim).  Returns out."""
        torch = _torch()
        c = self._c
        qs, qh = _rows(q, "q", None, c.head_dim, self.k_pages[0])
        _need(q.shape[0] == c.n_seqs, "q must have one row per sequence of the table (%d)" % c.n_seqs)
        heads = q.shape[1]
        if out is None:
            out = torch.empty((c.n_seqs, heads, c.head_dim), dtype=q.dtype, device=self.device)
        os_, oh = _rows(out, "out", heads, c.head_dim, q)
        _need(out.shape[0] == c.n_seqs, "out must have the shape of q")
        n = self._workspace.get(heads)
        if n is None:
            n = lib().msm_paged_attention_workspace(self._ref, heads)
            _check(0 if n else lib().msm_paged_attention(self._ref, layer, None, qs, qh, heads, 1.0, 0, None, os_, oh,
                                                         None, 0, None))
            self._workspace[heads] = n
        # taken from torch's allocator for every call: memory of the stream (or of the graph
        # that records the call), so calls on different streams do not share it
        ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        _check(lib().msm_paged_attention(self._ref, layer, q.data_ptr(), qs, qh, heads,
                                         1.0 / math.sqrt(c.head_dim) if scale is None else scale, window,
                                         out.data_ptr(), os_, oh, ws.data_ptr(), n, _stream(self.device)))
        return out

    def sync(self):
        """msm_pages_sync: waits for the current stream; raises MsmError for an error that a
        call met on the device (and clears it)."""
        _check(lib().msm_pages_sync(self._ref, _stream(self.device)))


def prompt_attention(q, k, v, q_starts, k_starts=None, window=0, scale=None, out=None):
    """msm_prompt_attention: causal attention of packed prompts.

    q [n_q, n_q_heads, head_dim], k and v [n_k, n_kv_heads, head_dim] (any strides that keep
    rows consecutive; ``cache.transpose(0, 1)`` of a verify-step cache [n_kv_heads, max_ctx,
    head_dim] is read in place), q_starts and k_starts int32 [n_seqs + 1] on the device
    (k_starts defaults to q_starts), scale defaults to 1 / sqrt(head_dim).  Returns out; a new
    one is uninitialised behind the last sequence."""
    torch = _torch()
    _need(q.is_cuda, "q must be a CUDA tensor")
    _need(q.dim() == 3 and k.dim() == 3, "q and k must be [tokens, heads, head_dim]")
    n_q, heads, hd = q.shape
    n_k, kv_heads, _ = k.shape
    _need(v.shape == k.shape, "v must have the shape of k")
    qt, qh = _rows(q, "q", heads, hd, q)
    kt, kh = _rows(k, "k", kv_heads, hd, q)
    vt, vh = _rows(v, "v", kv_heads, hd, q)
    if out is None:
        out = torch.empty((n_q, heads, hd), dtype=q.dtype, device=q.device)
    ot, oh = _rows(out, "out", heads, hd, q)
    _need(out.shape[0] == n_q, "out must have the shape of q")
    n_seqs = q_starts.numel() - 1
    qs = _int32(q_starts, "q_starts", None, q.device)
    ks = qs if k_starts is None else _int32(k_starts, "k_starts", n_seqs + 1, q.device)
    a = MsmPrompt(q.device.index, _dtype(q), n_seqs, n_q, n_k, heads, kv_heads, hd, window,
                  1.0 / math.sqrt(hd) if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                  out.data_ptr(), qt, qh, kt, kh, vt, vh, ot, oh, qs, ks)
    _check(lib().msm_prompt_attention(ctypes.byref(a), _stream(q.device)))
    return out
