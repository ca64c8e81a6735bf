"""Torch-facing wrappers of the paged KV cache and of the prompt attention (msm.h).

Argument marshalling only, like ``Model``: the work runs in the kernels of ``libmsm.so``.
The calls run on torch's current stream of the tensors' device, so ``torch.cuda.stream``
and graph capture apply to them.  What torch can tell about a tensor (its type, shape,
device, memory order) is checked here and raises ``ValueError``; everything else is checked
by the library and raises ``MsmError``.
"""
from __future__ import annotations

import ctypes
import struct

from . import MSM_BF16, MSM_FP16, MsmPages, MsmPrompt, _check, _ptr_array, lib

# msm_prompt in the C layout (a bytes object takes a third of the time of a ctypes structure)
_PROMPT = struct.Struct("9if4P8q3PI4x")
assert _PROMPT.size == ctypes.sizeof(MsmPrompt)


# Set at the first call: the torch module and what every call takes from it, the library, and
# msm_dtype by torch type.  (A small call is host time: 11 us for a short prompt's, of which the
# launch is 2.4.)
_torch = _empty = _raw_stream = _capturing = _INT32 = _LIBRARY = None
_CODES = {}


def _load():
    global _torch, _empty, _raw_stream, _capturing, _INT32, _LIBRARY
    import torch
    _LIBRARY = lib()
    _CODES.update({torch.bfloat16: MSM_BF16, torch.float16: MSM_FP16})
    _empty, _INT32 = torch.empty, torch.int32
    _raw_stream, _capturing = torch._C._cuda_getCurrentRawStream, torch._C._cuda_isCurrentStreamCapturing
    _torch = torch


def _need(ok, msg):
    if not ok:
        raise ValueError(msg)


def _rows(t, name, shape, dtype, index):
    """(first, second) strides of a tensor [n][heads][head_dim] of the given shape, type and
    CUDA device; a dimension of one element has no stride of its own."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise ValueError("%s must be %s, %s, on cuda:%d; got %s, %s, on %s"
                         % (name, list(shape), dtype, index, list(t.shape), t.dtype, t.device))
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError("%s: the elements of a row must be consecutive" % name)
    n0, n1, hd = shape
    return (s0 if n0 > 1 else n1 * hd), (s1 if n1 > 1 else hd)


def _int32(t, name, n, index):
    if t.dtype is not _INT32 or t.get_device() != index or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of %d entries on cuda:%d" % (name, n, index))
    return t.data_ptr()


def _c_int(x):
    """x as a C int that says the same: ctypes would take its low 32 bits (a window of 2^32 for none).
    Every index, and no window, is below the largest one; -1 is refused as any other negative number."""
    return -1 if x < 0 else x if x < 0x7FFFFFFF else 0x7FFFFFFF


class PagedCache:
    """A paged KV cache over the caller's tensors: ``k_pages`` and ``v_pages`` are lists of one
    [n_pages, n_kv_heads, page_rows, head_dim] tensor per layer (bfloat16 or float16),
    ``table`` int32 [n_seqs, max_pages] (-1 behind a sequence's last page), ``lens`` int32
    [n_seqs], ``refs`` int32 [n_pages].  ``PagedCache.allocate`` makes an empty one.

    ``resize``, ``fork``, ``compact`` and ``write`` change these tensors on the device, in
    stream order and without a host round trip; ``sync`` waits and raises what they met.  After a
    ``resize`` or ``fork`` that could not be done none of them changes anything until ``sync``."""

    def __init__(self, k_pages, v_pages, table, lens, refs):
        if _torch is None:
            _load()
        torch = _torch
        k_pages, v_pages = list(k_pages), list(v_pages)
        _need(len(k_pages) == len(v_pages) and k_pages, "one K and one V pool per layer")
        first = k_pages[0]
        _need(first.is_cuda, "the pools must be CUDA tensors")
        _need(first.dim() == 4, "a pool is [n_pages, n_kv_heads, page_rows, head_dim]")
        for t in k_pages + v_pages:
            _need(t.shape == first.shape and t.dtype == first.dtype and t.device == first.device and t.is_contiguous(),
                  "the pools must be contiguous and alike in shape, type and device")
        _need(table.dim() == 2, "table is [n_seqs, max_pages]")
        _need(first.dtype in _CODES, "the pools must be bfloat16 or float16, got %s" % first.dtype)
        n_pages, n_kv_heads, page_rows, head_dim = first.shape
        n_seqs, max_pages = table.shape
        dev = first.device
        self.k_pages, self.v_pages, self.table, self.lens, self.refs = k_pages, v_pages, table, lens, refs
        self.device = dev
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.scratch = torch.empty(max(1, _LIBRARY.msm_pages_scratch_ints(n_pages, n_seqs)), dtype=torch.int32,
                                   device=dev)
        kp, self._k_ptrs = _ptr_array([t.data_ptr() for t in k_pages])
        vp, self._v_ptrs = _ptr_array([t.data_ptr() for t in v_pages])
        self._c = MsmPages(dev.index, _CODES[first.dtype], len(k_pages), n_pages, page_rows, n_kv_heads, head_dim, n_seqs,
                           max_pages, kp, vp, _int32(table, "table", n_seqs * max_pages, dev.index),
                           _int32(lens, "lens", n_seqs, dev.index), _int32(refs, "refs", n_pages, dev.index),
                           self.status.data_ptr(), self.scratch.data_ptr())
        self._ref = ctypes.byref(self._c)
        self._lib = _LIBRARY
        self._index, self._n_seqs, self._kv_heads, self._head_dim = dev.index, n_seqs, n_kv_heads, head_dim
        self._dtype = first.dtype
        self._bytes = {}      # bytes of the attention's workspace by number of query heads
        self._workspace = {}  # workspaces by (stream, number of query heads)

    @classmethod
    def allocate(cls, n_layers, n_pages, page_rows, n_kv_heads, head_dim, n_seqs, max_pages, dtype=None, device=None):
        """An empty cache (bfloat16 by default)."""
        if _torch is None:
            _load()
        torch = _torch
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)

        def pools():
            return [torch.zeros((n_pages, n_kv_heads, page_rows, head_dim), dtype=dtype or torch.bfloat16, device=dev)
                    for _ in range(n_layers)]

        def ints(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=dev)
        return cls(pools(), pools(), ints(n_seqs, max_pages).fill_(-1), ints(n_seqs), ints(n_pages))

    def resize(self, new_lens):
        """msm_pages_resize: int32 [n_seqs] on the device, -1 = leave as it is."""
        _check(self._lib.msm_pages_resize(self._ref, _int32(new_lens, "new_lens", self._n_seqs, self._index),
                                          _raw_stream(self._index)))

    def fork(self, parent):
        """msm_pages_fork: int32 [n_seqs] on the device, -1 = none."""
        _check(self._lib.msm_pages_fork(self._ref, _int32(parent, "parent", self._n_seqs, self._index),
                                        _raw_stream(self._index)))

    def compact(self):
        """msm_pages_compact."""
        _check(self._lib.msm_pages_compact(self._ref, _raw_stream(self._index)))

    def write(self, layer, k, v, starts):
        """msm_pages_write: k, v [n_tokens, n_kv_heads, head_dim], starts int32 [n_seqs + 1]."""
        n, i = len(k), self._index
        if n > 0x7FFFFFFF:
            raise ValueError("more than 2^31 - 1 tokens")
        shape = (n, self._kv_heads, self._head_dim)
        kt, kh = _rows(k, "k", shape, self._dtype, i)
        vt, vh = _rows(v, "v", shape, self._dtype, i)
        _check(self._lib.msm_pages_write(self._ref, _c_int(layer), k.data_ptr(), v.data_ptr(), kt, kh, vt, vh,
                                         _int32(starts, "starts", self._n_seqs + 1, i), n, _raw_stream(i)))

    def attention(self, layer, q, window=0, scale=None, out=None):
        """msm_paged_attention: q [n_seqs, n_q_heads, head_dim]; scale defaults to
        1 / sqrt(head_dim).  Returns out."""
        if q.dim() != 3:
            raise ValueError("q must be [n_seqs, n_q_heads, head_dim]")
        heads, i, hd, layer = q.shape[1], self._index, self._head_dim, _c_int(layer)
        shape = (self._n_seqs, heads, hd)
        qs, qh = _rows(q, "q", shape, self._dtype, i)
        if out is None:
            out = _empty(shape, dtype=self._dtype, device=self.device)
            os_, oh = heads * hd, hd
        else:
            os_, oh = _rows(out, "out", shape, self._dtype, i)
        stream = _raw_stream(i)
        n = self._bytes.get(heads)
        if n is None:
            n = self._lib.msm_paged_attention_workspace(self._ref, heads)
            if n == 0:  # the call says what is wrong
                _check(self._lib.msm_paged_attention(self._ref, layer, None, qs, qh, heads, 1.0, 0, None, os_, oh, None,
                                                     0, None))
            self._bytes[heads] = n
        # one workspace per stream, and one per call that a graph records (graphs recorded on
        # one stream may be replayed on two)
        if _capturing():
            ws = _torch.zeros(n, dtype=_torch.uint8, device=self.device)
        else:
            ws = self._workspace.get((stream, heads))
            if ws is None:
                ws = self._workspace[stream, heads] = _torch.zeros(n, dtype=_torch.uint8, device=self.device)
        st = self._lib.msm_paged_attention(self._ref, layer, q.data_ptr(), qs, qh, heads,
                                           (hd or 1) ** -0.5 if scale is None else scale, _c_int(window), out.data_ptr(),
                                           os_, oh, ws.data_ptr(), n, stream)
        if st:
            _check(st)
        return out

    def sync(self):
        """msm_pages_sync: waits for the current stream; raises MsmError for an error that a
        call met on the device (and clears it)."""
        _check(self._lib.msm_pages_sync(self._ref, _raw_stream(self._index)))


def prompt_attention(q, k, v, q_starts, k_starts=None, window=0, scale=None, out=None, status=None):
    """msm_prompt_attention: causal attention of packed prompts.

    q [n_q, n_q_heads, head_dim], k and v [n_k, n_kv_heads, head_dim] (any strides that keep
    rows consecutive; ``cache.transpose(0, 1)`` of a verify-step cache [n_kv_heads, max_ctx,
    head_dim] is read in place), q_starts and k_starts int32 [n_seqs + 1] on the device
    (k_starts defaults to q_starts; a sequence without queries passes over keys, as the rows that a
    cache has to spare), scale defaults to 1 / sqrt(head_dim).  Returns out; a new
    one is uninitialised behind the last sequence.

    The kernel's own waits end after 2 s, which only a fault or a GPU that is busy elsewhere brings
    about: the rows that were not done are NaN then, and ``status``, an int32 tensor of one
    entry that holds 0, becomes MSM_ERR_DEVICE_TIMEOUT."""
    if _torch is None:
        _load()
    i, dtype, shape, k_shape = q.get_device(), q.dtype, q.shape, k.shape
    if i < 0:
        raise ValueError("q must be a CUDA tensor")
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError("expected bfloat16 or float16, got %s" % dtype)
    if len(shape) != 3 or len(k_shape) != 3 or k_shape[2] != shape[2]:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    n_q, heads, hd = shape
    n_k, kv_heads, _ = k_shape
    qt, qh = _rows(q, "q", shape, dtype, i)
    kt, kh = _rows(k, "k", k_shape, dtype, i)
    vt, vh = _rows(v, "v", k_shape, dtype, i)
    if out is None:
        out = _empty(shape, dtype=dtype, device=q.device)
        ot, oh = heads * hd, hd
    else:
        ot, oh = _rows(out, "out", shape, dtype, i)
    n_seqs = q_starts.numel() - 1
    qs = _int32(q_starts, "q_starts", n_seqs + 1, i)
    ks = qs if k_starts is None else _int32(k_starts, "k_starts", n_seqs + 1, i)
    a = _PROMPT.pack(i, code, n_seqs, n_q, n_k, heads, kv_heads, hd, _c_int(window),
                     (hd or 1) ** -0.5 if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                     out.data_ptr(), qt, qh, kt, kh, vt, vh, ot, oh, qs, ks,
                     0 if status is None else _int32(status, "status", 1, i), 0)
    st = _LIBRARY.msm_prompt_attention(a, _raw_stream(i))
    if st:
        _check(st)
    return out
