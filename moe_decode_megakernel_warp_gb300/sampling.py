"""Torch-facing wrapper of msm_sample (msm.h): next tokens drawn from logits.

Argument marshalling only; the work runs in the kernel of ``libmsm.so``, on torch's current stream of the
logits' device.
"""
from __future__ import annotations

import ctypes
import struct

from . import MSM_BF16, MSM_FP16, MSM_FP32, MsmSampling, _check, lib

# msm_sampling in the C layout (a bytes object takes a third of the time of a ctypes structure)
_SAMPLING = struct.Struct("4iPq8P")
assert _SAMPLING.size == ctypes.sizeof(MsmSampling)

# set at the first call
_empty = _raw_stream = _INT32 = _FLOAT32 = _sample = None
_CODES = {}


def _load():
    global _empty, _raw_stream, _INT32, _FLOAT32, _sample
    import torch
    _sample = lib().msm_sample
    _CODES.update({torch.bfloat16: MSM_BF16, torch.float16: MSM_FP16, torch.float32: MSM_FP32})
    _INT32, _FLOAT32 = torch.int32, torch.float32
    _raw_stream = torch._C._cuda_getCurrentRawStream
    _empty = torch.empty


def _entry(t, name, dtype, n, index):
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != index or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of %d entries on cuda:%d" % (name, dtype, n, index))
    return t.data_ptr()


def sample(logits, random, temperature=None, top_k=None, top_p=None, min_p=None, out=None, probs=None, kept=None):
    """msm_sample: draws a token per row of logits [n_rows, vocab] (float32, bfloat16 or float16; rows
    consecutive, any distance apart) with the row's number of ``random`` (float32 [n_rows], 0 .. 1).

    ``temperature``, ``top_p``, ``min_p`` (float32) and ``top_k`` (int32) are [n_rows] tensors on the logits'
    device, or None for 1, 1, 0 and no limit; temperature 0 takes the largest logit.  Returns the tokens,
    int32 [n_rows] (``out`` where it is given): -1 for a row that has none, or whose numbers are out of range.
    ``probs`` (float32 [n_rows]) becomes the tokens' probabilities among those kept, ``kept`` (int32
    [n_rows]) how many were."""
    if _empty is None:
        _load()
    i, code = logits.get_device(), _CODES.get(logits.dtype)
    if i < 0:
        raise ValueError("logits must be a CUDA tensor")
    if code is None:
        raise ValueError("expected float32, bfloat16 or float16, got %s" % logits.dtype)
    if logits.dim() != 2:
        raise ValueError("logits must be [n_rows, vocab]")
    n, vocab = logits.shape
    stride, one = logits.stride()
    if one != 1 and vocab > 1:
        raise ValueError("logits: the elements of a row must be consecutive")
    if n > 0x7FFFFFFF or vocab > 0x7FFFFFFF:
        raise ValueError("logits: more than 2^31 - 1 rows or columns")
    if random is None:
        raise ValueError("random is missing")
    if out is None:
        out = _empty(n, dtype=_INT32, device=logits.device)
    a = _SAMPLING.pack(i, code, n, vocab, logits.data_ptr(), stride if n > 1 else vocab,
                       _entry(temperature, "temperature", _FLOAT32, n, i), _entry(top_k, "top_k", _INT32, n, i),
                       _entry(top_p, "top_p", _FLOAT32, n, i), _entry(min_p, "min_p", _FLOAT32, n, i),
                       _entry(random, "random", _FLOAT32, n, i), _entry(out, "out", _INT32, n, i),
                       _entry(probs, "probs", _FLOAT32, n, i), _entry(kept, "kept", _INT32, n, i))
    st = _sample(a, _raw_stream(i))
    if st:
        _check(st)
    return out
