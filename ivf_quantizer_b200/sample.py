"""``sample_logits``: one draw per row of scores from its truncated softmax, with given uniforms,
through fgmm_sample_logits (include/fgmm.h).  CUDA tensors only; argument marshalling only."""
from __future__ import annotations

import operator

import torch

from ._lib import LIB
from .mx4 import _rows, call, empty


def _per_row(v, name, dtype, rows, device):
    if v is None:
        return None
    if not isinstance(v, torch.Tensor):
        return torch.full((rows,), v, dtype=dtype, device=device)
    if not (v.device == device and v.dtype == dtype and v.shape == (rows,) and v.is_contiguous()):
        raise ValueError(f"{name} must be a number or a contiguous {dtype} [rows] tensor on the "
                         "logits' device")
    return v


def _count(k, V):
    """top_k as a number: a whole one, of which 0 .. V is enough to say (V and 0 keep all)."""
    if k is None or isinstance(k, torch.Tensor):
        return k
    try:
        k = int(k) if isinstance(k, float) and k.is_integer() else operator.index(k)
    except TypeError:
        raise TypeError("top_k must be a whole number or an int32 [rows] tensor") from None
    return min(max(k, 0), V)


def sample_logits(logits: torch.Tensor, u: torch.Tensor, temperature=None, top_k=None, top_p=None,
                  min_p=None):
    """Draws one index per row of logits [rows, V] (float32 or bfloat16; -inf forbids an index).

    u: float64 [rows] uniforms in [0, 1).  temperature, top_p, min_p (float32) and top_k (int32):
    a number for all rows, a [rows] tensor (which saves the launch that fills one with the number),
    or None for no effect.  Truncation in the order top-k,
    top-p (of the weight that top-k left), min-p (relative to the largest weight); temperature 0
    takes the first maximum.

    Returns (ids int32 [rows], prob float32 [rows]), prob being the probability with which the
    index was drawn.  A row without a finite logit gives -1 and 0; one with a NaN or with a
    parameter outside its range gives -1 and NaN.
    """
    dt, rows, V, ld = _rows(logits, "logits")
    dev = logits.device
    if u is None:
        raise ValueError("u must be a float64 [rows] tensor")
    u = _per_row(u, "u", torch.float64, rows, dev)
    temperature = _per_row(temperature, "temperature", torch.float32, rows, dev)
    top_k = _per_row(_count(top_k, V), "top_k", torch.int32, rows, dev)
    top_p = _per_row(top_p, "top_p", torch.float32, rows, dev)
    min_p = _per_row(min_p, "min_p", torch.float32, rows, dev)
    ids = empty(rows, None, torch.int32, dev)
    prob = empty(rows, None, torch.float32, dev)
    call(LIB.fgmm_sample_logits, "fgmm_sample_logits", dev, logits.data_ptr(), dt, rows, V, ld,
         *[None if t is None else t.data_ptr() for t in (temperature, top_k, top_p, min_p)],
         u.data_ptr(), ids.data_ptr(), prob.data_ptr())
    return ids, prob
