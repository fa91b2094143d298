"""Python binding of the edits that logits take before they are ranked (adjust_logits): argument
marshalling over the C ABI, in the manner of decode."""
from __future__ import annotations

import struct
from typing import Optional

import torch

from . import _lib as L
from .api import _check, _ldtype
from .decode import _row_layout, _run_on, _want

# lilicorr_adjust, as bytes (a ctypes structure of as many fields takes three times as long to fill)
_ADJUST = struct.Struct("=QQi4x5qQqi4x7Qi4xQqqQ")


def _logit_rows(t, name: str):
    """(rows, V, row stride) of logits [..., V] whose rows lie a uniform stride apart."""
    if not isinstance(t, torch.Tensor) or t.dim() < 1:
        raise ValueError(f"{name} must be a tensor [..., V]")
    lay = _row_layout(t.shape, t.stride())
    if lay is None:
        raise ValueError(f"{name}'s rows must be contiguous, a uniform stride apart, and not overlap")
    return lay[0], lay[1], max(lay[2], lay[1])


def _table(t, name: str, rows: Optional[int], cols: Optional[int], dev: int):
    """The row stride of an int32 table whose rows are contiguous."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.dim() != 2 or t.get_device() != dev
            or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols)):
        _want(t, name, torch.int32, (rows, cols), dev, contiguous=False)
    st, step = t.stride()
    n, c = t.shape
    if (step != 1 and c > 1) or (n > 1 and st < c):
        raise ValueError(f"{name}'s rows must be contiguous and not overlap")
    return st if n > 1 else c


def adjust_logits(logits: torch.Tensor, history: Optional[torch.Tensor] = None, seen: Optional[torch.Tensor] = None,
                  counted_from: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                  presence: Optional[torch.Tensor] = None, frequency: Optional[torch.Tensor] = None,
                  bias_ids: Optional[torch.Tensor] = None, bias_values: Optional[torch.Tensor] = None,
                  mask: Optional[torch.Tensor] = None, mask_index: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """lilicorr_adjust_logits: penalties for repeated tokens, biases and grammar masks.

    logits [..., V] bf16/f32 (rows a uniform stride >= V apart), edited in place, or into
    `out` of the same shape and type, which shares nothing with them or with what else is read.  history [groups, cap] int32 token ids (groups divides
    the rows; consecutive rows share one: the beams or the drafted rows of a request), of
    which row r sees the first seen[r] ([rows] int32); repetition, presence and frequency
    [groups] f32, the last two counting from position counted_from ([groups] int32) on.
    bias_ids int32 and bias_values f32 [groups, n] add to single tokens (negative ids: none).
    mask [n, (V + 31) // 32] int32, bit v % 32 of word v // 32 set where token v may be taken;
    mask_index [rows] int32 names each row's (negative: none), else there is one for each row.
    Returns the written tensor."""
    rows, V, row = _logit_rows(logits, "logits")
    if not logits.is_cuda:
        raise ValueError("logits must be on a GPU")
    dev = logits.get_device()
    ld = _ldtype(logits)
    into, into_row = logits, row
    if out is not None and out is not logits:
        _want(out, "out", logits.dtype, logits.shape, dev, contiguous=False)
        into, into_row = out, _logit_rows(out, "out")[2]
    groups, cap, hist_row, n_bias, n_masks, mask_row = rows, 0, 0, 0, 0, 0
    if history is not None:
        hist_row = _table(history, "history", None, None, dev)
        groups, cap = history.shape
        if cap < 1:
            raise ValueError("history must hold a token; leave it out where there is none")
        if seen is None:
            raise ValueError("a history needs seen")
        _want(seen, "seen", torch.int32, (rows,), dev)
    elif any(t is not None for t in (seen, counted_from, repetition, presence, frequency)):
        raise ValueError("penalties need a history")
    if bias_ids is not None:
        if bias_values is None:
            raise ValueError("biases need ids and values")
        if history is None and isinstance(bias_ids, torch.Tensor) and bias_ids.dim() == 2:
            groups = bias_ids.shape[0]
        _want(bias_ids, "bias_ids", torch.int32, (groups, None), dev)
        _want(bias_values, "bias_values", torch.float32, bias_ids.shape, dev)
        n_bias = bias_ids.shape[1]
        if n_bias > 1024:
            raise ValueError("at most 1024 biases")
    elif bias_values is not None:
        raise ValueError("biases need ids and values")
    if rows and (groups < 1 or rows % groups):
        raise ValueError(f"{groups} groups do not divide {rows} rows")
    for t, name, dtype in ((counted_from, "counted_from", torch.int32), (repetition, "repetition", torch.float32),
                           (presence, "presence", torch.float32), (frequency, "frequency", torch.float32)):
        if t is not None:
            _want(t, name, dtype, (groups,), dev)
    if mask is not None:
        mask_row = _table(mask, "mask", None if mask_index is not None else rows, (V + 31) // 32, dev)
        n_masks = mask.shape[0]
        if mask_index is not None:
            _want(mask_index, "mask_index", torch.int32, (rows,), dev)
    elif mask_index is not None:
        raise ValueError("mask_index needs masks")
    if rows == 0 or V == 0:
        return into
    ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    raw, ctx = _run_on(dev, stream)
    a = _ADJUST.pack(logits.data_ptr(), into.data_ptr(), ld, rows, V, row, into_row, groups, ptr(history), hist_row, cap, ptr(seen),
                     ptr(counted_from), ptr(repetition), ptr(presence), ptr(frequency), ptr(bias_ids), ptr(bias_values), n_bias,
                     ptr(mask), n_masks, mask_row, ptr(mask_index))
    if ctx is None:
        st = L.lib().lilicorr_adjust_logits(a, raw)
    else:
        with ctx:
            st = L.lib().lilicorr_adjust_logits(a, raw)
    if st:
        _check(st, "lilicorr_adjust_logits")
    return into
