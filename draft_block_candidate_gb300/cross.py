"""Python binding of the attention over states of another length (cross_attention): argument
marshalling over the C ABI, in the manner of decode."""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import _lib as L
from .api import _check
from .decode import _fits32, _new_workspace, _rows, _run_on, _want


def cross_attention_workspace(q: torch.Tensor, k: torch.Tensor, max_new: int) -> torch.Tensor:
    """A workspace for cross_attention of tensors of these sizes."""
    _fits32(max_new, "max_new")
    if not isinstance(k, torch.Tensor) or k.dim() != 3 or not k.is_cuda:
        raise ValueError("k must be a tensor [total_kv, kv_heads, head_dim] on a GPU")
    with torch.cuda.device(k.device):
        n = int(L.lib().lilicorr_cross_attention_workspace_bytes(k.shape[2]))
        return _new_workspace(n, k.device, "lilicorr_cross_attention_workspace_bytes")


def cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor, kv_start: torch.Tensor,
                    kv_len: torch.Tensor, max_new: int, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    lse=None, workspace: Optional[torch.Tensor] = None, stream=None):
    """lilicorr_cross_attention: attention of each request's rows over all of its states.

    q [total, q_heads, head_dim], k and v [total_kv, kv_heads, head_dim] bf16 (strides by token
    and head multiples of 8; head_dim a multiple of 8, at most 128).  Request b has rows
    q_start[b] .. q_start[b+1]-1 of q (its beams, the tokens of a block, or both; at most
    max_new) and states kv_start[b] .. kv_start[b] + kv_len[b] - 1 of k and v; int32.  A padded
    batch [batch, T, ...] of states is k.flatten(0, 1) with kv_start = b * T.  k and v may hold no states at all.
    scale: 1 / sqrt(head_dim) by default.  out [total, q_heads, head_dim] bf16 (rows outside the
    requests keep what they hold; a new one holds zeros there).  lse: True, or a tensor
    [total, q_heads] f32 to write the natural-log sums of exponentials to (True: -inf outside
    the requests).  out and lse must not overlap one another or what is read.  Returns out, or
    (out, lse)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or not q.is_cuda:
        raise ValueError("q must be a tensor [total, q_heads, head_dim] on a GPU")
    dev = q.get_device()
    total, q_heads, D = q.shape
    qt, qh = _rows(q, "q", None, D, None, dev)
    kt, kh = _rows(k, "k", None, D, None, dev)
    total_kv, kv_heads, _ = k.shape
    vt, vh = _rows(v, "v", kv_heads, D, total_kv, dev)
    if not isinstance(kv_len, torch.Tensor) or kv_len.dim() != 1:
        raise ValueError("kv_len must be a tensor [batch]")
    batch = kv_len.shape[0]
    _want(kv_len, "kv_len", torch.int32, (batch,), dev)
    _want(kv_start, "kv_start", torch.int32, (batch,), dev)
    _want(q_start, "q_start", torch.int32, (batch + 1,), dev)
    _fits32(max_new, "max_new")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is not None:
        _want(out, "out", torch.bfloat16, (total, q_heads, D), dev)
    if workspace is not None:
        _want(workspace, "workspace", torch.uint8, (workspace.numel(),), dev)
    new_lse = lse is True
    if isinstance(lse, bool):
        lse = None
    elif lse is not None:
        _want(lse, "lse", torch.float32, (total, q_heads), dev)
    raw, ctx = _run_on(dev, stream)

    def call():
        if total_kv == 0:  # a state that no request may have stands for none, so that who asks for one is reported
            none = torch.zeros(1, kv_heads, D, dtype=torch.bfloat16, device=q.device)
            return cross_attention(q, none, none, q_start, (kv_start == 0).int() * 2 - 1, kv_len, max_new, scale, out, new_lse or lse,
                                   workspace)
        lib = L.lib()
        o, norm, ws = out, lse, workspace
        if o is None:
            o = torch.zeros(total, q_heads, D, dtype=torch.bfloat16, device=q.device)
        if new_lse:
            norm = torch.full((total, q_heads), -math.inf, dtype=torch.float32, device=q.device)
        if batch > 0 and total > 0:
            if ws is None:
                ws = _new_workspace(int(lib.lilicorr_cross_attention_workspace_bytes(D)), q.device, "lilicorr_cross_attention")
            st = lib.lilicorr_cross_attention(
                q.data_ptr(), qt, qh, total, q_heads, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, total_kv, kv_heads, D,
                q_start.data_ptr(), kv_start.data_ptr(), kv_len.data_ptr(), batch, max_new, scale, o.data_ptr(),
                None if norm is None else norm.data_ptr(), ws.data_ptr(), ws.numel(), raw)
            if st:
                _check(st, "lilicorr_cross_attention")
        return o if norm is None else (o, norm)

    if ctx is None:
        return call()
    with ctx:
        return call()
