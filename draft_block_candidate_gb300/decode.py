"""Python binding of the decoding entry points: argument marshalling over the C ABI.

Beam search's choice and the states that follow it (beam_select, beam_reorder), and the
paged 8-bit key / value cache with its writer and the attention that reads it (KV8Cache,
kv8_append, kv8_attention).  Tensors may lie on any one device: the call runs there, on
`stream` or on that device's current stream, and what it allocates belongs to that stream.
Functions raise ValueError on tensors that do not fit the call and LilicorrError on a
non-OK status.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import functools
import math
from typing import Optional, Sequence

import torch

from . import _lib as L
from .api import LilicorrError, _check, _ldtype

_HERE = contextlib.nullcontext()


def _run_on(dev: torch.device, stream):
    """Context in which `dev` and `stream` are current, and the raw stream."""
    if stream is None:
        raw = torch.cuda.current_stream(dev).cuda_stream
        return (_HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)), raw
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {dev}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _want(t, name: str, dtype, shape, dev=None, contiguous: bool = True) -> None:
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(ws: Optional[torch.Tensor], need: int, dev: torch.device, what: str) -> torch.Tensor:
    """The caller's workspace, looked over, or a new one."""
    if need == 0:
        raise LilicorrError(1, what)
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    _want(ws, "workspace", torch.uint8, (None,), dev)
    return ws


# ----------------------------------------------------------------------------- beam search

def _beam_rows(logits: torch.Tensor):
    if not isinstance(logits, torch.Tensor) or logits.dim() != 3:
        raise ValueError("logits must be a tensor [batch, beams, V]")
    if not logits.is_cuda:
        raise ValueError("logits must be on a GPU")
    batch, beams, V = logits.shape
    if batch < 1 or beams < 1 or V < 1:
        raise ValueError("logits must not be empty")
    sb, sw, sv = logits.stride()
    row = sw if beams > 1 else sb if batch > 1 else V
    if (V > 1 and sv != 1) or row < V or (batch > 1 and sb != beams * row):
        raise ValueError("logits rows must be contiguous and a uniform stride apart")
    return batch, beams, V, row, _ldtype(logits)


def beam_select_workspace(logits: torch.Tensor, n_out: int) -> torch.Tensor:
    """A workspace for beam_select of logits of this shape."""
    batch, beams, V, _, ld = _beam_rows(logits)
    n = int(L.lib().lilicorr_beam_select_workspace_bytes(batch, beams, V, n_out, ld))
    return _workspace(None, n, logits.device, "lilicorr_beam_select_workspace_bytes")


def beam_select(logits: torch.Tensor, scores: torch.Tensor, n_out: int,
                finished: Optional[torch.Tensor] = None, pad_id: int = 0,
                workspace: Optional[torch.Tensor] = None, out=None, stream=None):
    """lilicorr_beam_select: the n_out best continuations of each batch entry.

    logits [batch, beams, V] bf16/f32 (rows a uniform stride >= V apart), scores
    [batch, beams] f32 cumulative log-probabilities, finished [batch, beams] bool.  Returns
    (score [batch, n_out] f32, token int32, parent int32), best first; `out` may hold the
    three preallocated."""
    batch, beams, V, row, ld = _beam_rows(logits)
    dev = logits.device
    _want(scores, "scores", torch.float32, (batch, beams), dev)
    if finished is not None:
        _want(finished, "finished", torch.bool, (batch, beams), dev)
    if not -(1 << 31) <= pad_id < (1 << 31):
        raise ValueError("pad_id must fit 32 bits")
    ctx, raw = _run_on(dev, stream)
    with ctx:
        if out is None:
            ids = torch.empty(2, batch, max(n_out, 1), dtype=torch.int32, device=dev)
            out = (torch.empty(batch, max(n_out, 1), dtype=torch.float32, device=dev), ids[0], ids[1])
        else:
            for t, name, dt in zip(out, ("score", "token", "parent"),
                                   (torch.float32, torch.int32, torch.int32)):
                _want(t, name, dt, (batch, n_out), dev)
        lib = L.lib()
        if workspace is None:
            workspace = _workspace(None, int(lib.lilicorr_beam_select_workspace_bytes(
                batch, beams, V, n_out, ld)), dev, "lilicorr_beam_select")
        else:
            _want(workspace, "workspace", torch.uint8, (None,), dev)
        st = lib.lilicorr_beam_select(
            logits.data_ptr(), ld, batch, beams, V, row, n_out, scores.data_ptr(),
            None if finished is None else finished.data_ptr(), pad_id, out[0].data_ptr(),
            out[1].data_ptr(), out[2].data_ptr(), workspace.data_ptr(), workspace.numel(), raw)
    _check(st, "lilicorr_beam_select")
    return out


@functools.lru_cache(maxsize=1024)
def _state_layout(shape, sa, sb, esize: int):
    """(strides and sizes in bytes) of a state's rows as segments that are contiguous in both
    layouts, or None.  shape, strides: behind [batch, beams], in elements."""
    dims = [(n, a, b) for n, a, b in zip(shape, sa, sb) if n != 1]
    seg = 1
    while dims and dims[-1][1] == seg and dims[-1][2] == seg:
        seg *= dims.pop()[0]
    segs, da, db = 1, 0, 0
    if dims:
        segs, da, db = dims.pop()
        while dims and dims[-1][1] == segs * da and dims[-1][2] == segs * db:
            segs *= dims.pop()[0]
    if dims:
        return None
    return da * esize, db * esize, segs, seg * esize


def beam_reorder(states: Sequence[torch.Tensor], parent: torch.Tensor,
                 out: Optional[Sequence[torch.Tensor]] = None, stream=None):
    """lilicorr_beam_reorder: state[b, j] becomes state[b, parent[b, j]] for every state.

    states: tensors [batch, beams, ...] of any type; behind the beams their layout must
    come down to equal contiguous pieces a uniform stride apart (a slice cache[..., :t, :]
    of a contiguous cache does).  out: tensors of the same shapes and types to write
    instead; without it the states are gathered in place.  parent [batch, beams] int32.
    Returns the list of written tensors."""
    states = list(states)
    if not states:
        raise ValueError("no states")
    into = states if out is None else list(out)
    if len(into) != len(states):
        raise ValueError("out must hold one tensor for each state")
    if not isinstance(parent, torch.Tensor) or parent.dim() != 2:
        raise ValueError("parent must be a tensor [batch, beams]")
    batch, beams = parent.shape
    dev = parent.device
    _want(parent, "parent", torch.int32, (batch, beams))
    arr = (L.BeamState * len(states))()
    n = 0
    for s, o in zip(states, into):
        if s.dim() < 2 or s.shape[0] != batch or s.shape[1] != beams:
            raise ValueError(f"a state must have shape [{batch}, {beams}, ...], got {tuple(s.shape)}")
        if s.device != dev or o.device != dev:
            raise ValueError(f"states must be on {dev}")
        if o is not s and (o.shape != s.shape or o.dtype != s.dtype):
            raise ValueError("out must have the states' shapes and types")
        if s.numel() == 0:
            continue
        sa, sb = s.stride(), o.stride()
        es = s.element_size()
        lay = _state_layout(s.shape[2:], sa[2:], sb[2:], es)
        if lay is None:
            raise ValueError("a state's layout behind the beams is not equal contiguous pieces a "
                             "uniform stride apart")
        arr[n] = L.BeamState(s.data_ptr(), o.data_ptr(), sa[0] * es, sa[1] * es, lay[0],
                             sb[0] * es, sb[1] * es, lay[1], lay[2], lay[3])
        n += 1
    if n == 0:
        return into
    ctx, raw = _run_on(dev, stream)
    with ctx:
        st = L.lib().lilicorr_beam_reorder(arr, n, parent.data_ptr(), batch, beams, raw)
    _check(st, "lilicorr_beam_reorder")
    return into


# ------------------------------------------------------------------------- the 8-bit cache

class KV8Cache:
    """A paged key / value cache in e4m3 with one scale for each page and head.

    k, v [n_pages, kv_heads, page, head_dim] float8_e4m3fn; k_scale, v_scale
    [n_pages, kv_heads] f32.  page in {16, 32, 64, 128}, head_dim in {32, 64, 128}."""

    def __init__(self, n_pages: int, kv_heads: int, page: int, head_dim: int, device="cuda"):
        shape = (n_pages, kv_heads, page, head_dim)
        self._hold(*(torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                     for _ in range(2)),
                   *(torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2)))

    @classmethod
    def from_tensors(cls, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
                     v_scale: torch.Tensor) -> "KV8Cache":
        """A cache over tensors that the caller keeps."""
        c = cls.__new__(cls)
        c._hold(k, v, k_scale, v_scale)
        return c

    def _hold(self, k, v, k_scale, v_scale):
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a tensor [n_pages, kv_heads, page, head_dim]")
        _want(k, "k", torch.float8_e4m3fn, (None,) * 4)
        _want(v, "v", torch.float8_e4m3fn, k.shape, k.device)
        _want(k_scale, "k_scale", torch.float32, k.shape[:2], k.device)
        _want(v_scale, "v_scale", torch.float32, k.shape[:2], k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.kv_heads, self.page, self.head_dim = k.shape
        self.device = k.device
        if self.page not in (16, 32, 64, 128) or self.head_dim not in (32, 64, 128):
            raise ValueError("page must be 16, 32, 64 or 128 and head_dim 32, 64 or 128, got "
                             f"{self.page} and {self.head_dim}")
        self._desc = L.Kv8CacheDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                    v_scale.data_ptr(), *k.shape)

    @property
    def desc(self):
        return C.byref(self._desc)


def _rows(t, name: str, heads: Optional[int], D: int, total, dev) -> tuple:
    """Token and head strides of rows [total, heads, D] whose last dimension is contiguous."""
    _want(t, name, torch.bfloat16, (total, heads, D), dev, contiguous=False)
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    # a dimension of one has no stride of its own
    return (0 if t.shape[0] <= 1 else st), (0 if t.shape[1] == 1 else sh)


def _sequences(q_start, kv_len, block_table, dev):
    _want(kv_len, "kv_len", torch.int32, (None,), dev)
    batch = kv_len.shape[0]
    _want(q_start, "q_start", torch.int32, (batch + 1,), dev)
    _want(block_table, "block_table", torch.int32, (batch, None), dev, contiguous=False)
    rows, step = block_table.stride()
    cols = block_table.shape[1]
    if step != 1 and cols > 1:
        raise ValueError("block_table's rows must be contiguous")
    return batch, (rows if batch > 1 else cols), cols


def kv8_append(cache: KV8Cache, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor,
               kv_len: torch.Tensor, block_table: torch.Tensor, max_new: int,
               tail_src: Optional[torch.Tensor] = None, stream=None) -> None:
    """lilicorr_kv8_append: write the new tokens' keys and values into the cache.

    k, v [total, kv_heads, head_dim] bf16 (strides by token and head multiples of 8);
    sequence b's new tokens are rows q_start[b] .. q_start[b+1]-1 and end at position
    kv_len[b]; block_table [batch, cols] int32 names its pages; max_new bounds the new
    tokens of a sequence; tail_src [batch] int32 the page to copy the rows before the first
    new token from (-1: the table's own)."""
    dev = cache.device
    kt, kh = _rows(k, "k", cache.kv_heads, cache.head_dim, None, dev)
    vt, vh = _rows(v, "v", cache.kv_heads, cache.head_dim, k.shape[0], dev)
    batch, rows, cols = _sequences(q_start, kv_len, block_table, dev)
    if tail_src is not None:
        _want(tail_src, "tail_src", torch.int32, (batch,), dev)
    if batch == 0 or k.shape[0] == 0:
        return
    ctx, raw = _run_on(dev, stream)
    with ctx:
        st = L.lib().lilicorr_kv8_append(
            cache.desc, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, k.shape[0], q_start.data_ptr(),
            kv_len.data_ptr(), batch, block_table.data_ptr(), rows, cols, max_new,
            None if tail_src is None else tail_src.data_ptr(), raw)
    _check(st, "lilicorr_kv8_append")


def kv8_attention_workspace(q: torch.Tensor, cache: KV8Cache, block_table: torch.Tensor,
                            max_new: int) -> torch.Tensor:
    """A workspace for kv8_attention of these heads and at most max_new tokens a sequence."""
    with torch.cuda.device(cache.device):
        n = int(L.lib().lilicorr_kv8_attention_workspace_bytes(max_new, q.shape[1], cache.kv_heads,
                                                               cache.head_dim))
        return _workspace(None, n, cache.device, "lilicorr_kv8_attention_workspace_bytes")


def kv8_attention(q: torch.Tensor, cache: KV8Cache, q_start: torch.Tensor, kv_len: torch.Tensor,
                  block_table: torch.Tensor, max_new: int, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, lse=None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """lilicorr_kv8_attention: attention of each sequence's new tokens over its cached ones.

    q [total, q_heads, head_dim] bf16 (strides by token and head multiples of 8); sequences
    as kv8_append takes them; new token i of n sees the first kv_len - n + i + 1 tokens.
    scale: 1 / sqrt(head_dim) by default.  out [total, q_heads, head_dim] bf16 (rows outside
    the sequences keep what they hold; a new one holds zeros there).  lse: True, or a tensor
    [total, q_heads] f32 to write the natural-log sums of exponentials to (True: -inf outside
    the sequences).  Returns out, or (out, lse)."""
    dev = cache.device
    qt, qh = _rows(q, "q", None, cache.head_dim, None, dev)
    total, q_heads, D = q.shape
    batch, rows, cols = _sequences(q_start, kv_len, block_table, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    ctx, raw = _run_on(dev, stream)
    with ctx:
        if out is None:
            out = torch.zeros(total, q_heads, D, dtype=torch.bfloat16, device=dev)
        else:
            _want(out, "out", torch.bfloat16, (total, q_heads, D), dev)
        if lse is True:
            lse = torch.full((total, q_heads), -math.inf, dtype=torch.float32, device=dev)
        elif lse is False:
            lse = None
        elif lse is not None:
            _want(lse, "lse", torch.float32, (total, q_heads), dev)
        if batch > 0 and total > 0:
            lib = L.lib()
            if workspace is None:
                workspace = _workspace(None, int(lib.lilicorr_kv8_attention_workspace_bytes(
                    max_new, q_heads, cache.kv_heads, D)), dev, "lilicorr_kv8_attention")
            else:
                _want(workspace, "workspace", torch.uint8, (None,), dev)
            st = lib.lilicorr_kv8_attention(
                cache.desc, q.data_ptr(), qt, qh, total, q_heads, q_start.data_ptr(),
                kv_len.data_ptr(), batch, block_table.data_ptr(), rows, cols, max_new, scale,
                out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(),
                workspace.numel(), raw)
            _check(st, "lilicorr_kv8_attention")
    return out if lse is None else (out, lse)
