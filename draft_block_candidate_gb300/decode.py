"""Python binding of the decoding entry points: argument marshalling over the C ABI.

Beam search's choice and the states that follow it (beam_select, beam_reorder), and the
paged 8-bit key / value cache with its writer and the attention that reads it (KV8Cache,
kv8_append, kv8_attention).  Tensors may lie on any one device: the call runs there, on
`stream` or on that device's current stream, and what it allocates belongs to that stream.
Functions raise ValueError on tensors that do not fit the call and LilicorrError on a
non-OK status.

A call on one token's work takes a few microseconds on the device, so what the host does
per call matters: a tensor that fits is passed by one test (_want), and layouts that take
some working out are kept by shape and strides (_state_layout).
"""
from __future__ import annotations

import ctypes as C
import functools
import math
import struct
from typing import Optional, Sequence

import torch

from . import _lib as L
from .api import LilicorrError, _check, _ldtype


def _run_on(dev: int, stream):
    """The raw stream, and a context that makes the device and the stream current where they
    are not (else None)."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
        return raw, (None if torch._C._cuda_getDevice() == dev else torch.cuda.device(dev))
    if stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{dev}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _want(t, name: str, dtype, shape, dev: Optional[int], contiguous: bool = True) -> None:
    """Refuses a tensor of another type, shape (None: any extent), device or layout."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _fits32(n: int, name: str) -> None:
    """Refuses what ctypes would cut down to its low 32 bits."""
    if not -(1 << 31) <= n < (1 << 31):
        raise ValueError(f"{name} must fit 32 bits, got {n}")


def _new_workspace(need: int, dev, what: str) -> torch.Tensor:
    if need == 0:
        raise LilicorrError(1, what)
    return torch.empty(need, dtype=torch.uint8, device=dev)


# ----------------------------------------------------------------------------- beam search

def _beam_rows(logits: torch.Tensor):
    if not isinstance(logits, torch.Tensor) or logits.dim() != 3:
        raise ValueError("logits must be a tensor [batch, beams, V]")
    if not logits.is_cuda:
        raise ValueError("logits must be on a GPU")
    batch, beams, V = logits.shape
    if batch < 1 or beams < 1 or V < 1:
        raise ValueError("logits must not be empty")
    _fits32(beams, "beams")
    sb, sw, sv = logits.stride()
    row = sw if beams > 1 else sb if batch > 1 else V
    if (V > 1 and sv != 1) or row < V or (batch > 1 and sb != beams * row):
        raise ValueError("logits rows must be contiguous and a uniform stride apart")
    return batch, beams, V, row, _ldtype(logits)


def beam_select_workspace(logits: torch.Tensor, n_out: int) -> torch.Tensor:
    """A workspace for beam_select of logits of this shape."""
    batch, beams, V, _, ld = _beam_rows(logits)
    _fits32(n_out, "n_out")
    with torch.cuda.device(logits.device):
        n = int(L.lib().lilicorr_beam_select_workspace_bytes(batch, beams, V, n_out, ld))
        return _new_workspace(n, logits.device, "lilicorr_beam_select_workspace_bytes")


def beam_select(logits: torch.Tensor, scores: torch.Tensor, n_out: int,
                finished: Optional[torch.Tensor] = None, pad_id: int = 0,
                workspace: Optional[torch.Tensor] = None, out=None, stream=None):
    """lilicorr_beam_select: the n_out best continuations of each batch entry.

    logits [batch, beams, V] bf16/f32 (rows a uniform stride >= V apart), scores
    [batch, beams] f32 cumulative log-probabilities, finished [batch, beams] bool.  Returns
    (score [batch, n_out] f32, token int32, parent int32), best first; `out` may hold the
    three preallocated."""
    batch, beams, V, row, ld = _beam_rows(logits)
    dev = logits.get_device()
    _want(scores, "scores", torch.float32, (batch, beams), dev)
    if finished is not None:
        _want(finished, "finished", torch.bool, (batch, beams), dev)
    if workspace is not None:
        _want(workspace, "workspace", torch.uint8, (workspace.numel(),), dev)
    if out is not None:
        if len(out) != 3:
            raise ValueError("out must hold score, token and parent")
        _want(out[0], "score", torch.float32, (batch, n_out), dev)
        _want(out[1], "token", torch.int32, (batch, n_out), dev)
        _want(out[2], "parent", torch.int32, (batch, n_out), dev)
    if not 1 <= n_out <= 32 or beams > 32:
        raise ValueError("1 <= n_out <= 32 and at most 32 beams")
    _fits32(pad_id, "pad_id")
    raw, ctx = _run_on(dev, stream)

    def call():
        lib = L.lib()
        ws, o = workspace, out
        if o is None:
            shape, where = (batch, n_out), logits.device
            o = (torch.empty(shape, dtype=torch.float32, device=where),
                 torch.empty(shape, dtype=torch.int32, device=where),
                 torch.empty(shape, dtype=torch.int32, device=where))
        if ws is None:
            ws = _new_workspace(int(lib.lilicorr_beam_select_workspace_bytes(
                batch, beams, V, n_out, ld)), logits.device, "lilicorr_beam_select")
        st = lib.lilicorr_beam_select(
            logits.data_ptr(), ld, batch, beams, V, row, n_out, scores.data_ptr(),
            None if finished is None else finished.data_ptr(), pad_id, o[0].data_ptr(),
            o[1].data_ptr(), o[2].data_ptr(), ws.data_ptr(), ws.numel(), raw)
        if st:
            _check(st, "lilicorr_beam_select")
        return o

    if ctx is None:
        return call()
    with ctx:
        return call()


@functools.lru_cache(maxsize=4096)
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


_PAIR, _REST = struct.Struct("=QQ"), struct.Struct("=8q")


@functools.lru_cache(maxsize=4096)
def _state_fields(shape, sa, sb, esize: int):
    """lilicorr_beam_state behind its two pointers, as bytes, for a state of these strides."""
    lay = _state_layout(shape[2:], sa[2:], sb[2:], esize)
    if lay is None:
        raise ValueError("a state's layout behind the beams is not equal contiguous pieces a "
                         "uniform stride apart")
    return _REST.pack(sa[0] * esize, sa[1] * esize, lay[0], sb[0] * esize, sb[1] * esize, *lay[1:])


def beam_reorder(states: Sequence[torch.Tensor], parent: torch.Tensor,
                 out: Optional[Sequence[torch.Tensor]] = None, stream=None):
    """lilicorr_beam_reorder: state[b, j] becomes state[b, parent[b, j]] for every state.

    states: tensors [batch, beams, ...] of any type; behind the beams their layout must
    come down to equal contiguous pieces a uniform stride apart (a slice cache[..., :t, :]
    of a contiguous cache does).  out: tensors of the same shapes and types to write
    instead; without it the states are gathered in place.  States run side by side: no two may
    share memory that is written (one tensor twice, or out=[b, a] for [a, b], is refused).
    parent [batch, beams] int32.  Returns the list of written tensors."""
    into = list(states if out is None else out)
    if not into or len(into) != len(states):
        raise ValueError("there must be states, and out must hold one tensor for each")
    if not isinstance(parent, torch.Tensor) or parent.dim() != 2:
        raise ValueError("parent must be a tensor [batch, beams]")
    batch, beams = rows = parent.shape
    dev = parent.get_device()
    _fits32(beams, "beams")
    _want(parent, "parent", torch.int32, rows, dev)
    if dev < 0:
        raise ValueError("parent must be on a GPU")
    packed = []
    for s, o in zip(states, into):
        shape = s.shape
        if shape[:2] != rows:
            raise ValueError(f"a state must have shape [{batch}, {beams}, ...], got {tuple(shape)}")
        if s.get_device() != dev or o.get_device() != dev:
            raise ValueError(f"states must be on cuda:{dev}")
        if o is not s and (o.shape != shape or o.dtype != s.dtype):
            raise ValueError("out must have the states' shapes and types")
        if s.numel():
            packed.append(_PAIR.pack(s.data_ptr(), o.data_ptr()))
            packed.append(_state_fields(shape, s.stride(), o.stride(), s.element_size()))
    if packed:
        raw, ctx = _run_on(dev, stream)
        args = (b"".join(packed), len(packed) // 2, parent.data_ptr(), batch, beams, raw)
        if ctx is None:
            st = L.lib().lilicorr_beam_reorder(*args)
        else:
            with ctx:
                st = L.lib().lilicorr_beam_reorder(*args)
        if st:
            _check(st, "lilicorr_beam_reorder")
    return into


# ------------------------------------------------------------------------- the 8-bit cache

class KV8Cache:
    """A paged key / value cache in e4m3 with one scale for each page and head.

    k, v [n_pages, kv_heads, page, head_dim] float8_e4m3fn; k_scale, v_scale
    [n_pages, kv_heads] f32, positive, finite and at least 2^-126.  page in {16, 32, 64, 128}, head_dim in {32, 64, 128}."""

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
        dev = k.get_device()
        _want(k, "k", torch.float8_e4m3fn, k.shape, dev)
        _want(v, "v", torch.float8_e4m3fn, k.shape, dev)
        _want(k_scale, "k_scale", torch.float32, k.shape[:2], dev)
        _want(v_scale, "v_scale", torch.float32, k.shape[:2], dev)
        if not k.is_cuda:
            raise ValueError("the cache must be on a GPU")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.kv_heads, self.page, self.head_dim = k.shape
        self.device = k.device
        if self.page not in (16, 32, 64, 128) or self.head_dim not in (32, 64, 128):
            raise ValueError("page must be 16, 32, 64 or 128 and head_dim 32, 64 or 128, got "
                             f"{self.page} and {self.head_dim}")
        self._desc = L.Kv8CacheDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                    v_scale.data_ptr(), *k.shape)
        self._ref = C.addressof(self._desc)


def _rows(t, name: str, heads: Optional[int], D: int, total: Optional[int], dev: int) -> tuple:
    """Token and head strides of rows [total, heads, D] whose last dimension is contiguous."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.dim() != 3
            or t.get_device() != dev or t.shape[2] != D or (heads is not None and t.shape[1] != heads)
            or (total is not None and t.shape[0] != total)):
        _want(t, name, torch.bfloat16, (total, heads, D), dev, contiguous=False)
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    # a dimension of one has no stride of its own
    n, h, _ = t.shape
    return (st if n > 1 else 0), (sh if h > 1 else 0)


def _sequences(q_start, kv_len, block_table, dev: int) -> tuple:
    if not isinstance(kv_len, torch.Tensor) or kv_len.dim() != 1:
        raise ValueError("kv_len must be a tensor [batch]")
    batch = kv_len.shape[0]
    _want(kv_len, "kv_len", torch.int32, (batch,), dev)
    _want(q_start, "q_start", torch.int32, (batch + 1,), dev)
    if (not isinstance(block_table, torch.Tensor) or block_table.dtype is not torch.int32
            or block_table.dim() != 2 or block_table.get_device() != dev or block_table.shape[0] != batch):
        _want(block_table, "block_table", torch.int32, (batch, None), dev, contiguous=False)
    rows, step = block_table.stride()
    cols = block_table.shape[1]
    if step != 1 and cols > 1:
        raise ValueError("block_table's rows must be contiguous")
    _fits32(cols, "block_table's columns")
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
    dev = cache.device.index
    kt, kh = _rows(k, "k", cache.kv_heads, cache.head_dim, None, dev)
    total = k.shape[0]
    vt, vh = _rows(v, "v", cache.kv_heads, cache.head_dim, total, dev)
    batch, rows, cols = _sequences(q_start, kv_len, block_table, dev)
    _fits32(max_new, "max_new")
    if tail_src is not None:
        _want(tail_src, "tail_src", torch.int32, (batch,), dev)
    if batch == 0 or total == 0:
        return
    raw, ctx = _run_on(dev, stream)
    args = (cache._ref, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, total, q_start.data_ptr(),
            kv_len.data_ptr(), batch, block_table.data_ptr(), rows, cols, max_new,
            None if tail_src is None else tail_src.data_ptr(), raw)
    if ctx is None:
        st = L.lib().lilicorr_kv8_append(*args)
    else:
        with ctx:
            st = L.lib().lilicorr_kv8_append(*args)
    if st:
        _check(st, "lilicorr_kv8_append")


def kv8_attention_workspace(q: torch.Tensor, cache: KV8Cache, block_table: torch.Tensor,
                            max_new: int) -> torch.Tensor:
    """A workspace for kv8_attention of q's heads, these sequences and at most max_new new
    tokens of each."""
    _fits32(max_new, "max_new")
    with torch.cuda.device(cache.device):
        n = int(L.lib().lilicorr_kv8_attention_workspace_bytes(
            max_new, q.shape[1], cache.kv_heads, cache.head_dim))
        return _new_workspace(n, cache.device, "lilicorr_kv8_attention_workspace_bytes")


def kv8_attention(q: torch.Tensor, cache: KV8Cache, q_start: torch.Tensor, kv_len: torch.Tensor,
                  block_table: torch.Tensor, max_new: int, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, lse=None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """lilicorr_kv8_attention: attention of each sequence's new tokens over its cached ones.

    q [total, q_heads, head_dim] bf16 (strides by token and head multiples of 8); sequences
    as kv8_append takes them; new token i of n sees the first kv_len - n + i + 1 tokens.
    max_new * q_heads / kv_heads of at most 16 picks a kernel for few rows for the whole call.
    scale: 1 / sqrt(head_dim) by default.  out [total, q_heads, head_dim] bf16 (rows outside
    the sequences keep what they hold; a new one holds zeros there).  lse: True, or a tensor
    [total, q_heads] f32 to write the natural-log sums of exponentials to (True: -inf outside
    the sequences).  q, out and lse must not overlap.  Returns out, or (out, lse)."""
    dev = cache.device.index
    qt, qh = _rows(q, "q", None, cache.head_dim, None, dev)
    total, q_heads, D = q.shape
    batch, rows, cols = _sequences(q_start, kv_len, block_table, dev)
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
        lib = L.lib()
        o, norm, ws = out, lse, workspace
        if o is None:
            o = torch.zeros(total, q_heads, D, dtype=torch.bfloat16, device=cache.device)
        if new_lse:
            norm = torch.full((total, q_heads), -math.inf, dtype=torch.float32, device=cache.device)
        if batch > 0 and total > 0:
            if ws is None:
                ws = _new_workspace(int(lib.lilicorr_kv8_attention_workspace_bytes(
                    max_new, q_heads, cache.kv_heads, D)), cache.device, "lilicorr_kv8_attention")
            st = lib.lilicorr_kv8_attention(
                cache._ref, q.data_ptr(), qt, qh, total, q_heads, q_start.data_ptr(),
                kv_len.data_ptr(), batch, block_table.data_ptr(), rows, cols, max_new, scale,
                o.data_ptr(), None if norm is None else norm.data_ptr(), ws.data_ptr(),
                ws.numel(), raw)
            if st:
                _check(st, "lilicorr_kv8_attention")
        return o if norm is None else (o, norm)

    if ctx is None:
        return call()
    with ctx:
        return call()
