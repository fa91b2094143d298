"""Python binding of the 8-bit cache's pages that sequences share (kv8_fork, kv8_grow, kv8_free,
kv8_copy, kv8_compact): argument marshalling over the C ABI, in the manner of decode.

refs [n_pages] int32 (torch.zeros to begin with) counts the entries of block tables that name each
page; an entry is the page that its row holds there, or negative."""
from __future__ import annotations

import struct
from typing import Optional, Sequence

import torch

from . import _lib as L
from .api import _check
from .decode import KV8Cache, _fits32, _new_workspace, _row_layout, _run_on, _want


def _pool(refs) -> tuple:
    """(device, pages) of the counts of holders."""
    if isinstance(refs, torch.Tensor):
        dev, shape = refs.get_device(), refs.shape
        if refs.dtype is torch.int32 and len(shape) == 1 and dev >= 0 and refs.is_contiguous():
            return dev, shape[0]
        if len(shape) == 1 and dev >= 0:
            _want(refs, "refs", torch.int32, shape, dev)
    raise ValueError("refs must be a tensor [n_pages] on a GPU")


def _rows_of(table, dev: int, name: str = "table") -> tuple:
    """(rows, columns, row stride) of a table [..., cols] whose rows lie a uniform stride apart."""
    if not isinstance(table, torch.Tensor) or table.dtype is not torch.int32 or table.dim() < 2:
        raise ValueError(f"{name} must be an int32 tensor [..., cols]")
    if table.get_device() != dev:
        raise ValueError(f"{name} is on {table.device}, expected cuda:{dev}")
    lay = _row_layout(table.shape, table.stride())
    if lay is None:
        raise ValueError(f"{name}'s rows must be contiguous, a uniform stride apart, and not overlap")
    _fits32(lay[1], f"{name}'s columns")
    return lay


def _per_row(t, name: str, dtype, lead, dev: int) -> None:
    """A value for each row: of the table's shape without its columns, or flat."""
    if isinstance(t, torch.Tensor):
        if t.dtype is dtype and t.shape == lead and t.get_device() == dev and t.is_contiguous():
            return
        if t.dim() == 1:
            lead = (lead.numel(),)
    _want(t, name, dtype, lead, dev)


def _call(ctx, fn, name: str, args) -> None:
    if ctx is None:
        st = fn(*args)
    else:
        with ctx:
            st = fn(*args)
    if st:
        _check(st, name)


def kv8_pages_workspace(n_pages: int, rows: int, device="cuda") -> torch.Tensor:
    """A workspace for kv8_grow of so many rows, or kv8_compact, of a pool of n_pages."""
    n = int(L.lib().lilicorr_kv8_pages_workspace_bytes(n_pages, rows))
    return _new_workspace(n, device, "lilicorr_kv8_pages_workspace_bytes")


def kv8_fork(refs: torch.Tensor, table: torch.Tensor, parent: torch.Tensor, stream=None) -> None:
    """lilicorr_kv8_fork: row (b, j) of the table [batch, beams, cols] becomes row
    (b, parent[b, j]), in place, and refs counts the pages' holders anew.  parent [batch, beams]
    int32, as beam_select gives it; what else a hypothesis holds follows by beam_reorder."""
    dev, n_pages = _pool(refs)
    if not isinstance(table, torch.Tensor) or table.dtype is not torch.int32 or table.dim() != 3 or table.get_device() != dev:
        raise ValueError(f"table must be an int32 tensor [batch, beams, cols] on cuda:{dev}")
    batch, beams, cols = table.shape
    _want(parent, "parent", torch.int32, (batch, beams), dev)
    sb, sw, sc = table.stride()
    if cols > 1 and sc != 1:
        raise ValueError("table's rows must be contiguous")
    _fits32(cols, "table's columns")
    _fits32(beams, "beams")
    if 0 in table.shape:
        return
    if beams == 1:
        sw = cols
    raw, ctx = _run_on(dev, stream)
    _call(ctx, L.lib().lilicorr_kv8_fork, "lilicorr_kv8_fork",
          (refs.data_ptr(), n_pages, table.data_ptr(), sb if batch > 1 else beams * sw, sw, cols, parent.data_ptr(), batch, beams, raw))


def kv8_grow(refs: torch.Tensor, table: torch.Tensor, kv_len: torch.Tensor, new_tokens: torch.Tensor, page: int, max_new: int,
             out: Optional[Sequence[torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """lilicorr_kv8_grow: pages for the tokens that each row of the table [..., cols] writes next.

    kv_len int32 the tokens that the rows hold before, new_tokens int32 those to come (at most
    max_new of a row); both of the table's leading shape, or flat.  Returns (tail_src int32,
    granted bool) of the leading shape: the page whose earlier rows kv8_append is to copy, or
    -1, and whether the row has its pages; `out` may hold the two preallocated."""
    dev, n_pages = _pool(refs)
    rows, cols, row = _rows_of(table, dev)
    lead = table.shape[:-1]
    _per_row(kv_len, "kv_len", torch.int32, lead, dev)
    _per_row(new_tokens, "new_tokens", torch.int32, lead, dev)
    _fits32(page, "page")
    _fits32(max_new, "max_new")
    if out is not None:
        if len(out) != 2:
            raise ValueError("out must hold tail_src and granted")
        _per_row(out[0], "tail_src", torch.int32, lead, dev)
        _per_row(out[1], "granted", torch.bool, lead, dev)
    if workspace is not None:
        _want(workspace, "workspace", torch.uint8, (workspace.numel(),), dev)
    raw, ctx = _run_on(dev, stream)

    def call():
        o, ws = out, workspace
        if o is None:
            o = (torch.empty(lead, dtype=torch.int32, device=table.device), torch.empty(lead, dtype=torch.bool, device=table.device))
        if rows > 0:
            if ws is None:
                ws = kv8_pages_workspace(n_pages, rows, table.device)
            _call(None, L.lib().lilicorr_kv8_grow, "lilicorr_kv8_grow", (refs.data_ptr(), n_pages, table.data_ptr(), rows, row, cols, kv_len.data_ptr(),
                                              new_tokens.data_ptr(), page, max_new, o[0].data_ptr(), o[1].data_ptr(), ws.data_ptr(),
                                              ws.numel(), raw))
        return tuple(o)

    if ctx is None:
        return call()
    with ctx:
        return call()


def kv8_free(refs: torch.Tensor, table: torch.Tensor, keep: torch.Tensor, page: int, stream=None) -> None:
    """lilicorr_kv8_free: the rows of the table [..., cols] give up their pages behind the first
    `keep` tokens (int32, of the table's leading shape or flat): 0 ends a sequence, the length
    that is left after a check gives back what rejected tokens had."""
    dev, n_pages = _pool(refs)
    rows, cols, row = _rows_of(table, dev)
    _per_row(keep, "keep", torch.int32, table.shape[:-1], dev)
    _fits32(page, "page")
    if rows == 0 or cols == 0:
        return
    raw, ctx = _run_on(dev, stream)
    _call(ctx, L.lib().lilicorr_kv8_free, "lilicorr_kv8_free", (refs.data_ptr(), n_pages, table.data_ptr(), rows, row, cols, keep.data_ptr(), page, raw))


def _descriptions(caches: Sequence[KV8Cache]) -> bytes:
    """Their descriptions, one behind the other."""
    if not caches:
        raise ValueError("there must be caches")
    device = None
    for c in caches:
        if not isinstance(c, KV8Cache):
            raise ValueError("caches must be KV8Cache objects")
        if device is None:
            device = c.device
        elif c.device != device:
            raise ValueError("caches must be on one device")
    return b"".join([c._desc for c in caches])


# lilicorr_kv8_table, as bytes
_TABLE = struct.Struct("=QQqqqi4x")


def kv8_copy(caches: Sequence[KV8Cache], src: torch.Tensor, dst: torch.Tensor, into: Optional[Sequence[KV8Cache]] = None,
             stream=None) -> None:
    """lilicorr_kv8_copy: page src[i] of every cache (a layer each) is copied, with its scales, to
    page dst[i] of the same cache, or of the one beside it in `into`.  src, dst [n] int32;
    negative: no move.  A destination is no other move's source or destination."""
    have = _descriptions(caches)
    to = have if into is None else _descriptions(into)
    dev = caches[0].device.index
    if into is not None and (len(into) != len(caches) or into[0].device != caches[0].device):
        raise ValueError("into must hold a cache for each, on the same device")
    if not isinstance(src, torch.Tensor) or src.dim() != 1:
        raise ValueError("src must be a tensor [n]")
    _want(src, "src", torch.int32, src.shape, dev)
    _want(dst, "dst", torch.int32, src.shape, dev)
    if src.shape[0] == 0:
        return
    raw, ctx = _run_on(dev, stream)
    _call(ctx, L.lib().lilicorr_kv8_copy, "lilicorr_kv8_copy", (have, to, len(caches), src.data_ptr(), dst.data_ptr(), src.shape[0], raw))


def kv8_compact(caches: Sequence[KV8Cache], refs: torch.Tensor, tables: Sequence[torch.Tensor], out=None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """lilicorr_kv8_compact: the live pages of every cache (a layer each) move to the front.

    refs and the tables [..., cols], all of those that it counts, follow in place, or in `out`,
    (refs, tables) of the same shapes.  Returns live [1] int32, the number of live pages, which
    are now the first ones."""
    have = _descriptions(caches)
    dev, n_pages = _pool(refs)
    if caches[0].device.index != dev:
        raise ValueError(f"caches must be on cuda:{dev}")
    refs_to, to = refs, tables
    if out is not None:
        refs_to, to = out
        _want(refs_to, "refs of out", torch.int32, (n_pages,), dev)
    if len(to) != len(tables):
        raise ValueError("out must hold one table for each")
    packed = []
    for t, o in zip(tables, to):
        rows, cols, row = _rows_of(t, dev)
        if o is not t and (not isinstance(o, torch.Tensor) or o.shape != t.shape):
            raise ValueError("out's tables must have the tables' shapes")
        orow = row if o is t else _rows_of(o, dev, "a table of out")[2]
        if rows and cols:
            packed.append(_TABLE.pack(t.data_ptr(), o.data_ptr(), rows, row, orow, cols))
    if workspace is not None:
        _want(workspace, "workspace", torch.uint8, (workspace.numel(),), dev)
    raw, ctx = _run_on(dev, stream)

    def call():
        live = torch.empty(1, dtype=torch.int32, device=refs.device)
        ws = kv8_pages_workspace(n_pages, 1, refs.device) if workspace is None else workspace
        _call(None, L.lib().lilicorr_kv8_compact, "lilicorr_kv8_compact", (have, len(caches), refs.data_ptr(), refs_to.data_ptr(), n_pages,
                                             b"".join(packed), len(packed), live.data_ptr(), ws.data_ptr(),
                                             ws.numel(), raw))
        return live

    if ctx is None:
        return call()
    with ctx:
        return call()
