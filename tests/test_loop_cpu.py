"""Refusals of the entry points around the cache and the logits, before anything touches a device."""
import ctypes as C

import pytest
import torch

INVALID, WORKSPACE = 1, 7
FAKE = 0x100000  # an aligned address that no call may reach


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from draft_block_candidate_gb300 import _lib
    return _lib.lib()


def adjust(lib, null=False, **kw):
    from draft_block_candidate_gb300 import _lib as L
    a = dict(logits=FAKE, out=FAKE, ldtype=1, rows=8, V=1000, row_stride=1000, out_stride=1000, groups=4, history=FAKE,
             history_stride=64, cap=64, seen=FAKE, n_bias=0, n_masks=0)
    a.update(kw)
    return lib.lilicorr_adjust_logits(None if null else C.byref(L.Adjust(**a)), None)


@pytest.mark.parametrize("kw", [
    dict(null=True), dict(logits=None), dict(out=None), dict(ldtype=2), dict(rows=0), dict(rows=1 << 31), dict(V=0),
    dict(V=1 << 31, row_stride=1 << 31, out_stride=1 << 31), dict(row_stride=999), dict(out_stride=999), dict(logits=FAKE + 1),
    dict(out_stride=1008), dict(out=FAKE + 4000), dict(out=FAKE - 2), dict(groups=0), dict(groups=3), dict(seen=None), dict(cap=0),
    dict(cap=1 << 29, history_stride=1 << 29), dict(history_stride=63), dict(history=None, repetition=FAKE),
    dict(history=None, counted_from=FAKE), dict(n_bias=-1), dict(n_bias=1025, bias_id=FAKE, bias=FAKE), dict(n_bias=3),
    dict(n_bias=3, bias_id=FAKE), dict(mask=FAKE, n_masks=0, mask_stride=32), dict(mask=FAKE, n_masks=8, mask_stride=31),
    dict(mask=FAKE, n_masks=7, mask_stride=32), dict(mask_index=FAKE),
    dict(rows=1 << 22, groups=1 << 20, V=1 << 24, row_stride=1 << 24, out_stride=1 << 24)])
def test_adjust_refuses(lib, kw):
    assert adjust(lib, **kw) == INVALID


def test_adjust_is_packed_as_the_structure_lies():
    from draft_block_candidate_gb300 import _lib as L
    from draft_block_candidate_gb300.logits import _ADJUST
    names = [n for n, _ in L.Adjust._fields_]
    a = L.Adjust.from_buffer_copy(_ADJUST.pack(*range(1, len(names) + 1)))
    assert _ADJUST.size == C.sizeof(L.Adjust)
    assert [getattr(a, n) for n in names] == list(range(1, len(names) + 1))


POOL = dict(refs=FAKE, n=100, table=FAKE, rows=4, stride=8, cols=8)
POOL_BAD = [dict(refs=None), dict(refs=FAKE + 2), dict(n=0), dict(n=1 << 31), dict(table=None), dict(table=FAKE + 1), dict(rows=0), dict(cols=0),
            dict(stride=7)]


def fork(lib, parent=FAKE, beams=4, batch_stride=32, **kw):
    a = {**POOL, **kw}
    return lib.lilicorr_kv8_fork(a["refs"], a["n"], a["table"], batch_stride, a["stride"], a["cols"], parent, a["rows"], beams, None)


def grow(lib, kv=FAKE, new=FAKE, page=64, max_new=4, tail=FAKE, granted=FAKE, ws=FAKE, size=1 << 20, **kw):
    a = {**POOL, **kw}
    return lib.lilicorr_kv8_grow(a["refs"], a["n"], a["table"], a["rows"], a["stride"], a["cols"], kv, new, page, max_new, tail, granted,
                                 ws, size, None)


def free(lib, keep=FAKE, page=64, **kw):
    a = {**POOL, **kw}
    return lib.lilicorr_kv8_free(a["refs"], a["n"], a["table"], a["rows"], a["stride"], a["cols"], keep, page, None)


@pytest.mark.parametrize("kw", POOL_BAD)
def test_a_bad_pool_or_table_is_refused(lib, kw):
    assert fork(lib, **kw) == grow(lib, **kw) == free(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(parent=None), dict(parent=FAKE + 3), dict(beams=0), dict(beams=33), dict(batch_stride=31),
                                dict(rows=1 << 30, cols=1 << 20, stride=1 << 20, batch_stride=1 << 22)])
def test_fork_refuses(lib, kw):
    assert fork(lib, **kw) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(kv=None), INVALID), (dict(new=None), INVALID), (dict(tail=None), INVALID), (dict(granted=None), INVALID), (dict(page=48), INVALID),
    (dict(max_new=0), INVALID), (dict(max_new=(1 << 24) + 1), INVALID), (dict(cols=1 << 26, stride=1 << 26), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 64), WORKSPACE), (dict(size=500), WORKSPACE)])
def test_grow_refuses(lib, kw, code):
    assert grow(lib, **kw) == code


@pytest.mark.parametrize("kw", [dict(keep=None), dict(page=0), dict(rows=1 << 30, cols=1 << 20, stride=1 << 20)])
def test_free_refuses(lib, kw):
    assert free(lib, **kw) == INVALID


def test_pages_workspace(lib):
    f = lib.lilicorr_kv8_pages_workspace_bytes
    assert f(100, 4) > 800 and f(0, 4) == f(1 << 31, 4) == f(100, 0) == f(100, 1 << 31) == 0


def caches(n=2, **kw):
    from draft_block_candidate_gb300 import _lib as L
    a = dict(k_pages=FAKE, v_pages=FAKE, k_scale=FAKE, v_scale=FAKE, n_pages=10, kv_heads=2, page=64, head_dim=128)
    return (L.Kv8CacheDesc * n)(*(L.Kv8CacheDesc(**{**a, **(kw if i == n - 1 else {})}) for i in range(n)))


BAD = [dict(k_pages=None), dict(v_scale=None), dict(n_pages=0), dict(n_pages=11), dict(kv_heads=3), dict(page=32), dict(head_dim=64),
       dict(head_dim=96), dict(v_pages=FAKE + 8)]


@pytest.mark.parametrize("kw", BAD)
def test_caches_that_differ_are_refused(lib, kw):
    good, bad = caches(), caches(**kw)
    assert lib.lilicorr_kv8_copy(bad, good, 2, FAKE, FAKE, 3, None) == INVALID
    assert lib.lilicorr_kv8_copy(good, bad, 2, FAKE, FAKE, 3, None) == INVALID
    assert lib.lilicorr_kv8_compact(bad, 2, FAKE, FAKE, 10, None, 0, FAKE, FAKE, 1 << 20, None) == INVALID


def test_copy_refuses(lib):
    c = caches()
    for args in ((None, c, 2, FAKE, FAKE, 3), (c, None, 2, FAKE, FAKE, 3), (c, c, 0, FAKE, FAKE, 3), (c, c, 2, None, FAKE, 3),
                 (c, c, 2, FAKE, None, 3), (c, c, 2, FAKE + 2, FAKE, 3), (c, c, 2, FAKE, FAKE, 0), (c, c, 2, FAKE, FAKE, 1 << 31)):
        assert lib.lilicorr_kv8_copy(*args, None) == INVALID


def test_compact_refuses(lib):
    from draft_block_candidate_gb300 import _lib as L

    def call(c=None, n=2, refs=FAKE, to=FAKE, pages=10, table=None, live=FAKE, ws=FAKE, size=1 << 20, **kw):
        t = dict(table=FAKE, out=FAKE, rows=4, row_stride=8, out_stride=8, cols=8)
        t.update(kw)
        return lib.lilicorr_kv8_compact(caches() if c is None else c, n, refs, to, pages, C.byref(L.Kv8Table(**t)), 1, live, ws, size, None)

    for kw in (dict(n=0), dict(refs=None), dict(to=None), dict(to=FAKE + 8), dict(pages=9), dict(live=None), dict(rows=0), dict(cols=0),
               dict(row_stride=7), dict(out_stride=9), dict(out=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(size=100)):
        assert call(**kw) == WORKSPACE


def cross(lib, q=FAKE, qt=1024, qh=128, total=8, heads=8, k=2 * FAKE, kt=512, kh=128, v=3 * FAKE, vt=512, vh=128, total_kv=100, kv_heads=2,
          D=128, q_start=FAKE, kv_start=FAKE, kv_len=FAKE, batch=2, max_new=4, scale=0.1, out=8 * FAKE, lse=None, ws=FAKE, size=1 << 30):
    return lib.lilicorr_cross_attention(q, qt, qh, total, heads, k, kt, kh, v, vt, vh, total_kv, kv_heads, D, q_start, kv_start, kv_len,
                                        batch, max_new, scale, out, lse, ws, size, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(q=FAKE + 8), dict(k=FAKE + 2), dict(qt=1020), dict(kh=4), dict(vt=-512), dict(vh=1 << 40),
    dict(D=0), dict(D=136), dict(D=20), dict(q_start=None), dict(kv_start=None), dict(kv_len=None), dict(batch=0), dict(batch=1 << 21),
    dict(total=0), dict(total=1 << 31), dict(total_kv=0), dict(total_kv=1 << 31), dict(max_new=0), dict(max_new=1 << 25), dict(kv_heads=0),
    dict(kv_heads=3), dict(kv_heads=1025, heads=1025), dict(heads=0), dict(heads=2 * 1025), dict(kt=0), dict(vh=0), dict(kt=120), dict(out=None),
    dict(out=FAKE + 8), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-3e38), dict(max_new=1 << 22, heads=2048), dict(out=FAKE),
    dict(max_new=1 << 20, heads=1024, kv_heads=1024, total_kv=1 << 30, kt=1 << 18, vt=1 << 18, v=1 << 60),
    dict(out=2 * FAKE + 1024), dict(out=3 * FAKE), dict(lse=8 * FAKE + 64), dict(lse=FAKE + 128)])
def test_cross_refuses(lib, kw):
    assert cross(lib, **kw) == INVALID


def test_cross_workspace(lib):
    f = lib.lilicorr_cross_attention_workspace_bytes
    assert f(64) > 0 and f(128) > f(64) and f(0) == f(136) == f(12) == 0
    assert cross(lib, ws=None) == cross(lib, ws=FAKE + 64) == cross(lib, size=64) == WORKSPACE


def test_python_refuses_cpu_tensors_and_bad_layouts():
    import draft_block_candidate_gb300 as lc
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for call in (lambda: lc.adjust_logits(torch.zeros(2, 100)), lambda: lc.adjust_logits(torch.zeros(4, 6)[:, ::2]),
                 lambda: lc.adjust_logits(3), lambda: lc.kv8_fork(i32(5), i32(1, 2, 3), i32(1, 2)),
                 lambda: lc.kv8_grow(i32(5), i32(2, 3), i32(2), i32(2), 16, 1), lambda: lc.kv8_free(i32(5), i32(2, 3), i32(2), 16),
                 lambda: lc.kv8_copy([], i32(1), i32(1)), lambda: lc.kv8_compact([], i32(5), [])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("shape,strides,want", [
    ((100,), (1,), (1, 100, 100)), ((4, 100), (100, 1), (4, 100, 100)), ((4, 100), (128, 1), (4, 100, 128)),
    ((2, 3, 100), (384, 128, 1), (6, 100, 128)), ((2, 3, 100), (400, 128, 1), None), ((4, 100), (200, 2), None), ((4, 100), (0, 1), None),
    ((1, 4, 1, 100), (7, 100, 3, 1), (4, 100, 100)), ((5, 1), (3, 9), (5, 1, 3))])
def test_logit_rows(shape, strides, want):
    from draft_block_candidate_gb300.logits import _logit_rows
    t = torch.zeros(2000).as_strided(shape, strides)
    if want is None:
        with pytest.raises(ValueError):
            _logit_rows(t, "logits")
    else:
        assert _logit_rows(t, "logits") == want
