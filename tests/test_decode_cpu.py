"""Refusals of the decoding entry points, before anything touches a device."""
import ctypes as C

import pytest
import torch

INVALID, WORKSPACE = 1, 7
FAKE = 0x10000  # an aligned address that no call may reach


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from draft_block_candidate_gb300 import _lib
    return _lib.lib()


def select(lib, **kw):
    a = dict(logits=FAKE, dt=1, batch=2, beams=4, V=1000, stride=1000, M=8, scores=FAKE, finished=None, pad=0,
             score=FAKE, token=FAKE, parent=FAKE, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return lib.lilicorr_beam_select(a["logits"], a["dt"], a["batch"], a["beams"], a["V"], a["stride"], a["M"], a["scores"],
                                    a["finished"], a["pad"], a["score"], a["token"], a["parent"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), INVALID), (dict(scores=None), INVALID), (dict(score=None), INVALID), (dict(token=None), INVALID),
    (dict(parent=None), INVALID), (dict(logits=FAKE + 1), INVALID), (dict(batch=0), INVALID), (dict(beams=0), INVALID),
    (dict(beams=33), INVALID), (dict(M=0), INVALID), (dict(M=33), INVALID), (dict(V=0), INVALID), (dict(stride=999), INVALID),
    (dict(V=1 << 31, stride=1 << 31), INVALID), (dict(dt=2), INVALID), (dict(batch=1 << 30), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 16), WORKSPACE), (dict(bytes=8), WORKSPACE)])
def test_select_refuses(lib, kw, code):
    assert select(lib, **kw) == code


def test_select_workspace_is_zero_for_unsupported_sizes(lib):
    f = lib.lilicorr_beam_select_workspace_bytes
    assert f(2, 4, 1000, 8, 1) > 0
    assert f(0, 4, 1000, 8, 1) == f(2, 33, 1000, 8, 1) == f(2, 4, 0, 8, 1) == f(2, 4, 1000, 33, 1) == f(2, 4, 1000, 8, 5) == 0


def reorder(lib, n=1, parent=FAKE, batch=2, beams=4, null=False, **kw):
    from draft_block_candidate_gb300 import _lib as L
    a = dict(src=1 << 20, dst=2 << 20, src_batch_stride=1024, src_beam_stride=256, src_seg_stride=64, dst_batch_stride=1024,
             dst_beam_stride=256, dst_seg_stride=64, segments=4, seg_bytes=64)
    a.update(kw)
    s = L.BeamState(**a)
    return lib.lilicorr_beam_reorder(None if null else C.byref(s), n, parent, batch, beams, None)


@pytest.mark.parametrize("kw", [
    dict(null=True), dict(n=0), dict(parent=None), dict(batch=0), dict(beams=0), dict(beams=33), dict(src=None), dict(dst=None),
    dict(segments=0), dict(seg_bytes=0), dict(seg_bytes=1 << 32), dict(src_beam_stride=-256), dict(dst_seg_stride=-1),
    dict(dst_beam_stride=0), dict(dst_beam_stride=128), dict(dst_seg_stride=32), dict(dst_batch_stride=512),
    dict(dst=(1 << 20) + 64), dict(dst=(1 << 20) - 64), dict(dst=1 << 20, dst_batch_stride=2048),
    dict(batch=1 << 20, seg_bytes=1 << 31, src_seg_stride=1 << 31, dst_seg_stride=1 << 31, src_beam_stride=1 << 33,
         dst_beam_stride=1 << 33, src_batch_stride=1 << 35, dst_batch_stride=1 << 35, dst=1 << 56)])
def test_reorder_refuses(lib, kw):
    assert reorder(lib, **kw) == INVALID


def test_reorder_refuses_strides_that_pass_64_bits(lib):
    apart = dict(src_batch_stride=1 << 45, dst_batch_stride=1 << 45, dst=1 << 40)
    assert reorder(lib, batch=1 << 20, **apart) == INVALID
    assert reorder(lib, batch=1 << 20, **{**apart, "src_batch_stride": 1024}) == INVALID
    assert reorder(lib, segments=1 << 32, src_seg_stride=1 << 40, dst_seg_stride=64, dst_batch_stride=1 << 41,
                   dst_beam_stride=1 << 39) == INVALID


def cache(**kw):
    from draft_block_candidate_gb300 import _lib as L
    a = dict(k_pages=FAKE, v_pages=FAKE, k_scale=FAKE, v_scale=FAKE, n_pages=10, kv_heads=2, page=64, head_dim=128)
    a.update(kw)
    return C.byref(L.Kv8CacheDesc(**a))


BATCH = dict(total=8, q_start=FAKE, kv_len=FAKE, batch=2, table=FAKE, table_stride=4, cols=4, max_new=4)
CACHE_BAD = [dict(k_pages=None), dict(v_pages=None), dict(k_scale=None), dict(v_scale=None), dict(n_pages=0),
             dict(n_pages=1 << 31), dict(kv_heads=0), dict(page=48), dict(page=256), dict(head_dim=96), dict(head_dim=256),
             dict(k_pages=FAKE + 8), dict(v_scale=FAKE + 2)]
BATCH_BAD = [dict(q_start=None), dict(kv_len=None), dict(table=None), dict(batch=0), dict(batch=1 << 21), dict(cols=0),
             dict(cols=1 << 26, table_stride=1 << 26), dict(table_stride=3), dict(total=-1), dict(total=1 << 31),
             dict(max_new=0), dict(max_new=1 << 25)]


def append(lib, c=None, k=FAKE, kt=256, kh=128, v=FAKE, vt=256, vh=128, **kw):
    a = dict(BATCH)
    a.update(kw)
    return lib.lilicorr_kv8_append(cache() if c is None else c, k, kt, kh, v, vt, vh, a["total"], a["q_start"], a["kv_len"],
                                   a["batch"], a["table"], a["table_stride"], a["cols"], a["max_new"], None, None)


@pytest.mark.parametrize("kw", BATCH_BAD + [
    dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(kt=252), dict(vh=4), dict(kt=-256), dict(vt=1 << 41),
    dict(batch=1 << 20, max_new=1 << 20, cols=1 << 20, table_stride=1 << 20)])
def test_append_refuses(lib, kw):
    assert append(lib, **kw) == INVALID


def attention(lib, c=None, q=FAKE, qt=1024, qh=128, heads=8, scale=0.1, out=FAKE, ws=FAKE, bytes=1 << 34, **kw):
    a = dict(BATCH)
    a.update(kw)
    return lib.lilicorr_kv8_attention(cache() if c is None else c, q, qt, qh, a["total"], heads, a["q_start"], a["kv_len"],
                                      a["batch"], a["table"], a["table_stride"], a["cols"], a["max_new"], scale, out, None, ws,
                                      bytes, None)


@pytest.mark.parametrize("kw", BATCH_BAD + [
    dict(q=None), dict(q=FAKE + 8), dict(qt=1020), dict(qh=4), dict(heads=0), dict(heads=7), dict(heads=2 * 1025),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None), dict(out=FAKE + 2)])
def test_attention_refuses(lib, kw):
    assert attention(lib, **kw) == INVALID


def test_attention_refuses_more_rows_than_32_bits_count(lib):
    assert attention(lib, cache(kv_heads=1), heads=1024, max_new=1 << 22) == INVALID
    assert lib.lilicorr_kv8_attention_workspace_bytes(1 << 22, 1024, 1, 128) == 0


@pytest.mark.parametrize("kw", CACHE_BAD)
def test_a_bad_cache_is_refused(lib, kw):
    assert append(lib, cache(**kw)) == INVALID
    assert attention(lib, cache(**kw)) == INVALID


def test_null_cache_is_refused(lib):
    assert lib.lilicorr_kv8_append(None, FAKE, 8, 8, FAKE, 8, 8, 1, FAKE, FAKE, 1, FAKE, 1, 1, 1, None, None) == INVALID


def test_attention_workspace(lib):
    f = lib.lilicorr_kv8_attention_workspace_bytes
    assert f(1, 8, 2, 128) > 0 and f(64, 64, 8, 64) > 0
    assert f(0, 8, 2, 128) == f(1, 7, 2, 128) == f(1, 8, 0, 128) == f(1, 8, 2, 96) == 0
    assert attention(lib, ws=None) == attention(lib, ws=FAKE + 64) == attention(lib, bytes=64) == WORKSPACE


def test_python_refuses_cpu_tensors_and_bad_layouts():
    import draft_block_candidate_gb300 as lc
    x = torch.zeros(2, 4, 100)
    with pytest.raises(ValueError):
        lc.beam_select(x, torch.zeros(2, 4), 4)
    with pytest.raises(ValueError):
        lc.beam_select(torch.zeros(8, 100), torch.zeros(2, 4), 4)
    with pytest.raises(ValueError):
        lc.beam_reorder([torch.zeros(2, 4, 3)], torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        lc.beam_reorder([], torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        lc.KV8Cache(4, 2, 64, 128, device="cpu")


@pytest.mark.parametrize("shape,a,b,want", [
    ((), (), (), (0, 0, 1, 4)), ((5,), (1,), (1,), (0, 0, 1, 20)), ((3, 5), (5, 1), (5, 1), (0, 0, 1, 60)),
    ((3, 5), (8, 1), (5, 1), (32, 20, 3, 20)), ((2, 3, 5), (24, 8, 1), (15, 5, 1), (32, 20, 6, 20)),
    ((2, 1, 5), (24, 7, 1), (5, 9, 1), (96, 20, 2, 20)), ((2, 3, 5), (25, 8, 1), (15, 5, 1), None),
    ((4,), (2,), (2,), (8, 8, 4, 4))])
def test_state_layouts(shape, a, b, want):
    from draft_block_candidate_gb300.decode import _state_layout
    assert _state_layout(shape, a, b, 4) == want
