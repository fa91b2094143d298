"""What the operators around the loop take and refuse at their limits, before anything touches a device."""
import ctypes as C

import pytest
import torch

INVALID = 1


@pytest.mark.parametrize("shape", [(0, 100), (4, 0, 100), (0, 3, 100), (2, 0, 5, 7), (3, 0, 0)])
def test_rows_of_an_empty_tensor(shape):
    """No rows have any layout, whichever extent is 0."""
    from draft_block_candidate_gb300.logits import _logit_rows
    assert _logit_rows(torch.zeros(shape), "logits") == (0, shape[-1], shape[-1])


FAR = 1 << 32


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from draft_block_candidate_gb300 import _lib
    return _lib.lib()


def adjust(lib, **kw):
    """A call whose arrays lie far apart."""
    from draft_block_candidate_gb300 import _lib as L
    a = dict(logits=FAR, out=FAR, ldtype=1, rows=8, V=1000, row_stride=1024, out_stride=1024, groups=4, history=2 * FAR, history_stride=64, cap=50,
             seen=3 * FAR, counted_from=4 * FAR, repetition=5 * FAR, presence=6 * FAR, frequency=7 * FAR, bias_id=8 * FAR, bias=9 * FAR, n_bias=3,
             mask=10 * FAR, n_masks=5, mask_stride=40, mask_index=11 * FAR)
    a.update(kw)
    return lib.lilicorr_adjust_logits(C.byref(L.Adjust(**a)), None)


# (array, its bytes); rows of the logits are 2,000 bytes (1,000 of bf16), 2,048 apart
ARRAYS = [("history", (3 * 64 + 50) * 4), ("seen", 32), ("counted_from", 16), ("repetition", 16), ("presence", 16), ("frequency", 16), ("bias_id", 48),
          ("bias", 48), ("mask", (4 * 40 + 32) * 4), ("mask_index", 32)]


@pytest.mark.parametrize("name,size", ARRAYS)
@pytest.mark.parametrize("out", [FAR, 13 * FAR])
def test_adjust_refuses_to_write_what_it_reads(lib, name, size, out):
    """In place and apart: at the first and last byte of the rows, across a row's beginning, within one."""
    for at in (out - size + 4, out, out + 1996, out + 2048 - size + 4, out + 3000, out + 7 * 2048 + 1996):
        assert adjust(lib, out=out, **{name: at}) == INVALID, at - out


@pytest.mark.parametrize("name", [n for n, _ in ARRAYS])
def test_adjust_refuses_misaligned_arrays(lib, name):
    at = (2 + [n for n, _ in ARRAYS].index(name)) * FAR
    assert adjust(lib, **{name: at + 2}) == INVALID


@pytest.mark.parametrize("name", ["kv", "new", "tail"])
def test_grow_refuses_misaligned_arrays(lib, name):
    a = dict(kv=3 * FAR, new=4 * FAR, tail=5 * FAR)
    a[name] += 2
    assert lib.lilicorr_kv8_grow(FAR, 100, 2 * FAR, 4, 8, 8, a["kv"], a["new"], 64, 4, a["tail"], 6 * FAR, 7 * FAR, 1 << 20, None) == INVALID


def cross(lib, **kw):
    """(status, message) of a call whose arrays lie far apart."""
    a = dict(q=FAR, k=2 * FAR, v=3 * FAR, q_start=4 * FAR, kv_start=5 * FAR, kv_len=6 * FAR, out=8 * FAR, lse=9 * FAR)
    a.update(kw)
    st = lib.lilicorr_cross_attention(a["q"], 1024, 128, 8, 8, a["k"], 512, 128, a["v"], 512, 128, 100, 2, 128, a["q_start"], a["kv_start"], a["kv_len"],
                                      2, 4, 0.1, a["out"], a["lse"], 10 * FAR, 1 << 30, None)
    return st, lib.lilicorr_last_error()  # (without a GPU's driver there is no tensor map, which is refused alike)


@pytest.mark.parametrize("name", ["q_start", "kv_start", "kv_len", "lse"])
def test_cross_refuses_misaligned_arrays(lib, name):
    at = dict(q_start=4, kv_start=5, kv_len=6, lse=9)[name] * FAR
    st, why = cross(lib, **{name: at + 2})
    assert st == INVALID and b"4-byte aligned" in why


@pytest.mark.parametrize("name,size", [("q_start", 12), ("kv_start", 8), ("kv_len", 8)])
def test_cross_refuses_to_write_what_it_reads(lib, name, size):
    """At the first and the last word of out (8 x 8 x 128 bf16) and of lse (8 x 8)."""
    for at in (8 * FAR + 4 - size, 8 * FAR + 8 * 8 * 128 * 2 - 4, 9 * FAR + 4 - size, 9 * FAR + 8 * 8 * 4 - 4):
        st, why = cross(lib, **{name: at})
        assert st == INVALID and b"overlap" in why


@pytest.mark.parametrize("name", ["q_start", "kv_len", "table", "lse", "tail"])
def test_the_cache_refuses_misaligned_arrays(lib, name):
    from draft_block_candidate_gb300 import _lib as L
    cache = C.byref(L.Kv8CacheDesc(k_pages=FAR, v_pages=2 * FAR, k_scale=3 * FAR, v_scale=4 * FAR, n_pages=10, kv_heads=2, page=64, head_dim=128))
    a = dict(q_start=5 * FAR, kv_len=6 * FAR, table=7 * FAR, lse=8 * FAR, tail=9 * FAR)
    a[name] += 2
    if name != "tail":
        assert lib.lilicorr_kv8_attention(cache, 10 * FAR, 1024, 128, 8, 8, a["q_start"], a["kv_len"], 2, a["table"], 4, 4, 4, 0.1, 11 * FAR, a["lse"],
                                          12 * FAR, 1 << 30, None) == INVALID
    if name != "lse":
        assert lib.lilicorr_kv8_append(cache, 10 * FAR, 256, 128, 11 * FAR, 256, 128, 8, a["q_start"], a["kv_len"], 2, a["table"], 4, 4, 4, a["tail"],
                                       None) == INVALID
