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
