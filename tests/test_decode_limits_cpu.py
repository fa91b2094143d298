"""Refusals of the decoding entry points where memory is shared or a number does not fit, before anything touches a device."""
import ctypes as C

from tests.test_decode_cpu import BATCH, FAKE, INVALID, attention, cache, lib  # noqa: F401


def states(*pairs):
    from draft_block_candidate_gb300 import _lib as L
    return (L.BeamState * len(pairs))(*[
        L.BeamState(src=s << 20, dst=d << 20, src_batch_stride=1024, src_beam_stride=256, src_seg_stride=64,
                    dst_batch_stride=1024, dst_beam_stride=256, dst_seg_stride=64, segments=4, seg_bytes=64) for s, d in pairs])


def test_reorder_refuses_one_state_twice(lib):  # noqa: F811
    for pairs in ([(1, 1), (1, 1)], [(1, 2), (3, 2)], [(1, 2), (2, 1)], [(1, 2), (2, 3)], [(5, 6), (1, 2), (7, 7), (3, 2)], [(1, 1), (1, 2)]):
        assert lib.lilicorr_beam_reorder(C.byref(states(*pairs)), len(pairs), FAKE, 2, 4, None) == INVALID, pairs


def test_attention_refuses_to_write_over_its_queries(lib):  # noqa: F811
    span = (7 * 1024 + 7 * 128 + 128) * 2  # bytes of q's 8 rows of 8 heads
    for q in (FAKE, FAKE + span - 16, FAKE - span + 16):
        assert attention(lib, q=q + (1 << 30), out=FAKE + (1 << 30)) == INVALID
    a = BATCH
    for out, lse in ((2 << 30, (1 << 30) + 64), (2 << 30, (2 << 30) + 8 * 8 * 128 * 2 - 4), (2 << 30, (2 << 30) - 8 * 8 * 4 + 4)):
        assert lib.lilicorr_kv8_attention(cache(), 1 << 30, 1024, 128, a["total"], 8, a["q_start"], a["kv_len"], a["batch"], a["table"],
                                          a["table_stride"], a["cols"], a["max_new"], 0.1, out, lse, FAKE, 1 << 34, None) == INVALID
