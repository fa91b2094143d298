"""Refusals of the decoding entry points where memory is shared or a number does not fit, before anything touches a device."""
import ctypes as C

from tests.test_decode_cpu import FAKE, INVALID, attention, lib, reorder  # noqa: F401


def states(*pairs):
    from draft_block_candidate_gb300 import _lib as L
    return (L.BeamState * len(pairs))(*[
        L.BeamState(src=s << 20, dst=d << 20, src_batch_stride=1024, src_beam_stride=256, src_seg_stride=64,
                    dst_batch_stride=1024, dst_beam_stride=256, dst_seg_stride=64, segments=4, seg_bytes=64) for s, d in pairs])


def test_reorder_refuses_one_state_twice(lib):  # noqa: F811
    for pairs in ([(1, 1), (1, 1)], [(1, 2), (3, 2)], [(1, 2), (2, 1)], [(1, 2), (2, 3)], [(5, 6), (1, 2), (7, 7), (3, 2)], [(1, 1), (1, 2)]):
        assert lib.lilicorr_beam_reorder(C.byref(states(*pairs)), len(pairs), FAKE, 2, 4, None) == INVALID, pairs
