"""ctypes declarations of the C ABI in include/lilicorr.h (no logic here)."""
from __future__ import annotations

import ctypes as C
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblilicorr.so")

F32, BF16 = 0, 1

STATUS = {
    0: "LILICORR_OK", 1: "LILICORR_ERR_INVALID_ARG", 2: "LILICORR_ERR_UNSUPPORTED",
    3: "LILICORR_ERR_WEIGHTS_MISSING", 4: "LILICORR_ERR_WEIGHTS_SURPLUS",
    5: "LILICORR_ERR_WEIGHTS_SHAPE", 6: "LILICORR_ERR_CUDA", 7: "LILICORR_ERR_WORKSPACE",
    8: "LILICORR_ERR_DEVICE",
}

# Every function the header declares, with (restype, argtypes).
_P = C.c_void_p
SIGNATURES = {
    "lilicorr_weights_create": (C.c_int, [_P, _P, C.c_int32, C.c_int, C.POINTER(C.c_void_p)]),
    "lilicorr_weights_destroy": (None, [_P]),
    "lilicorr_weights_dims": (C.c_int, [_P, _P]),
    "lilicorr_workspace_bytes": (C.c_size_t, [_P, C.c_int64, C.c_int32, C.c_int32]),
    "lilicorr_rerank": (C.c_int, [_P, _P, C.c_int, C.c_int64, C.c_int32, C.c_int64, C.c_int32,
                                  _P, _P, _P, _P, _P, _P, _P, C.c_size_t, _P]),
    "lilicorr_workspace_bytes_host": (C.c_size_t, [_P, C.c_int64, C.c_int32, C.c_int32, C.c_int]),
    "lilicorr_rerank_host": (C.c_int, [_P, _P, C.c_int, C.c_int64, C.c_int32, C.c_int64,
                                       C.c_int32, _P, _P, _P, _P, _P, _P, C.c_size_t, _P]),
    "lilicorr_topk_lse_workspace_bytes": (C.c_size_t, [C.c_int64, C.c_int32, C.c_int64,
                                                       C.c_int32, C.c_int]),
    "lilicorr_topk_lse": (C.c_int, [_P, C.c_int, C.c_int64, C.c_int32, C.c_int64, C.c_int32,
                                    _P, _P, _P, _P, C.c_size_t, _P]),
    "lilicorr_topk_lse_noalloc": (C.c_int, [_P, C.c_int, C.c_int64, C.c_int32, C.c_int64,
                                            C.c_int32, _P, _P, _P, _P]),
    "lilicorr_greedy_walk": (C.c_int, [_P, _P, _P, C.c_int64, C.c_int32, C.c_int32, _P, _P, _P,
                                       _P]),
    "lilicorr_viterbi": (C.c_int, [_P, _P, _P, C.c_int64, C.c_int32, C.c_int32, _P, _P, _P, _P,
                                   _P]),
    "lilicorr_sample_walk": (C.c_int, [_P, _P, _P, _P, _P, C.c_int64, C.c_int32, C.c_int32,
                                       _P, _P, _P, _P, _P]),
    "lilicorr_topk_lse_shard_record_bytes": (C.c_size_t, [C.c_int32]),
    "lilicorr_topk_lse_shard": (C.c_int, [_P, C.c_int, C.c_int64, C.c_int32, C.c_int64,
                                          C.c_int64, C.c_int64, C.c_int32, _P, _P, C.c_size_t,
                                          _P]),
    "lilicorr_topk_lse_merge": (C.c_int, [_P, C.c_int32, C.c_int64, C.c_int32, _P, _P, _P, _P]),
    "lilicorr_lm_head_workspace_bytes": (C.c_size_t, [C.c_int64, C.c_int64, C.c_int32,
                                                      C.c_int32]),
    "lilicorr_lm_head_topk_lse": (C.c_int, [_P, _P, C.c_int64, C.c_int64, C.c_int32, C.c_int32,
                                            _P, _P, _P, _P, C.c_size_t, _P]),
    "lilicorr_beam_select_workspace_bytes": (C.c_size_t, [C.c_int64, C.c_int32, C.c_int64,
                                                          C.c_int32, C.c_int]),
    "lilicorr_beam_select": (C.c_int, [_P, C.c_int, C.c_int64, C.c_int32, C.c_int64, C.c_int64,
                                       C.c_int32, _P, _P, C.c_int32, _P, _P, _P, _P, C.c_size_t,
                                       _P]),
    "lilicorr_beam_reorder": (C.c_int, [_P, C.c_int32, _P, C.c_int64, C.c_int32, _P]),
    "lilicorr_kv8_append": (C.c_int, [_P, _P, C.c_int64, C.c_int64, _P, C.c_int64, C.c_int64,
                                      C.c_int64, _P, _P, C.c_int64, _P, C.c_int64, C.c_int32,
                                      C.c_int32, _P, _P]),
    "lilicorr_kv8_attention_workspace_bytes": (C.c_size_t, [C.c_int32, C.c_int32, C.c_int32,
                                                            C.c_int32]),
    "lilicorr_kv8_attention": (C.c_int, [_P, _P, C.c_int64, C.c_int64, C.c_int64, C.c_int32, _P,
                                         _P, C.c_int64, _P, C.c_int64, C.c_int32, C.c_int32,
                                         C.c_float, _P, _P, _P, C.c_size_t, _P]),
    "lilicorr_adjust_logits": (C.c_int, [_P, _P]),
    "lilicorr_kv8_pages_workspace_bytes": (C.c_size_t, [C.c_int64, C.c_int64]),
    "lilicorr_kv8_fork": (C.c_int, [_P, C.c_int64, _P, C.c_int64, C.c_int64, C.c_int32, _P, C.c_int64,
                                    C.c_int32, _P]),
    "lilicorr_kv8_grow": (C.c_int, [_P, C.c_int64, _P, C.c_int64, C.c_int64, C.c_int32, _P, _P,
                                    C.c_int32, C.c_int32, _P, _P, _P, C.c_size_t, _P]),
    "lilicorr_kv8_free": (C.c_int, [_P, C.c_int64, _P, C.c_int64, C.c_int64, C.c_int32, _P, C.c_int32,
                                    _P]),
    "lilicorr_kv8_copy": (C.c_int, [_P, _P, C.c_int32, _P, _P, C.c_int64, _P]),
    "lilicorr_kv8_compact": (C.c_int, [_P, C.c_int32, _P, _P, C.c_int64, _P, C.c_int32, _P, _P,
                                       C.c_size_t, _P]),
    "lilicorr_cross_attention_workspace_bytes": (C.c_size_t, [C.c_int32]),
    "lilicorr_cross_attention": (C.c_int, [_P, C.c_int64, C.c_int64, C.c_int64, C.c_int32,
                                           _P, C.c_int64, C.c_int64, _P, C.c_int64, C.c_int64, C.c_int64,
                                           C.c_int32, C.c_int32, _P, _P, _P, C.c_int64, C.c_int32,
                                           C.c_float, _P, _P, _P, C.c_size_t, _P]),
    "lilicorr_status_string": (C.c_char_p, [C.c_int]),
    "lilicorr_last_error": (C.c_char_p, []),
    "lilicorr_launch_count": (C.c_uint64, []),
    "lilicorr_device_error": (C.c_int, [C.POINTER(C.c_uint32)]),
    "lilicorr_diag_wait_timeout": (C.c_int, [_P, C.c_int64, C.c_uint32, _P, _P, _P, _P]),
    "lilicorr_stage_timing": (None, [C.c_int]),
    "lilicorr_stage_times": (C.c_int32, [C.POINTER(C.c_double), C.POINTER(C.c_int64),
                                         C.c_int32, C.POINTER(C.c_int64)]),
    "lilicorr_stage_name": (C.c_char_p, [C.c_int32]),
}


class Dims(C.Structure):
    _fields_ = [("layers", C.c_int32), ("hidden", C.c_int32), ("heads", C.c_int32),
                ("ffn", C.c_int32), ("d_e", C.c_int32), ("B_max", C.c_int32),
                ("K_max", C.c_int32), ("V", C.c_int64), ("sigma", C.c_float),
                ("rms_eps", C.c_float)]


class Tensor(C.Structure):
    _fields_ = [("name", C.c_char_p), ("host_data", C.c_void_p), ("dtype", C.c_int),
                ("ndim", C.c_int32), ("shape", C.c_int64 * 4)]


class BeamState(C.Structure):
    _fields_ = [("src", C.c_void_p), ("dst", C.c_void_p)] + [
        (n, C.c_int64) for n in ("src_batch_stride", "src_beam_stride", "src_seg_stride",
                                 "dst_batch_stride", "dst_beam_stride", "dst_seg_stride",
                                 "segments", "seg_bytes")]


class Kv8CacheDesc(C.Structure):
    _fields_ = [("k_pages", C.c_void_p), ("v_pages", C.c_void_p), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("n_pages", C.c_int64), ("kv_heads", C.c_int32),
                ("page", C.c_int32), ("head_dim", C.c_int32)]


class Adjust(C.Structure):
    _fields_ = ([("logits", C.c_void_p), ("out", C.c_void_p), ("ldtype", C.c_int)]
                + [(n, C.c_int64) for n in ("rows", "V", "row_stride", "out_stride", "groups")]
                + [("history", C.c_void_p), ("history_stride", C.c_int64), ("cap", C.c_int32)]
                + [(n, C.c_void_p) for n in ("seen", "counted_from", "repetition", "presence",
                                             "frequency", "bias_id", "bias")]
                + [("n_bias", C.c_int32), ("mask", C.c_void_p), ("n_masks", C.c_int64),
                   ("mask_stride", C.c_int64), ("mask_index", C.c_void_p)])


class Kv8Table(C.Structure):
    _fields_ = [("table", C.c_void_p), ("out", C.c_void_p), ("rows", C.c_int64),
                ("row_stride", C.c_int64), ("out_stride", C.c_int64), ("cols", C.c_int32)]


class Taps(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("choice", "cand_id", "cand_logit", "lse",
                                          "pair_scores", "nodes", "hidden", "out_vec",
                                          "in_vec", "anchor_vec")]


_lib = None


def lib():
    """The loaded library.  Raises if it has not been built: there is no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(nvcc, sm_103a); the rerank has no non-CUDA path")
        h = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib
