"""Thin Python binding of the C ABI in include/decode_attn.h (argument marshalling only).

Every step of the computation runs in the CUDA library libdecode_attn.so; this module
only converts arguments and raises DecodeAttnError for non-zero return codes. PyTorch is
used for device memory and streams. If the library has not been built this module raises
on first use: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
from typing import Optional

from . import build as _build

DA_F32, DA_F16, DA_BF16 = 0, 1, 2
DA_SOFTMAX_SYNC, DA_SOFTMAX_UNIFIED, DA_SOFTMAX_UNIFIED_LOCAL = 0, 1, 2
ERRORS = {0: "DA_OK", -1: "DA_ERR_INVALID_ARG", -2: "DA_ERR_UNSUPPORTED",
          -3: "DA_ERR_WORKSPACE_TOO_SMALL", -4: "DA_ERR_BAD_BLOCK_TABLE", -5: "DA_ERR_CUDA",
          -6: "DA_ERR_DEVICE_TIMEOUT", -7: "DA_ERR_BAD_SEQ_LEN", -8: "DA_ERR_HISTOGRAM_RANGE",
          -9: "DA_ERR_RANGE_TOO_WIDE", -10: "DA_ERR_NO_PAGES"}
DA_ERR_RANGE_TOO_WIDE = -9
MAX_HIST_BINS = 32768
MAX_TREE = 64
POOL_HEAD = 4
ADAPTER_PARTS = 4
DTYPE_CODES = {"f32": DA_F32, "f16": DA_F16, "bf16": DA_BF16}
ROPE_CODES = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3, "by_index": 4}
SCALING_CODES = {"tensor": 1, "row": 2, "group": 3}
MODE_CODES = {"sync": DA_SOFTMAX_SYNC, "unified": DA_SOFTMAX_UNIFIED,
              "unified_local": DA_SOFTMAX_UNIFIED_LOCAL}


class DecodeAttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {ERRORS.get(code, code)}: {decode_attn_strerror(code)}")


class da_problem(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int),
        ("num_q_heads", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("paged", ctypes.c_int),
        ("page_size", ctypes.c_int),
        ("max_blocks_per_seq", ctypes.c_int),
        ("num_physical_blocks", ctypes.c_int),
        ("max_seq_len", ctypes.c_int),
        ("qkv_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("mode", ctypes.c_int),
        ("unified_max", ctypes.c_float),
        ("range_lo", ctypes.c_float),
        ("range_hi", ctypes.c_float),
        ("validate", ctypes.c_int),
        ("num_sms", ctypes.c_int),
        ("kv_fp8", ctypes.c_int),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("debug_stall_stage", ctypes.c_int),
    ]


class da_plan_info(ctypes.Structure):
    _fields_ = [
        ("grid_ctas", ctypes.c_int),
        ("num_splits", ctypes.c_int),
        ("unit_tokens", ctypes.c_int),
        ("stage_tokens", ctypes.c_int),
        ("stages", ctypes.c_int),
        ("recompute_splits", ctypes.c_int),
        ("max_splits", ctypes.c_int),
        ("workspace_bytes", ctypes.c_size_t),
        ("smem_bytes", ctypes.c_size_t),
        ("split_tokens", ctypes.c_int),
        ("split_tokens_min", ctypes.c_int),
        ("kv_heads_per_group", ctypes.c_int),
    ]


class da_stats(ctypes.Structure):
    _fields_ = [
        ("grid_ctas", ctypes.c_int),
        ("num_splits", ctypes.c_int),
        ("rows_flagged", ctypes.c_longlong),
        ("splits_flagged", ctypes.c_longlong),
        ("recompute_launched", ctypes.c_int),
        ("split_tokens", ctypes.c_int),
        ("split_tokens_min", ctypes.c_int),
    ]


class da_run_args(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("scale", ctypes.c_float),
        ("num_splits", ctypes.c_int),
        ("out", ctypes.c_void_p),
        ("out_lse", ctypes.c_void_p),
        ("row_flags", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("cuda_stream", ctypes.c_void_p),
        ("stats", ctypes.POINTER(da_stats)),
        ("split_event_begin", ctypes.c_void_p),
        ("split_event_end", ctypes.c_void_p),
    ]


class da_rope_config(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int),
        ("rotary_dim", ctypes.c_int),
        ("interleaved", ctypes.c_int),
        ("scaling", ctypes.c_int),
        ("base", ctypes.c_double),
        ("factor", ctypes.c_double),
        ("original_max_position", ctypes.c_double),
        ("low", ctypes.c_double),
        ("high", ctypes.c_double),
        ("attn_factor", ctypes.c_double),
    ]


class da_rope_args(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("dtype", ctypes.c_int),
        ("rows", ctypes.c_int),
        ("heads", ctypes.c_int),
        ("x_row_stride", ctypes.c_int64),
        ("x_head_stride", ctypes.c_int64),
        ("out_row_stride", ctypes.c_int64),
        ("out_head_stride", ctypes.c_int64),
        ("positions", ctypes.c_void_p),
        ("transpose", ctypes.c_int),
        ("cuda_stream", ctypes.c_void_p),
    ]


class da_kv_write_args(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_row_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v_row_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("rows", ctypes.c_int),
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("row_offsets", ctypes.c_void_p),
        ("start", ctypes.c_void_p),
        ("rope", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
        ("q", ctypes.c_void_p),
        ("q_out", ctypes.c_void_p),
        ("q_row_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("q_out_row_stride", ctypes.c_int64),
        ("q_out_head_stride", ctypes.c_int64),
        ("amax", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("cuda_stream", ctypes.c_void_p),
    ]


class da_kv_read_args(ctypes.Structure):
    _fields_ = [
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("row_offsets", ctypes.c_void_p),
        ("start", ctypes.c_void_p),
        ("rows", ctypes.c_int),
        ("k_out", ctypes.c_void_p),
        ("v_out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("cuda_stream", ctypes.c_void_p),
    ]


class da_tree_plan_info(ctypes.Structure):
    _fields_ = [
        ("grid_ctas", ctypes.c_int),
        ("row_tiles", ctypes.c_int),
        ("tile_rows", ctypes.c_int),
        ("tile_tokens", ctypes.c_int),
        ("stages", ctypes.c_int),
        ("max_tree", ctypes.c_int),
        ("workspace_bytes", ctypes.c_size_t),
        ("smem_bytes", ctypes.c_size_t),
    ]


class da_tree_args(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("row_offsets", ctypes.c_void_p),
        ("ctx_lens", ctypes.c_void_p),
        ("tree_mask", ctypes.c_void_p),
        ("rows", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("out", ctypes.c_void_p),
        ("out_lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("cuda_stream", ctypes.c_void_p),
    ]


class da_pages_reserve_args(ctypes.Structure):
    _fields_ = [
        ("pool", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("row_offsets", ctypes.c_void_p),
        ("ctx_lens", ctypes.c_void_p),
        ("rows", ctypes.c_int),
        ("seq_lens", ctypes.c_void_p),
        ("slots", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("cuda_stream", ctypes.c_void_p),
    ]


class da_pages_release_args(ctypes.Structure):
    _fields_ = [
        ("pool", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("keep_lens", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("cuda_stream", ctypes.c_void_p),
    ]


class da_norm_config(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int),
        ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
    ]


class da_norm_args(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("residual", ctypes.c_void_p),
        ("weight", ctypes.c_void_p),
        ("residual_out", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("dtype", ctypes.c_int),
        ("weight_f32", ctypes.c_int),
        ("scaling", ctypes.c_int),
        ("group", ctypes.c_int),
        ("rows", ctypes.c_int),
        ("heads", ctypes.c_int),
        ("x_row_stride", ctypes.c_int64),
        ("x_head_stride", ctypes.c_int64),
        ("residual_row_stride", ctypes.c_int64),
        ("residual_head_stride", ctypes.c_int64),
        ("residual_out_row_stride", ctypes.c_int64),
        ("residual_out_head_stride", ctypes.c_int64),
        ("out_row_stride", ctypes.c_int64),
        ("out_head_stride", ctypes.c_int64),
        ("codes_row_stride", ctypes.c_int64),
        ("codes_head_stride", ctypes.c_int64),
        ("cuda_stream", ctypes.c_void_p),
    ]


class da_adapter_config(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("width", ctypes.c_int),
        ("parts", ctypes.c_int),
        ("out_sizes", ctypes.c_int * ADAPTER_PARTS),
        ("rank", ctypes.c_int),
    ]


class da_adapter_args(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("a", ctypes.c_void_p),
        ("b", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("row_offsets", ctypes.c_void_p),
        ("adapter_ids", ctypes.c_void_p),
        ("rows", ctypes.c_int),
        ("batch", ctypes.c_int),
        ("adapters", ctypes.c_int),
        ("x_row_stride", ctypes.c_int64),
        ("y_row_stride", ctypes.c_int64),
        ("out_row_stride", ctypes.c_int64),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("cuda_stream", ctypes.c_void_p),
    ]


_lib = None
P = ctypes.c_void_p


def library_path() -> str:
    return _build.LIB


def lib():
    """Load libdecode_attn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(path)
        L.decode_attn_plan.argtypes = [ctypes.POINTER(da_problem), ctypes.c_int,
                                       ctypes.POINTER(P), ctypes.POINTER(ctypes.c_size_t)]
        L.decode_attn_plan_info.argtypes = [P, ctypes.POINTER(da_plan_info)]
        L.decode_attn_workspace_init.argtypes = [P, P, ctypes.c_size_t, P]
        L.decode_attn_run.argtypes = [P, P, P, P, P, P, ctypes.c_float, ctypes.c_int, P, P, P,
                                      P, ctypes.c_size_t, P, ctypes.POINTER(da_stats)]
        L.decode_attn_run_ex.argtypes = [P, ctypes.POINTER(da_run_args)]
        L.decode_attn_run_static.argtypes = [P, P, P, P, P, P, ctypes.c_float, ctypes.c_int, P,
                                             P, P, P, ctypes.POINTER(da_stats)]
        L.decode_attn_check_status.argtypes = [P, P, P]
        L.decode_attn_debug_gather.argtypes = [P, P, P, P, P]
        L.decode_attn_logit_histogram.argtypes = [P, P, P, P, P, ctypes.c_float, ctypes.c_float,
                                                  ctypes.c_float, ctypes.c_int, P, P]
        F = ctypes.POINTER(ctypes.c_float)
        L.decode_attn_choose_phi.argtypes = [ctypes.POINTER(ctypes.c_ulonglong), ctypes.c_int,
                                             ctypes.c_float, ctypes.c_float, ctypes.c_double,
                                             ctypes.c_float, F, F, F]
        L.decode_attn_rope_create.argtypes = [ctypes.POINTER(da_rope_config), ctypes.POINTER(P)]
        L.decode_attn_rope_frequencies.argtypes = [P, ctypes.POINTER(ctypes.c_double)]
        L.decode_attn_rope_apply.argtypes = [P, ctypes.POINTER(da_rope_args)]
        L.decode_attn_kv_write.argtypes = [P, ctypes.POINTER(da_kv_write_args)]
        L.decode_attn_kv_read.argtypes = [P, ctypes.POINTER(da_kv_read_args)]
        L.decode_attn_tree_plan.argtypes = [ctypes.POINTER(da_problem), ctypes.c_int,
                                            ctypes.POINTER(P), ctypes.POINTER(ctypes.c_size_t)]
        L.decode_attn_tree_plan_info.argtypes = [P, ctypes.POINTER(da_tree_plan_info)]
        L.decode_attn_tree_debug_stall.argtypes = [P, ctypes.c_int]
        L.decode_attn_tree_workspace_init.argtypes = [P, P, ctypes.c_size_t, P]
        L.decode_attn_tree_run.argtypes = [P, ctypes.POINTER(da_tree_args)]
        L.decode_attn_tree_check_status.argtypes = [P, P, P]
        L.decode_attn_tree_destroy.argtypes = [P]
        L.decode_attn_tree_destroy.restype = None
        L.decode_attn_pages_init.argtypes = [P, P, P]
        L.decode_attn_pages_reserve.argtypes = [P, ctypes.POINTER(da_pages_reserve_args)]
        L.decode_attn_pages_release.argtypes = [P, ctypes.POINTER(da_pages_release_args)]
        L.decode_attn_norm_apply.argtypes = [ctypes.POINTER(da_norm_config), ctypes.POINTER(da_norm_args)]
        L.decode_attn_adapters_apply.argtypes = [ctypes.POINTER(da_adapter_config),
                                                 ctypes.POINTER(da_adapter_args)]
        L.decode_attn_adapters_workspace.argtypes = [ctypes.POINTER(da_adapter_config), ctypes.c_int,
                                                     ctypes.POINTER(ctypes.c_size_t)]
        L.decode_attn_adapters_check_status.argtypes = [P, P]
        L.decode_attn_rope_destroy.argtypes = [P]
        L.decode_attn_rope_destroy.restype = None
        L.decode_attn_destroy.argtypes = [P]
        L.decode_attn_destroy.restype = None
        L.decode_attn_strerror.argtypes = [ctypes.c_int]
        L.decode_attn_strerror.restype = ctypes.c_char_p
        L.decode_attn_abi_version.argtypes = []
        for name in ("decode_attn_plan", "decode_attn_plan_info", "decode_attn_workspace_init",
                     "decode_attn_run", "decode_attn_run_ex", "decode_attn_run_static",
                     "decode_attn_check_status",
                     "decode_attn_debug_gather", "decode_attn_logit_histogram",
                     "decode_attn_choose_phi",
                     "decode_attn_rope_create", "decode_attn_rope_frequencies",
                     "decode_attn_rope_apply", "decode_attn_kv_write", "decode_attn_kv_read",
                     "decode_attn_tree_plan", "decode_attn_tree_plan_info",
                     "decode_attn_tree_debug_stall",
                     "decode_attn_tree_workspace_init", "decode_attn_tree_run",
                     "decode_attn_tree_check_status", "decode_attn_pages_init",
                     "decode_attn_pages_reserve", "decode_attn_pages_release",
                     "decode_attn_norm_apply", "decode_attn_adapters_apply",
                     "decode_attn_adapters_workspace", "decode_attn_adapters_check_status",
                     "decode_attn_abi_version"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int, where: str):
    if rc != 0:
        raise DecodeAttnError(rc, where)


def header_symbols() -> list:
    """Entry points declared in include/decode_attn.h."""
    path = os.path.join(_build.INCLUDE, "decode_attn.h")
    with open(path) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(decode_attn_[a-z_]+)\s*\(", text)))


# ---- the C entry points, same names ---------------------------------------------------------
def decode_attn_abi_version() -> int:
    return lib().decode_attn_abi_version()


def decode_attn_strerror(code: int) -> str:
    return lib().decode_attn_strerror(code).decode()


def decode_attn_plan(problem: da_problem, num_splits: int = 0):
    """Returns (plan handle, workspace bytes)."""
    plan = P()
    ws = ctypes.c_size_t()
    _check(lib().decode_attn_plan(ctypes.byref(problem), num_splits, ctypes.byref(plan),
                                  ctypes.byref(ws)), "decode_attn_plan")
    return plan, ws.value


def decode_attn_plan_info(plan) -> da_plan_info:
    info = da_plan_info()
    _check(lib().decode_attn_plan_info(plan, ctypes.byref(info)), "decode_attn_plan_info")
    return info


def decode_attn_workspace_init(plan, workspace: int, workspace_bytes: int, stream: int = 0):
    _check(lib().decode_attn_workspace_init(plan, workspace, workspace_bytes, stream or None),
           "decode_attn_workspace_init")


def decode_attn_run(plan, q: int, k_cache: int, v_cache: int, block_table: Optional[int],
                    seq_lens: int, scale: float, num_splits: int, out: int,
                    out_lse: Optional[int], row_flags: Optional[int], workspace: int,
                    workspace_bytes: int, stream: int = 0, want_stats: bool = False):
    """Pointers are integers (device addresses). Returns da_stats when want_stats."""
    st = da_stats() if want_stats else None
    _check(lib().decode_attn_run(plan, q, k_cache, v_cache, block_table or None, seq_lens,
                                 scale, num_splits, out, out_lse or None, row_flags or None,
                                 workspace, workspace_bytes, stream or None,
                                 ctypes.byref(st) if st is not None else None),
           "decode_attn_run")
    return st


def decode_attn_run_ex(plan, args: da_run_args):
    _check(lib().decode_attn_run_ex(plan, ctypes.byref(args)), "decode_attn_run_ex")


def decode_attn_run_static(plan, q: int, k_cache: int, v_cache: int, block_table: Optional[int],
                           seq_lens: int, scale: float, num_splits: int, out: int,
                           out_lse: Optional[int], row_flags: Optional[int], stream: int = 0,
                           want_stats: bool = False):
    """decode_attn_run on the library's fixed per-device scratch: for callers that cannot
    allocate a workspace. Pointers are integers (device addresses); nothing is allocated
    here either. Returns da_stats when want_stats."""
    st = da_stats() if want_stats else None
    _check(lib().decode_attn_run_static(plan, q, k_cache, v_cache, block_table or None,
                                        seq_lens, scale, num_splits, out, out_lse or None,
                                        row_flags or None, stream or None,
                                        ctypes.byref(st) if st is not None else None),
           "decode_attn_run_static")
    return st


def decode_attn_check_status(plan, workspace: int, stream: int = 0):
    _check(lib().decode_attn_check_status(plan, workspace, stream or None),
           "decode_attn_check_status")


def decode_attn_debug_gather(plan, block_table: Optional[int], seq_lens: int, offsets_out: int,
                             stream: int = 0):
    _check(lib().decode_attn_debug_gather(plan, block_table or None, seq_lens, offsets_out,
                                          stream or None), "decode_attn_debug_gather")


def decode_attn_logit_histogram(plan, q: int, k_cache: int, block_table: Optional[int],
                                seq_lens: int, scale: float, lo: float, hi: float, nbins: int,
                                counts: int, stream: int = 0):
    """Accumulate the histogram of one step's scaled logits into the device uint64 buffer
    `counts` ([nbins + 2]: below lo, the nbins bins of [lo, hi), at or above hi)."""
    _check(lib().decode_attn_logit_histogram(plan, q, k_cache, block_table or None, seq_lens,
                                             scale, lo, hi, nbins, counts, stream or None),
           "decode_attn_logit_histogram")


def decode_attn_choose_phi(counts, lo: float, hi: float, coverage: float = 0.9999,
                           max_width: float = float("inf")):
    """(phi, x_lo, x_hi, applies) from a host histogram (a sequence of nbins + 2 counts).
    applies is False when the covered range is wider than max_width (the unified max should
    not be used for this data); other failures raise."""
    n = len(counts) - 2
    if n < 1:
        raise ValueError("a histogram holds at least one bin and the two outer counts")
    arr = (ctypes.c_ulonglong * len(counts))(*[int(c) for c in counts])
    phi, x_lo, x_hi = ctypes.c_float(), ctypes.c_float(), ctypes.c_float()
    rc = lib().decode_attn_choose_phi(arr, n, lo, hi, coverage, max_width, ctypes.byref(phi),
                                      ctypes.byref(x_lo), ctypes.byref(x_hi))
    if rc not in (0, DA_ERR_RANGE_TOO_WIDE):
        _check(rc, "decode_attn_choose_phi")
    return phi.value, x_lo.value, x_hi.value, rc == 0


def decode_attn_rope_create(config: da_rope_config):
    rope = P()
    _check(lib().decode_attn_rope_create(ctypes.byref(config), ctypes.byref(rope)),
           "decode_attn_rope_create")
    return rope


def decode_attn_rope_frequencies(rope, pairs: int) -> list:
    """The scaled frequencies (radians per position) of the handle's rotary_dim / 2 pairs."""
    theta = (ctypes.c_double * pairs)()
    _check(lib().decode_attn_rope_frequencies(rope, theta), "decode_attn_rope_frequencies")
    return list(theta)


def decode_attn_rope_apply(rope, args: da_rope_args):
    _check(lib().decode_attn_rope_apply(rope, ctypes.byref(args)), "decode_attn_rope_apply")


def decode_attn_rope_destroy(rope):
    lib().decode_attn_rope_destroy(rope)


def decode_attn_kv_write(plan, args: da_kv_write_args):
    _check(lib().decode_attn_kv_write(plan, ctypes.byref(args)), "decode_attn_kv_write")


def decode_attn_kv_read(plan, args: da_kv_read_args):
    _check(lib().decode_attn_kv_read(plan, ctypes.byref(args)), "decode_attn_kv_read")


def decode_attn_tree_plan(problem: da_problem, max_tree: int):
    """Returns (tree plan handle, workspace bytes)."""
    plan = P()
    ws = ctypes.c_size_t()
    _check(lib().decode_attn_tree_plan(ctypes.byref(problem), max_tree, ctypes.byref(plan),
                                       ctypes.byref(ws)), "decode_attn_tree_plan")
    return plan, ws.value


def decode_attn_tree_plan_info(plan) -> da_tree_plan_info:
    info = da_tree_plan_info()
    _check(lib().decode_attn_tree_plan_info(plan, ctypes.byref(info)),
           "decode_attn_tree_plan_info")
    return info


def decode_attn_tree_debug_stall(plan, tensor: int):
    _check(lib().decode_attn_tree_debug_stall(plan, tensor), "decode_attn_tree_debug_stall")


def decode_attn_tree_workspace_init(plan, workspace: int, workspace_bytes: int, stream: int = 0):
    _check(lib().decode_attn_tree_workspace_init(plan, workspace, workspace_bytes, stream or None),
           "decode_attn_tree_workspace_init")


def decode_attn_tree_run(plan, args: da_tree_args):
    _check(lib().decode_attn_tree_run(plan, ctypes.byref(args)), "decode_attn_tree_run")


def decode_attn_tree_check_status(plan, workspace: int, stream: int = 0):
    _check(lib().decode_attn_tree_check_status(plan, workspace, stream or None),
           "decode_attn_tree_check_status")


def decode_attn_tree_destroy(plan):
    lib().decode_attn_tree_destroy(plan)


def decode_attn_pages_init(plan, pool: int, stream: int = 0):
    _check(lib().decode_attn_pages_init(plan, pool, stream or None), "decode_attn_pages_init")


def decode_attn_pages_reserve(plan, args: da_pages_reserve_args):
    _check(lib().decode_attn_pages_reserve(plan, ctypes.byref(args)), "decode_attn_pages_reserve")


def decode_attn_pages_release(plan, args: da_pages_release_args):
    _check(lib().decode_attn_pages_release(plan, ctypes.byref(args)), "decode_attn_pages_release")


def decode_attn_norm_apply(config: da_norm_config, args: da_norm_args):
    _check(lib().decode_attn_norm_apply(ctypes.byref(config), ctypes.byref(args)),
           "decode_attn_norm_apply")


def decode_attn_adapters_apply(config: da_adapter_config, args: da_adapter_args):
    _check(lib().decode_attn_adapters_apply(ctypes.byref(config), ctypes.byref(args)),
           "decode_attn_adapters_apply")


def decode_attn_adapters_workspace(config: da_adapter_config, rows: int) -> int:
    """Bytes of the workspace with which a call over `rows` rows is fastest."""
    n = ctypes.c_size_t()
    _check(lib().decode_attn_adapters_workspace(ctypes.byref(config), rows, ctypes.byref(n)),
           "decode_attn_adapters_workspace")
    return n.value


def decode_attn_adapters_check_status(workspace: int, stream: int = 0):
    _check(lib().decode_attn_adapters_check_status(workspace, stream or None),
           "decode_attn_adapters_check_status")


def decode_attn_destroy(plan):
    lib().decode_attn_destroy(plan)


def make_problem(*, batch, num_q_heads, num_kv_heads, head_dim, qkv_dtype, out_dtype, paged=False,
                 page_size=16, max_blocks_per_seq=0, num_physical_blocks=0, max_seq_len=0,
                 mode="sync", unified_max=0.0, range_lo=-64.0, range_hi=64.0, validate=False,
                 num_sms=0, kv_dtype=None, k_scale=1.0, v_scale=1.0,
                 debug_stall_stage=0) -> da_problem:
    """kv_dtype=None: K / V stored as qkv_dtype; "e4m3": an FP8 cache of codes standing for
    code * k_scale and code * v_scale (q stays qkv_dtype, which must be bf16)."""
    if kv_dtype not in (None, qkv_dtype, "e4m3"):
        raise ValueError("K / V are stored as qkv_dtype or as e4m3")
    fp8 = kv_dtype == "e4m3"
    return da_problem(batch, num_q_heads, num_kv_heads, head_dim, int(bool(paged)), page_size,
                      max_blocks_per_seq, num_physical_blocks, max_seq_len,
                      DTYPE_CODES[qkv_dtype], DTYPE_CODES[out_dtype], MODE_CODES[mode],
                      unified_max, range_lo, range_hi, int(bool(validate)), num_sms, int(fp8),
                      k_scale if fp8 else 1.0, v_scale if fp8 else 1.0, int(debug_stall_stage))


# ---- torch-facing convenience (marshalling only) -------------------------------------------
_torch = None


def _use_torch():
    global _torch
    import torch
    _torch = torch


class _Workspace:
    """An object with a workspace. Its memory belongs to the stream that was current when it was made; a call on
    another stream is noted with the allocator, so that the memory goes to nobody else before that call's
    kernels have ended, whenever the object is dropped."""

    workspace = _noted = _noted_stream = None

    def _make_workspace(self, size, device):
        """Zero-filled, which needs no init call, and ready for any stream."""
        device = _torch.device("cuda") if device is None else _torch.device(device)
        self.workspace = self._noted = _torch.zeros(size, dtype=_torch.uint8, device=device)
        stream = _torch.cuda.current_stream(self.workspace.device)
        self._noted_stream = stream.cuda_stream
        if not _torch.cuda.is_current_stream_capturing():
            stream.synchronize()

    def _workspace_on(self, index, stream):
        """Its address, for a call on `stream` (None: device `index`'s current one)."""
        ws = self.workspace
        raw = _torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
        if raw != self._noted_stream or ws is not self._noted:
            ws.record_stream(_torch.cuda.current_stream(index) if stream is None else stream)
            self._noted, self._noted_stream = ws, raw
        return ws.data_ptr()


class DecodeAttention(_Workspace):
    """A plan plus its workspace on the current CUDA device.

    run() takes torch tensors already on the device, passes their addresses and the
    current stream to decode_attn_run, and returns (out, lse, row_flags)."""

    def __init__(self, problem: da_problem, num_splits: int = 0, device=None):
        _use_torch()
        self.problem = problem
        self.plan, self.workspace_bytes = decode_attn_plan(problem, num_splits)
        self.info = decode_attn_plan_info(self.plan)
        from .workloads import TORCH_DTYPES
        names = {v: k for k, v in DTYPE_CODES.items()}
        self._qkv_dtype = TORCH_DTYPES[names[problem.qkv_dtype]]
        self._out_dtype = TORCH_DTYPES[names[problem.out_dtype]]
        self.device = _torch.device(device) if device is not None else _torch.device("cuda")
        self._make_workspace(self.workspace_bytes, self.device)

    def __del__(self):
        plan = getattr(self, "plan", None)
        if plan is not None and _lib is not None:
            decode_attn_destroy(plan)
            self.plan = None

    def run(self, q, k_cache, v_cache, block_table, seq_lens, scale: float, num_splits: int = -1,
            out=None, out_lse=None, row_flags=None, stream=None, want_stats: bool = False,
            split_events=None):
        import torch
        pr = self.problem
        qkv = self._qkv_dtype
        # an FP8 cache holds E4M3 codes: torch.float8_e4m3fn, or their bytes as uint8
        kv_ok = (torch.uint8, torch.float8_e4m3fn) if pr.kv_fp8 else (qkv,)
        for name, t, ok in (("q", q, (qkv,)), ("k_cache", k_cache, kv_ok),
                            ("v_cache", v_cache, kv_ok)):
            if t.device.type != "cuda" or t.dtype not in ok or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CUDA tensor of {ok}")
        if seq_lens.dtype != torch.int32 or seq_lens.device.type != "cuda":
            raise ValueError("seq_lens must be an int32 CUDA tensor")
        if block_table is not None and (block_table.dtype != torch.int32 or
                                        not block_table.is_contiguous()):
            raise ValueError("block_table must be a contiguous int32 CUDA tensor")
        B, H = pr.batch, pr.num_q_heads
        if out is None:
            out = torch.empty((B, H, pr.head_dim), dtype=self._out_dtype, device=q.device)
        if out_lse is None:
            out_lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
        if row_flags is None:
            row_flags = torch.empty((B, H), dtype=torch.uint8, device=q.device)
        s = stream if stream is not None else torch.cuda.current_stream(q.device)
        st = da_stats() if want_stats else None
        args = da_run_args(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                           None if block_table is None else block_table.data_ptr(),
                           seq_lens.data_ptr(), float(scale), num_splits, out.data_ptr(),
                           out_lse.data_ptr(), row_flags.data_ptr(),
                           self._workspace_on(q.get_device(), s),
                           self.workspace_bytes, s.cuda_stream or None,
                           ctypes.pointer(st) if st is not None else None,
                           split_events[0].cuda_event if split_events else None,
                           split_events[1].cuda_event if split_events else None)
        decode_attn_run_ex(self.plan, args)
        if want_stats:
            return out, out_lse, row_flags, st
        return out, out_lse, row_flags


# What a call of the wrappers below costs on the host is of the order of the kernel it launches, so torch is
# imported once, checks look at an attribute at a time, and the argument structures are packed in one go.
class _Entry:
    """A C entry point that takes (handle, structure of `args`, whose last field is the stream)."""

    FORMATS = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int: "i", ctypes.c_float: "f",
               ctypes.c_size_t: "N"}

    def __init__(self, name, args):
        packer = struct.Struct("@" + "".join(self.FORMATS[t] for _, t in args._fields_) + "0P")
        if packer.size != ctypes.sizeof(args):
            raise RuntimeError(f"{args.__name__} has no packed form")
        self.name, self.pack = name, packer.pack
        self.fn = ctypes.CFUNCTYPE(ctypes.c_int, P, ctypes.c_char_p)((name, lib()))

    def __call__(self, handle, index, stream, *values):
        """Call with the structure's other fields `values` (0: a null pointer) on the given stream (the
        device's current one unless given), with device `index` current."""
        if stream is not None:
            s = stream.cuda_stream
        else:
            s = _torch._C._cuda_getCurrentRawStream(index)   # current_stream() without its objects
        args = self.pack(*values, s)
        if _torch._C._cuda_getDevice() == index:
            rc = self.fn(handle, args)
        else:
            with _torch.cuda.device(index):
                rc = self.fn(handle, args)
        if rc:
            raise DecodeAttnError(rc, self.name)


_entries = {}


def _entry(name, args):
    _use_torch()
    if name not in _entries:
        _entries[name] = _Entry(name, args)
    return _entries[name]


def _refuse_devices(index, **tensors):
    """Says which of the tensors is not on one CUDA device with the others."""
    for name, t in tensors.items():
        if t is not None and t.get_device() < 0:
            raise ValueError(f"{name} must be a CUDA tensor")
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, other tensors on cuda:{index}")


def _rows_tensor(name, t, dtype, heads, d):
    """A [rows, heads, d] tensor whose heads are contiguous (rows and heads may be strided). Returns its
    rows, and the strides of rows and heads."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError(f"{name} must be a [rows, {heads}, {d}] tensor of {dtype}")
    row, head, one = t.stride()
    if one != 1 and t.numel():
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return shape[0], row, head


def _int32(name, t, numel):
    if t.dtype is not _torch.int32 or t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {numel} elements")


def _empty(shape, dtype, device, stream):
    """A result's memory, from the pool of the stream that writes it: memory of another stream's pool may
    still be in use there."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def _rotation():
    """The autograd function of Rope.apply, made once torch is there."""
    class Rotation(_torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, rope, positions, transpose, stream):
            ctx.save_for_backward(positions)
            ctx.rope, ctx.transpose = rope, transpose
            return rope._rotate(x, positions, None, transpose, stream)

        @staticmethod
        def backward(ctx, grad):
            (positions,) = ctx.saved_tensors
            if grad.stride(-1) != 1:
                grad = grad.contiguous()
            # on the stream that autograd runs this on: the one that was current in the forward call
            return ctx.rope.apply(grad, positions, transpose=not ctx.transpose), None, None, None, None

    return Rotation


_Rotation = None


class Rope:
    """A rotary embedding: its frequencies, scaled for long contexts by `scaling` ("none", "linear",
    "ntk", "by_parts", "by_index"; see da_rope_scaling), and its layout.

    apply() rotates a [rows, heads, head_dim] tensor; KVCacheIO.write() takes the handle to rotate
    q and k on their way into the cache."""

    def __init__(self, head_dim: int, rotary_dim: Optional[int] = None, interleaved: bool = False,
                 base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original_max_position: float = 0.0, low: float = 1.0, high: float = 32.0,
                 attn_factor: float = 1.0):
        if scaling not in ROPE_CODES:
            raise ValueError(f"scaling must be one of {sorted(ROPE_CODES)}")
        self._apply = _entry("decode_attn_rope_apply", da_rope_args)
        self.head_dim = head_dim
        self.rotary_dim = head_dim if rotary_dim is None else rotary_dim
        self.handle = decode_attn_rope_create(da_rope_config(
            head_dim, self.rotary_dim, int(bool(interleaved)), ROPE_CODES[scaling], base, factor,
            original_max_position, low, high, attn_factor))
        from .workloads import TORCH_DTYPES
        self._codes = {TORCH_DTYPES[k]: v for k, v in DTYPE_CODES.items()}

    def __del__(self):
        handle = getattr(self, "handle", None)
        if handle is not None and _lib is not None:
            decode_attn_rope_destroy(handle)
            self.handle = None

    def frequencies(self) -> list:
        return decode_attn_rope_frequencies(self.handle, self.rotary_dim // 2)

    def apply(self, x, positions, out=None, transpose: bool = False, stream=None):
        """Rows of x (fp32, fp16 or bf16; rows and heads may be strided) rotated by `positions`
        (int32 [rows]), into `out` (x itself: in place; allocated on the call's stream when None).
        transpose: the transposed map, which takes the gradient of the output to the gradient of x.
        Autograd records the call where x requires a gradient; `out` cannot be given then."""
        if (x.requires_grad or (out is not None and out.requires_grad)) and _torch.is_grad_enabled():
            if out is not None:
                raise ValueError("autograd cannot record a call with an out")
            global _Rotation
            if _Rotation is None:
                _Rotation = _rotation()
            return _Rotation.apply(x, self, positions, transpose, stream)
        return self._rotate(x, positions, out, transpose, stream)

    def _rotate(self, x, positions, out, transpose, stream):
        dtype, shape = x.dtype, x.shape
        code = self._codes.get(dtype)
        if code is None:
            raise ValueError("x must be fp32, fp16 or bf16")
        if len(shape) != 3:
            raise ValueError("x must be a [rows, heads, head_dim] tensor")
        if out is None:
            out = _empty(shape, dtype, x.device, stream)
        heads = shape[1]
        rows, x_row, x_head = _rows_tensor("x", x, dtype, heads, self.head_dim)
        out_rows, out_row, out_head = _rows_tensor("out", out, dtype, heads, self.head_dim)
        if out_rows != rows:
            raise ValueError("out must have as many rows as x")
        _int32("positions", positions, rows)
        index = x.get_device()
        if index < 0 or positions.get_device() != index or out.get_device() != index:
            _refuse_devices(index, x=x, positions=positions, out=out)
        if rows and heads:
            self._apply(self.handle, index, stream, x.data_ptr(), out.data_ptr(), code, rows, heads,
                        x_row, x_head, out_row, out_head, positions.data_ptr(), 1 if transpose else 0)
        return out


class _Cache:
    """What a problem says of its cache, and the checks of a call's cache, block table and row layout."""

    def __init__(self, pr: da_problem):
        import torch
        from .workloads import TORCH_DTYPES
        names = {v: k for k, v in DTYPE_CODES.items()}
        self.dtype, self.out_dtype = TORCH_DTYPES[names[pr.qkv_dtype]], TORCH_DTYPES[names[pr.out_dtype]]
        self.kv_dtypes = (torch.uint8, torch.float8_e4m3fn) if pr.kv_fp8 else (self.dtype,)
        self.batch, self.hq, self.hkv, self.d = (pr.batch, pr.num_q_heads, pr.num_kv_heads,
                                                 pr.head_dim)
        self.paged = bool(pr.paged)
        self.table = pr.batch * pr.max_blocks_per_seq
        self.shape = ((pr.num_physical_blocks, pr.page_size, self.hkv, self.d) if self.paged else
                      (pr.batch, pr.max_seq_len, self.hkv, self.d))

    def check(self, k_cache, v_cache, block_table, row_offsets, start):
        """Returns the device's index and the block table's address (0: none)."""
        for t in (k_cache, v_cache):
            if t is not None and (t.shape != self.shape or t.dtype not in self.kv_dtypes or
                                  not t.is_contiguous()):
                raise ValueError(f"{'k_cache' if t is k_cache else 'v_cache'} must be a contiguous "
                                 f"{self.shape} tensor of {self.kv_dtypes}")
        if (block_table is None) == self.paged:
            raise ValueError("a paged cache takes a block_table, a contiguous one none")
        _int32("row_offsets", row_offsets, self.batch + 1)
        _int32("the sequences' lengths", start, self.batch)
        index, table = row_offsets.get_device(), 0
        if block_table is not None:
            _int32("block_table", block_table, self.table)
            table = block_table.data_ptr()
        if index < 0 or start.get_device() != index or \
                (k_cache is not None and k_cache.get_device() != index) or \
                (v_cache is not None and v_cache.get_device() != index) or \
                (block_table is not None and block_table.get_device() != index):
            _refuse_devices(index, row_offsets=row_offsets, start=start, k_cache=k_cache, v_cache=v_cache,
                            block_table=block_table)
        return index, table


class KVCacheIO(_Workspace):
    """Writes rows of K and V into a cache of the problem's shape and storage, and reads them back.

    The rows of a step lie one after another, sequence by sequence: row_offsets (int32
    [batch + 1]) says which rows are whose, start (int32 [batch]) the cache position of each
    sequence's first row. With findings=True (or the problem's validate) the device records rows
    without a place in the cache, which check_status() reports. Autograd records neither call."""

    def __init__(self, problem: da_problem, findings: bool = False, device=None):
        self._write = _entry("decode_attn_kv_write", da_kv_write_args)
        self._read = _entry("decode_attn_kv_read", da_kv_read_args)
        self.problem = problem
        self.plan, self.workspace_bytes = decode_attn_plan(problem, 0)
        self._cache = _Cache(problem)
        if findings or problem.validate:
            self._make_workspace(self.workspace_bytes, device)

    def __del__(self):
        plan = getattr(self, "plan", None)
        if plan is not None and _lib is not None:
            decode_attn_destroy(plan)
            self.plan = None

    def write(self, k, v, k_cache, v_cache, block_table, row_offsets, start, rope=None,
              positions=None, q=None, q_out=None, amax=None, stream=None):
        """Write the rows of k and v ([rows, H_kv, d], strided rows and heads allowed); with `rope`
        rotate k, and q into q_out (allocated when None, q itself: in place). `positions`: rotary
        positions other than the cache positions. `amax`: a float32 [2] tensor that takes the
        running largest |k| and |v|. Returns q_out (None without q)."""
        c, ws = self._cache, self.workspace
        index, table = c.check(k_cache, v_cache, block_table, row_offsets, start)
        if k_cache is None or v_cache is None:
            raise ValueError("k_cache and v_cache must both be given")
        rows, k_row, k_head = _rows_tensor("k", k, c.dtype, c.hkv, c.d)
        v_rows, v_row, v_head = _rows_tensor("v", v, c.dtype, c.hkv, c.d)
        if v_rows != rows:
            raise ValueError("v must have as many rows as k")
        away = k.get_device() != index or v.get_device() != index
        q_row = q_head = out_row = out_head = q_at = out_at = at = most = 0
        if q is not None:
            q_rows, q_row, q_head = _rows_tensor("q", q, c.dtype, c.hq, c.d)
            if q_out is None:
                q_out = _empty(q.shape, c.dtype, q.device, stream)
            out_rows, out_row, out_head = _rows_tensor("q_out", q_out, c.dtype, c.hq, c.d)
            if q_rows != rows or out_rows != rows:
                raise ValueError("q and q_out must have as many rows as k")
            q_at, out_at = q.data_ptr(), q_out.data_ptr()
            away = away or q.get_device() != index or q_out.get_device() != index
        elif q_out is not None:
            raise ValueError("q_out without q")
        if rope is None and (q is not None or positions is not None):
            raise ValueError("q and positions need a rope")
        if positions is not None:
            _int32("positions", positions, rows)
            at = positions.data_ptr()
            away = away or positions.get_device() != index
        if amax is not None:
            if amax.dtype is not _torch.float32 or amax.numel() != 2 or not amax.is_contiguous():
                raise ValueError("amax must be a contiguous float32 tensor of 2 elements")
            most = amax.data_ptr()
            away = away or amax.get_device() != index
        if away or (ws is not None and ws.get_device() != index):
            _refuse_devices(index, k=k, v=v, q=q, q_out=q_out, positions=positions, amax=amax,
                            workspace=ws)
        if rows:
            self._write(self.plan, index, stream, k.data_ptr(), v.data_ptr(), k_row, k_head, v_row,
                        v_head, rows, k_cache.data_ptr(), v_cache.data_ptr(), table,
                        row_offsets.data_ptr(), start.data_ptr(),
                        0 if rope is None else rope.handle.value, at, q_at, out_at, q_row, q_head,
                        out_row, out_head, most,
                        0 if ws is None else self._workspace_on(index, stream), self.workspace_bytes)
        return q_out

    def read(self, k_cache, v_cache, block_table, row_offsets, start, k_out, v_out, stream=None):
        """Fill k_out and v_out (contiguous [rows, H_kv, d]; either may be None, its cache too) with
        the rows' K and V. Returns (k_out, v_out)."""
        c, ws = self._cache, self.workspace
        index, table = c.check(k_cache, v_cache, block_table, row_offsets, start)
        if (k_out is None) != (k_cache is None) or (v_out is None) != (v_cache is None) or \
                (k_out is None and v_out is None):
            raise ValueError("give k_out with k_cache, v_out with v_cache, or all four")
        rows, places = -1, []
        for t in (k_out, v_out):
            if t is None:
                places.append(0)
                continue
            n, _, _ = _rows_tensor("k_out / v_out", t, c.dtype, c.hkv, c.d)
            if not t.is_contiguous() or (rows >= 0 and n != rows):
                raise ValueError("k_out and v_out must be contiguous, with as many rows")
            if t.get_device() != index:
                _refuse_devices(index, k_out=k_out, v_out=v_out)
            rows = n
            places.append(t.data_ptr())
        if ws is not None and ws.get_device() != index:
            _refuse_devices(index, workspace=ws)
        if rows:
            self._read(self.plan, index, stream, 0 if k_cache is None else k_cache.data_ptr(),
                       0 if v_cache is None else v_cache.data_ptr(), table, row_offsets.data_ptr(),
                       start.data_ptr(), rows, places[0], places[1],
                       0 if ws is None else self._workspace_on(index, stream), self.workspace_bytes)
        return k_out, v_out

    def check_status(self, stream=None):
        """Synchronise, then raise the first finding recorded since the last call."""
        if self.workspace is None:
            raise ValueError("made without findings")
        _check_workspace(decode_attn_check_status, self, stream)


def _check_workspace(fn, of, stream):
    with _torch.cuda.device(of.workspace.device):
        s = stream if stream is not None else _torch.cuda.current_stream()
        fn(of.plan, of._workspace_on(of.workspace.get_device(), s), s.cuda_stream)


class TreeAttention(_Workspace):
    """Attention of drafted tokens over a cache that already holds their K and V, one tree (or
    chain) of up to max_tree tokens a sequence: a plan plus its workspace. Two runs of one object
    must not overlap on the GPU, and a captured graph needs the object as long as it is replayed."""

    def __init__(self, problem: da_problem, max_tree: int = MAX_TREE, device=None):
        self._run = _entry("decode_attn_tree_run", da_tree_args)
        self.problem = problem
        self.plan, self.workspace_bytes = decode_attn_tree_plan(problem, max_tree)
        self.info = decode_attn_tree_plan_info(self.plan)
        self._cache = _Cache(problem)
        self._make_workspace(self.workspace_bytes, device)
        self.device = self.workspace.device

    def __del__(self):
        plan = getattr(self, "plan", None)
        if plan is not None and _lib is not None:
            decode_attn_tree_destroy(plan)
            self.plan = None

    def run(self, q, k_cache, v_cache, block_table, row_offsets, ctx_lens, tree_mask, scale: float,
            out=None, out_lse=None, stream=None):
        """q [rows, H_q, d]: the drafted tokens' queries, sequence by sequence (row_offsets); their K
        and V lie in the cache from position ctx_lens[b] on. tree_mask: int64 (or uint64) [rows],
        bit j of a row's word set iff it attends to its sequence's drafted token j; None: a chain.
        Returns (out, lse)."""
        c, ws, mask = self._cache, self.workspace, 0
        index, table = c.check(k_cache, v_cache, block_table, row_offsets, ctx_lens)
        if k_cache is None or v_cache is None:
            raise ValueError("k_cache and v_cache must both be given")
        rows, _, _ = _rows_tensor("q", q, c.dtype, c.hq, c.d)
        if out is None:
            out = _empty(q.shape, c.out_dtype, q.device, stream)
        if out_lse is None:
            out_lse = _empty((rows, c.hq), _torch.float32, q.device, stream)
        out_rows, _, _ = _rows_tensor("out", out, c.out_dtype, c.hq, c.d)
        if out_rows != rows or not q.is_contiguous() or not out.is_contiguous():
            raise ValueError("q and out must be contiguous, with as many rows")
        if out_lse.dtype is not _torch.float32 or out_lse.shape != (rows, c.hq) or \
                not out_lse.is_contiguous():
            raise ValueError("out_lse must be a contiguous float32 [rows, H_q] tensor")
        away = q.get_device() != index or out.get_device() != index or \
            out_lse.get_device() != index or ws.get_device() != index
        if tree_mask is not None:
            if tree_mask.dtype not in (_torch.int64, _torch.uint64) or tree_mask.shape != (rows,) or \
                    not tree_mask.is_contiguous():
                raise ValueError("tree_mask must be a contiguous int64 [rows] tensor")
            mask = tree_mask.data_ptr()
            away = away or tree_mask.get_device() != index
        if away:
            _refuse_devices(index, q=q, out=out, out_lse=out_lse, tree_mask=tree_mask, workspace=ws)
        if rows:
            self._run(self.plan, index, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                      table, row_offsets.data_ptr(), ctx_lens.data_ptr(), mask, rows, scale,
                      out.data_ptr(), out_lse.data_ptr(), self._workspace_on(index, stream),
                      self.workspace_bytes)
        return out, out_lse

    def check_status(self, stream=None):
        """Synchronise, then raise the first finding recorded since the last call."""
        _check_workspace(decode_attn_tree_check_status, self, stream)


class PageTables(_Workspace):
    """Pages of the problem's paged cache: new_pool() makes a pool with every page free, reserve() takes a
    step's pages off it and enters them in the block table, release() gives back what sequences lose.

    A pool is an int32 tensor [POOL_HEAD + num_physical_blocks] (the C header says what is in it). Calls on
    one pool must not overlap on the GPU. With findings=True (or the problem's validate) the device records
    bad lengths and entries, and steps that the pool had too few pages for, which check_status() reports."""

    def __init__(self, problem: da_problem, findings: bool = False, device=None):
        self._reserve = _entry("decode_attn_pages_reserve", da_pages_reserve_args)
        self._release = _entry("decode_attn_pages_release", da_pages_release_args)
        self.problem = problem
        self.plan, self.workspace_bytes = decode_attn_plan(problem, 0)
        if not problem.paged:
            raise ValueError("a contiguous cache has no pages")
        self._batch, self._table = problem.batch, problem.batch * problem.max_blocks_per_seq
        self._pool = POOL_HEAD + problem.num_physical_blocks
        if findings or problem.validate:
            self._make_workspace(self.workspace_bytes, device)

    def __del__(self):
        plan = getattr(self, "plan", None)
        if plan is not None and _lib is not None:
            decode_attn_destroy(plan)
            self.plan = None

    def new_pool(self, device=None, stream=None):
        """A pool whose pages are all free, page 0 on top."""
        device = _torch.device("cuda") if device is None else _torch.device(device)
        pool = _empty((self._pool,), _torch.int32, device, stream)
        with _torch.cuda.device(pool.device):
            s = stream if stream is not None else _torch.cuda.current_stream()
            decode_attn_pages_init(self.plan, pool.data_ptr(), s.cuda_stream)
        return pool

    def _checked(self, pool, block_table, lens):
        """The device's index, once the three are what they should be."""
        _int32("pool", pool, self._pool)
        _int32("block_table", block_table, self._table)
        _int32("the sequences' lengths", lens, self._batch)
        index, ws = pool.get_device(), self.workspace
        if index < 0 or block_table.get_device() != index or lens.get_device() != index or \
                (ws is not None and ws.get_device() != index):
            _refuse_devices(index, pool=pool, block_table=block_table, lengths=lens, workspace=ws)
        return index

    def reserve(self, pool, block_table, row_offsets, ctx_lens, rows: int, seq_lens=None, slots=None,
                positions=None, stream=None):
        """Pages for a step of `rows` rows: sequence b holds ctx_lens[b] tokens and gets the rows row_offsets[b]
        to row_offsets[b + 1]. Returns (seq_lens, slots, positions): the lengths then (ctx_lens itself: in
        place), each row's cache row (-1: none) and position; allocated when None. Where the pool has too few
        pages nothing is taken, every slot is -1 and pool[1] says how many were missing; nor where row_offsets
        fall anywhere, which is a bad length."""
        index, batch = self._checked(pool, block_table, ctx_lens), self._batch
        _int32("row_offsets", row_offsets, batch + 1)
        if rows < 0:
            raise ValueError("rows must not be negative")
        away = row_offsets.get_device() != index
        if seq_lens is None:
            seq_lens = _empty((batch,), _torch.int32, pool.device, stream)
        else:
            _int32("seq_lens", seq_lens, batch)
            away = away or seq_lens.get_device() != index
        if slots is None:
            slots = _empty((rows,), _torch.int32, pool.device, stream)
        else:
            _int32("slots", slots, rows)
            away = away or slots.get_device() != index
        if positions is None:
            positions = _empty((rows,), _torch.int32, pool.device, stream)
        else:
            _int32("positions", positions, rows)
            away = away or positions.get_device() != index
        if away:
            _refuse_devices(index, pool=pool, row_offsets=row_offsets, seq_lens=seq_lens, slots=slots,
                            positions=positions)
        self._reserve(self.plan, index, stream, pool.data_ptr(), block_table.data_ptr(), row_offsets.data_ptr(),
                      ctx_lens.data_ptr(), rows, seq_lens.data_ptr(), slots.data_ptr(), positions.data_ptr(),
                      0 if self.workspace is None else self._workspace_on(index, stream), self.workspace_bytes)
        return seq_lens, slots, positions

    def release(self, pool, block_table, seq_lens, keep_lens, stream=None):
        """Cut sequences back from seq_lens[b] to keep_lens[b] tokens (0: it has ended): the pages they lose
        go back to the pool, and their entries become -1."""
        index = self._checked(pool, block_table, seq_lens)
        _int32("keep_lens", keep_lens, self._batch)
        if keep_lens.get_device() != index:
            _refuse_devices(index, pool=pool, keep_lens=keep_lens)
        self._release(self.plan, index, stream, pool.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                      keep_lens.data_ptr(), 0 if self.workspace is None else self._workspace_on(index, stream),
                      self.workspace_bytes)

    def check_status(self, stream=None):
        """Synchronise, then raise the first finding recorded since the last call."""
        if self.workspace is None:
            raise ValueError("made without findings")
        _check_workspace(decode_attn_check_status, self, stream)


def _refuse_autograd(**tensors):
    if _torch.is_grad_enabled():
        for name, t in tensors.items():
            if t is not None and t.requires_grad:
                raise ValueError(f"{name} requires a gradient, which this call has none of: use no_grad()")


class RMSNorm:
    """A root-mean-square norm of rows of n elements: y = u (weight + weight_offset) / sqrt(mean(u^2) + eps),
    u = x + residual where one is given, rounded to the type.

    x is [rows, n], or [rows, heads, n] (q or k heads), fp32, fp16 or bf16; rows and heads may be strided.
    The weight ([n], None: without one) is of x's type or fp32. Autograd records neither call; tensors that
    require a gradient are refused outside no_grad()."""

    def __init__(self, n: int, eps: float = 1e-6, weight_offset: float = 0.0):
        self._apply = _entry("decode_attn_norm_apply", da_norm_args)
        if not 1 <= n <= 32768:
            raise ValueError("n must be 1 to 32768")
        self.n, self.config = n, da_norm_config(n, eps, weight_offset)
        self._at = ctypes.addressof(self.config)
        from .workloads import TORCH_DTYPES
        self._codes = {TORCH_DTYPES[k]: v for k, v in DTYPE_CODES.items()}

    def apply(self, x, weight=None, residual=None, out=None, residual_out=None, stream=None):
        """y in x's type, into `out` (x itself: in place; allocated when None). With a residual returns
        (out, u): u goes into residual_out (x or residual itself: in place; allocated when None)."""
        out, total, _, _ = self._call(x, weight, residual, out, residual_out, None, None, 0, 0, True, stream)
        return out if residual is None else (out, total)

    def quantise(self, x, weight=None, residual=None, scaling: str = "row", group: int = 128, codes=None,
                 scales=None, out=None, residual_out=None, stream=None):
        """E4M3 codes of y / scale (float8_e4m3fn, or their bytes where `codes` is uint8). scaling "tensor":
        `scales` is a float32 tensor of one element; "row": one found for each row (and head); "group": one for
        each `group` (32, 64 or 128) elements. Where `out` is given it takes y too. Returns
        (codes, scales, u), u as in apply() and None without a residual."""
        kind = SCALING_CODES.get(scaling)
        if kind is None:
            raise ValueError(f"scaling must be one of {sorted(SCALING_CODES)}")
        if kind == 3 and group not in (32, 64, 128):
            raise ValueError("group must be 32, 64 or 128")
        _, total, codes, scales = self._call(x, weight, residual, out, residual_out, codes, scales, kind, group, False,
                                             stream)
        return codes, scales, total

    def _strides(self, name, t, shape, dtype, index):
        """Strides of rows and heads of a tensor that has to be like x."""
        if t.shape != shape or t.dtype is not dtype:
            raise ValueError(f"{name} must be a {list(shape)} tensor of {dtype}")
        st = t.stride()
        if st[-1] != 1 and self.n > 1 and t.numel():
            raise ValueError(f"the last dimension of {name} must be contiguous")
        if t.get_device() != index:
            _refuse_devices(index, **{name: t})
        return st[0], 0 if len(st) == 2 else st[1]

    def _call(self, x, weight, residual, out, residual_out, codes, scales, kind, group, want_out, stream):
        shape, dtype, n = x.shape, x.dtype, self.n
        code, dims = self._codes.get(dtype), len(shape)
        if code is None:
            raise ValueError("x must be fp32, fp16 or bf16")
        if (dims != 2 and dims != 3) or shape[-1] != n:
            raise ValueError(f"x must be a [rows, {n}] or [rows, heads, {n}] tensor")
        if _torch.is_grad_enabled() and (
                x.requires_grad or (weight is not None and weight.requires_grad) or
                (residual is not None and residual.requires_grad) or (out is not None and out.requires_grad) or
                (residual_out is not None and residual_out.requires_grad)):
            _refuse_autograd(x=x, weight=weight, residual=residual, out=out, residual_out=residual_out)
        rows, heads, index = shape[0], 1 if dims == 2 else shape[1], x.get_device()
        x_row, x_head = self._strides("x", x, shape, dtype, index)
        plain = heads * n     # strides of what is allocated here: plain, n
        r_row = r_head = u_row = u_head = o_row = o_head = c_row = c_head = 0
        r_at = u_at = o_at = c_at = s_at = w_at = wide = 0
        if weight is not None:
            wide = 1 if weight.dtype is _torch.float32 else 0
            if (not wide and weight.dtype is not dtype) or weight.shape != (n,) or not weight.is_contiguous():
                raise ValueError(f"weight must be a contiguous [{n}] tensor of {dtype} or float32")
            w_at = weight.data_ptr()
            if weight.get_device() != index:
                _refuse_devices(index, weight=weight)
        if residual is not None:
            r_row, r_head = self._strides("residual", residual, shape, dtype, index)
            r_at = residual.data_ptr()
        elif residual_out is not None:
            raise ValueError("residual_out without a residual")
        if residual_out is not None:
            u_row, u_head = self._strides("residual_out", residual_out, shape, dtype, index)
        if out is not None:
            o_row, o_head = self._strides("out", out, shape, dtype, index)
        if codes is not None:
            if codes.dtype is not _torch.float8_e4m3fn and codes.dtype is not _torch.uint8:
                raise ValueError("codes must be float8_e4m3fn or uint8")
            c_row, c_head = self._strides("codes", codes, shape, codes.dtype, index)
        if kind:
            many = (1,) if kind == 1 else shape[:-1] if kind == 2 else (*shape[:-1], -(-n // group))
            if scales is None:
                if kind == 1:
                    raise ValueError("scaling by tensor takes scales")
            elif scales.dtype is not _torch.float32 or not scales.is_contiguous() or \
                    (scales.numel() != 1 if kind == 1 else scales.shape != many):
                raise ValueError(f"scales must be a contiguous float32 tensor {list(many)}")
            elif scales.get_device() != index:
                _refuse_devices(index, scales=scales)
        if index < 0:
            _refuse_devices(index, x=x)
        # results that are not given
        if residual is not None:
            if residual_out is None:
                residual_out, u_row, u_head = _empty(shape, dtype, x.device, stream), plain, n
            u_at = residual_out.data_ptr()
        if want_out and out is None:
            out, o_row, o_head = _empty(shape, dtype, x.device, stream), plain, n
        if out is not None:
            o_at = out.data_ptr()
        if kind:
            if codes is None:
                codes, c_row, c_head = _empty(shape, _torch.float8_e4m3fn, x.device, stream), plain, n
            if scales is None:
                scales = _empty(many, _torch.float32, x.device, stream)
            c_at, s_at = codes.data_ptr(), scales.data_ptr()
        if rows and heads:
            self._apply(self._at, index, stream, x.data_ptr(), r_at, w_at, u_at, o_at, c_at, s_at, code, wide, kind,
                        group, rows, heads, x_row, x_head, r_row, r_head, u_row, u_head, o_row, o_head, c_row, c_head)
        return out, residual_out, codes, scales


class Adapters(_Workspace):
    """Low-rank adapters of many requests beside a shared projection of rows of `width` to columns in parts
    of out_sizes (q, k and v, for instance): out = y + scales[a] (x A_a^T) B_a^T, part by part.

    a: [adapters, parts * rank, width] (or [adapters, parts, rank, width]), b: [adapters, columns, rank],
    contiguous, of `dtype` ("f32", "f16", "bf16") as x and y are. Autograd does not record the call; tensors
    that require a gradient are refused outside no_grad().

    Long steps for which it pays take a workspace for their low-rank sums, from the allocator for each call. With
    findings=True the object keeps one, whose findings check_status() reports; two such calls must not overlap on
    the GPU. A captured graph needs the object as long as it is replayed, and a step as long as its own made ahead of
    the capture (a ValueError without); a longer one later leaves it what it has."""

    LONG = 1024   # rows from which a step may use a workspace

    def __init__(self, width: int, out_sizes, rank: int, dtype: str = "bf16", findings: bool = False):
        self._apply = _entry("decode_attn_adapters_apply", da_adapter_args)
        out_sizes = [int(n) for n in out_sizes]
        if not 1 <= len(out_sizes) <= ADAPTER_PARTS or min(out_sizes) < 1 or width < 1:
            raise ValueError(f"a projection has 1 to {ADAPTER_PARTS} parts, of at least a column each")
        if rank not in (8, 16, 32, 64, 128):
            raise ValueError("rank must be 8, 16, 32, 64 or 128")
        if dtype not in DTYPE_CODES:
            raise ValueError(f"dtype must be one of {sorted(DTYPE_CODES)}")
        from .workloads import TORCH_DTYPES
        self.width, self.out_sizes, self.rank, self.dtype = width, out_sizes, rank, TORCH_DTYPES[dtype]
        self.columns = sum(out_sizes)
        self.config = da_adapter_config(DTYPE_CODES[dtype], width, len(out_sizes),
                                        (ctypes.c_int * ADAPTER_PARTS)(*out_sizes), rank)
        self._at = ctypes.addressof(self.config)
        self._one = (len(out_sizes) * rank * width, self.columns * rank)
        self._findings, self.workspace_bytes, self._outgrown = findings, 0, []

    def _rows(self, name, t, n):
        if t.dtype is not self.dtype or len(t.shape) != 2 or t.shape[1] != n:
            raise ValueError(f"{name} must be a [rows, {n}] tensor of {self.dtype}")
        row, one = t.stride()
        if one != 1 and n > 1 and t.numel():
            raise ValueError(f"the last dimension of {name} must be contiguous")
        return row

    def apply(self, x, y, a, b, scales, row_offsets, adapter_ids, out=None, stream=None):
        """x [rows, width] and y [rows, columns] (rows may be strided), rows by request (row_offsets int32
        [batch + 1]), adapter_ids int32 [batch] (-1: none), scales float32 [adapters] or None. Returns out
        (y itself: in place; allocated when None)."""
        if _torch.is_grad_enabled() and (x.requires_grad or y.requires_grad or a.requires_grad or b.requires_grad or
                                         (scales is not None and scales.requires_grad) or
                                         (out is not None and out.requires_grad)):
            _refuse_autograd(x=x, y=y, a=a, b=b, scales=scales, out=out)
        x_row, y_row = self._rows("x", x, self.width), self._rows("y", y, self.columns)
        if out is None:
            out = _empty(y.shape, self.dtype, y.device, stream)
        out_row = self._rows("out", out, self.columns)
        rows, n = x.shape[0], a.shape[0]
        if y.shape[0] != rows or out.shape[0] != rows:
            raise ValueError("x, y and out must have as many rows")
        if a.dtype is not self.dtype or n < 1 or a.numel() != n * self._one[0] or a.shape[-1] != self.width or \
                not a.is_contiguous():
            raise ValueError(f"a must be a contiguous [adapters, {len(self.out_sizes) * self.rank}, {self.width}] "
                             f"tensor of {self.dtype}")
        if b.dtype is not self.dtype or b.shape != (n, self.columns, self.rank) or not b.is_contiguous():
            raise ValueError(f"b must be a contiguous [{n}, {self.columns}, {self.rank}] tensor of {self.dtype}")
        batch = adapter_ids.numel()
        _int32("adapter_ids", adapter_ids, batch)
        _int32("row_offsets", row_offsets, batch + 1)
        if batch < 1:
            raise ValueError("a step has at least one request")
        scale_at, index = 0, x.get_device()
        away = index < 0 or y.get_device() != index or out.get_device() != index or a.get_device() != index or \
            b.get_device() != index or row_offsets.get_device() != index or adapter_ids.get_device() != index
        if scales is not None:
            if scales.dtype is not _torch.float32 or scales.numel() != n or not scales.is_contiguous():
                raise ValueError(f"scales must be a contiguous float32 tensor of {n} elements")
            scale_at = scales.data_ptr()
            away = away or scales.get_device() != index
        if away:
            _refuse_devices(index, x=x, y=y, out=out, a=a, b=b, scales=scales, row_offsets=row_offsets,
                            adapter_ids=adapter_ids)
        if rows:
            # long steps' low-rank sums, from the pool of the call's stream and its again after the call
            ws = at = size = 0
            if rows >= self.LONG and self.dtype is not _torch.float32:
                size = decode_attn_adapters_workspace(self.config, rows)
                if size and self._findings:
                    if size > self.workspace_bytes:
                        with _torch.cuda.stream(stream):
                            if _torch.cuda.is_current_stream_capturing():
                                raise ValueError("a captured step needs one as long made ahead of the capture: its "
                                                 "workspace would be cleared by each replay, and by nothing before")
                        if self.workspace is not None:     # graphs may hold its address: kept, and twice as large
                            self._outgrown.append(self.workspace)      # from then on, so that they stay few
                            size = max(size, 2 * self.workspace_bytes)
                        self._make_workspace(size, x.device)
                        self.workspace_bytes = size
                    if self.workspace.get_device() != index:
                        _refuse_devices(index, workspace=self.workspace)
                    at, size = self._workspace_on(index, stream), self.workspace_bytes
                elif size:
                    ws = _empty((size,), _torch.uint8, x.device, stream)
                    at = ws.data_ptr()
            self._apply(self._at, index, stream, x.data_ptr(), y.data_ptr(), out.data_ptr(), a.data_ptr(),
                        b.data_ptr(), scale_at, row_offsets.data_ptr(), adapter_ids.data_ptr(), rows, batch, n,
                        x_row, y_row, out_row, at, size)
        return out

    def check_status(self, stream=None):
        """Synchronise, then raise the finding recorded since the last call, if there is one."""
        if not self._findings:
            raise ValueError("made without findings")
        for ws in self._outgrown + ([self.workspace] if self.workspace is not None else []):
            with _torch.cuda.device(ws.device):
                s = stream if stream is not None else _torch.cuda.current_stream()
                decode_attn_adapters_check_status(ws.data_ptr(), s.cuda_stream)
