"""ctypes view of the C ABI in include/moe_rerouting_v2.h.

Loads the in-tree libmoe_rerouting_v2.so. There is no fallback: if the library
has not been built, loading raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_rerouting_v2.so")

# mrr_status
SUCCESS = 0
ERROR_INVALID_VALUE = 1
ERROR_INVALID_SHAPE = 2
ERROR_UNSUPPORTED_DTYPE = 3
ERROR_MISALIGNED = 4
ERROR_WORKSPACE_TOO_SMALL = 5
ERROR_BAD_COUNTS = 6
ERROR_HIP = 7

# mrr_args.direction
FORWARD = 0
INVERSE = 1

# mrr_dtype
F16, BF16, I8, F8_E5M2, F8_E4M3FN, HIF8, F4_E2M1, F4_E1M2, I32, I64, F32, F8_E8M0 = range(12)

EXPORTS = ("mrr_workspace_size", "mrr_validate", "mrr_describe_plan", "moe_rerouting_v2",
           "moe_rerouting_v2_offsets", "moe_rerouting_v2_gather", "mrr_get_device_status", "mrr_status_string",
           "mrr_source_hash", "moe_rerouting_v2_noalloc", "mrr_mx_quantize", "mrr_mx_dequantize",
           "mrr_grouped_mm_validate", "mrr_mx_grouped_mm", "mrr_few_tokens_workspace_size",
           "mrr_few_tokens_validate", "mrr_few_tokens")
NOALLOC_SCRATCH_BYTES = 8 << 20  # MRR_NOALLOC_SCRATCH_BYTES


class MrrArgs(ctypes.Structure):
    """struct mrr_args, field for field."""

    _fields_ = [
        ("tokens", ctypes.c_void_p),
        ("tokens_dtype", ctypes.c_int32),
        ("A", ctypes.c_int64),
        ("H", ctypes.c_int64),
        ("expert_token_num_per_rank", ctypes.c_void_p),
        ("counts_dtype", ctypes.c_int32),
        ("N", ctypes.c_int64),
        ("E", ctypes.c_int64),
        ("per_token_scales", ctypes.c_void_p),
        ("scales_dtype", ctypes.c_int32),
        ("scales_ndim", ctypes.c_int32),
        ("scales_dims", ctypes.c_int64 * 3),
        ("expert_topk_weight", ctypes.c_void_p),
        ("permute_tokens", ctypes.c_void_p),
        ("permute_per_token_scales", ctypes.c_void_p),
        ("permute_token_idx", ctypes.c_void_p),
        ("expert_token_num", ctypes.c_void_p),
        ("permute_topk_weight", ctypes.c_void_p),
        ("expert_token_num_type", ctypes.c_int64),
        ("idx_type", ctypes.c_int64),
        ("direction", ctypes.c_int64),
    ]


class MrrPlanInfo(ctypes.Structure):
    """struct mrr_plan_info, field for field."""

    _fields_ = [
        ("fused", ctypes.c_int32),
        ("token_vec_bytes", ctypes.c_int32),
        ("scale_vec_bytes", ctypes.c_int32),
        ("rows_per_workgroup", ctypes.c_int32),
        ("threads_per_workgroup", ctypes.c_int32),
        ("gather_workgroups", ctypes.c_int64),
        ("token_row_bytes", ctypes.c_int64),
        ("scale_row_bytes", ctypes.c_int64),
        ("scale_inline_bytes", ctypes.c_int32),
        ("offsets_workgroups", ctypes.c_int64),
        ("gather_kernel", ctypes.c_int32),
        ("gather_launches", ctypes.c_int64),
        ("one_launch_workgroups", ctypes.c_int64),
    ]


class MrrMxArgs(ctypes.Structure):
    """struct mrr_mx_args, field for field."""

    _fields_ = [
        ("wide", ctypes.c_void_p),
        ("wide_dtype", ctypes.c_int32),
        ("rows", ctypes.c_int64),
        ("H", ctypes.c_int64),
        ("packed", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
    ]


class MrrGroupedMmArgs(ctypes.Structure):
    """struct mrr_grouped_mm_args, field for field."""

    _fields_ = [
        ("tokens", ctypes.c_void_p),
        ("token_scales", ctypes.c_void_p),
        ("A", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("weight", ctypes.c_void_p),
        ("weight_scales", ctypes.c_void_p),
        ("E", ctypes.c_int64),
        ("N", ctypes.c_int64),
        ("expert_token_num", ctypes.c_void_p),
        ("counts_dtype", ctypes.c_int32),
        ("expert_token_num_type", ctypes.c_int64),
        ("gated", ctypes.c_int64),
        ("row_weight", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("out_dtype", ctypes.c_int32),
    ]


class MrrFewTokensArgs(ctypes.Structure):
    """struct mrr_few_tokens_args, field for field."""

    _fields_ = [
        ("x", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("T", ctypes.c_int64),
        ("H", ctypes.c_int64),
        ("E", ctypes.c_int64),
        ("I", ctypes.c_int64),
        ("top_k", ctypes.c_int64),
        ("router_logits", ctypes.c_void_p),
        ("renormalize", ctypes.c_int64),
        ("expert_ids", ctypes.c_void_p),
        ("expert_weight", ctypes.c_void_p),
        ("weights_dtype", ctypes.c_int32),
        ("gate_up", ctypes.c_void_p),
        ("gate_up_scales", ctypes.c_void_p),
        ("down", ctypes.c_void_p),
        ("down_scales", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
    ]


_lock = threading.Lock()
_lib = None


def load() -> ctypes.CDLL:
    """The loaded library; raises RuntimeError if it has not been built, or was
    built from sources other than the ones beside it (mrr_source_hash)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with `python -m moe_token_re_amd.build` "
                    "(there is no CPU fallback)")
            from . import build

            lib = ctypes.CDLL(LIB_PATH)
            if not hasattr(lib, "mrr_source_hash"):
                raise RuntimeError(f"{LIB_PATH} carries no source hash: rebuild it "
                                   "with `python -m moe_token_re_amd.build`")
            lib.mrr_source_hash.argtypes = []
            lib.mrr_source_hash.restype = ctypes.c_char_p
            built, current = lib.mrr_source_hash().decode(), build.source_hash()
            if built != current:
                raise RuntimeError(f"{LIB_PATH} was built from other sources (hash {built}, sources {current}): "
                                   "rebuild it with `python -m moe_token_re_amd.build`")
            P = ctypes.POINTER(MrrArgs)
            vp, sz = ctypes.c_void_p, ctypes.c_size_t
            lib.mrr_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]
            lib.mrr_workspace_size.restype = sz
            lib.mrr_validate.argtypes = [P, vp, sz]
            lib.mrr_validate.restype = ctypes.c_int
            lib.mrr_describe_plan.argtypes = [P, vp, sz, ctypes.POINTER(MrrPlanInfo)]
            lib.mrr_describe_plan.restype = ctypes.c_int
            for name in ("moe_rerouting_v2", "moe_rerouting_v2_offsets", "moe_rerouting_v2_gather"):
                fn = getattr(lib, name)
                fn.argtypes = [P, vp, sz, vp]
                fn.restype = ctypes.c_int
            lib.moe_rerouting_v2_noalloc.argtypes = [P, vp]
            lib.moe_rerouting_v2_noalloc.restype = ctypes.c_int
            lib.mrr_get_device_status.argtypes = [vp, vp]
            lib.mrr_get_device_status.restype = ctypes.c_int
            for name in ("mrr_mx_quantize", "mrr_mx_dequantize"):
                fn = getattr(lib, name)
                fn.argtypes = [ctypes.POINTER(MrrMxArgs), vp]
                fn.restype = ctypes.c_int
            for name, struct in (("grouped_mm", MrrGroupedMmArgs), ("few_tokens", MrrFewTokensArgs)):
                check = getattr(lib, f"mrr_{name}_validate")
                check.argtypes = [ctypes.POINTER(struct), vp, sz]
                check.restype = ctypes.c_int
            lib.mrr_mx_grouped_mm.argtypes = [ctypes.POINTER(MrrGroupedMmArgs), vp, sz, vp]
            lib.mrr_mx_grouped_mm.restype = ctypes.c_int
            lib.mrr_few_tokens.argtypes = [ctypes.POINTER(MrrFewTokensArgs), vp, sz, vp]
            lib.mrr_few_tokens.restype = ctypes.c_int
            lib.mrr_few_tokens_workspace_size.argtypes = [ctypes.c_int64] * 3
            lib.mrr_few_tokens_workspace_size.restype = sz
            lib.mrr_status_string.argtypes = [ctypes.c_int]
            lib.mrr_status_string.restype = ctypes.c_char_p
            _lib = lib
        return _lib


_binding = None


def binding():
    """The native binding of the experts' operators (_mrr_torch.so), built with
    the library; raises RuntimeError like load()."""
    global _binding
    if _binding is None:
        load()
        import torch  # noqa: F401  (the binding needs its libraries, wherever they are)

        try:
            from . import _mrr_torch
        except ImportError as e:
            raise RuntimeError("the native binding is missing or does not fit this torch: build it with "
                               "`python -m moe_token_re_amd.build`") from e
        if _mrr_torch.source_hash != library_source_hash():
            raise RuntimeError("_mrr_torch.so was built from other sources: rebuild it with "
                               "`python -m moe_token_re_amd.build`")
        _binding = _mrr_torch
    return _binding


class _NoBinding:
    """In the place of a binding that is not there: it makes no call."""

    quantize = dequantize = grouped_mm = few_tokens = staticmethod(lambda *args: None)


_plain_calls = None


def plain_calls():
    """What makes the experts' operators' plain calls: the native binding, or, where
    it was not built or does not fit, nothing: the Python code beside it makes every
    call then, more slowly, and a warning says so once. The library itself has to be
    there, as for load()."""
    global _plain_calls
    if _plain_calls is None:
        load()
        try:
            _plain_calls = binding()
        except RuntimeError as e:
            warnings.warn(f"{e}; until then small calls take about twice the host time", RuntimeWarning, stacklevel=3)
            _plain_calls = _NoBinding
    return _plain_calls


def library_source_hash() -> str:
    """The source hash compiled into the loaded library (equal to the current
    sources' hash, or load() would have refused it)."""
    return load().mrr_source_hash().decode()


def status_string(code: int) -> str:
    return load().mrr_status_string(code).decode()
