"""The operators around an expert layer on the host, without a GPU: the
library's checks of their arguments (fake addresses, never dereferenced), the
workspaces' sizes, and the Python binding's refusals."""
import ctypes
import os

import pytest
import torch

import moe_token_re_amd as moe
from moe_token_re_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="library not built")

NAMES = ("x residual weight y scales sum grad grad_sum grad_x grad_weight logits expert_weight expert_ids grad_logits "
         "tokens per_token_scales permute_tokens permute_per_token_scales permute_token_idx expert_token_num "
         "permute_topk_weight rows row_values choice_values grad_rows ws").split()
AT = {n: (i + 1) << 44 for i, n in enumerate(NAMES)}
OK, VALUE, SHAPE, DTYPE = _lib.SUCCESS, _lib.ERROR_INVALID_VALUE, _lib.ERROR_INVALID_SHAPE, _lib.ERROR_UNSUPPORTED_DTYPE
MISALIGNED, SMALL = _lib.ERROR_MISALIGNED, _lib.ERROR_WORKSPACE_TOO_SMALL


def filled(struct, sizes, absent=()):
    """A struct whose pointers are the fake addresses of their names."""
    a = struct()
    for name, kind in struct._fields_:
        if name in sizes:
            setattr(a, name, sizes[name])
        elif kind is ctypes.c_void_p and name not in absent:
            setattr(a, name, AT[name])
    return a


def check(entry, a, change, *ws):
    for k, v in change.items():
        if k == "scales_dims":
            v = (ctypes.c_int64 * 3)(*v)
        setattr(a, k, v)
    return getattr(_lib.load(), entry)(ctypes.byref(a), *ws)


NORM = dict(dtype=_lib.BF16, rows=8, H=256, weight_dtype=_lib.F32, eps=1e-6, y_dtype=_lib.I8, scales_dtype=_lib.F32)
WIDE = {"y_dtype": _lib.BF16, "scales": None}
MX4 = {"y_dtype": _lib.F4_E2M1, "scales_dtype": _lib.F8_E8M0}


@pytest.mark.parametrize("change,code", [
    ({}, OK), (WIDE, OK), (MX4, OK), ({"y_dtype": _lib.F8_E4M3FN}, OK), ({**MX4, "y_dtype": _lib.F8_E4M3FN}, OK),
    ({"residual": None, "sum": None}, OK), ({"weight_dtype": _lib.BF16}, OK), ({"H": 16384}, OK), ({"H": 1}, OK),
    ({"rows": 0, "x": None, "y": None, "weight": None, "scales": None, "residual": None, "sum": None}, OK),
    ({"eps": 2.0 ** -126}, OK), ({"scales_dtype": -5, **WIDE}, OK),
    ({"dtype": _lib.I8}, DTYPE), ({"weight_dtype": _lib.F16}, DTYPE), ({"y_dtype": _lib.F16}, DTYPE),
    ({"y_dtype": _lib.F8_E5M2}, DTYPE), ({"y_dtype": _lib.F4_E2M1}, DTYPE), ({"scales_dtype": _lib.F8_E8M0}, DTYPE),
    ({"scales_dtype": _lib.F16}, DTYPE), ({"H": 0}, SHAPE), ({"H": 16385}, SHAPE), ({"rows": -1}, SHAPE),
    ({"rows": 1 << 31}, SHAPE), ({**MX4, "H": 33}, SHAPE), ({"eps": 0.0}, VALUE), ({"eps": -1.0}, VALUE),
    ({"eps": float("nan")}, VALUE), ({"eps": float("inf")}, VALUE), ({"eps": 1e-39}, VALUE), ({"x": None}, VALUE),
    ({"y": None}, VALUE), ({"weight": None}, VALUE), ({"scales": None}, VALUE), ({**WIDE, "scales": AT["scales"]}, VALUE),
    ({"sum": None}, VALUE), ({"residual": None}, VALUE), ({"sum": AT["residual"]}, VALUE), ({"y": AT["x"] + 64}, VALUE),
    ({"scales": AT["y"] + 8 * 256 - 4}, VALUE), ({"sum": AT["weight"] + 1020}, VALUE), ({"x": AT["x"] + 1}, MISALIGNED),
    ({"scales": AT["scales"] + 2}, MISALIGNED), ({"weight": AT["weight"] + 2}, MISALIGNED), ({"y": AT["y"] + 1}, OK),
    ({**WIDE, "y": AT["y"] + 1}, MISALIGNED), ({**MX4, "scales": AT["scales"] + 1}, OK),
])
def test_norm_checks(change, code):
    assert check("mrr_rms_norm_validate", filled(_lib.MrrRmsNormArgs, NORM), change) == code


def norm_backward(change, ws=AT["ws"], ws_bytes=1 << 30):
    a = filled(_lib.MrrRmsNormBackwardArgs, dict(dtype=_lib.F16, rows=8, H=256, weight_dtype=_lib.F32, eps=1e-6))
    return check("mrr_rms_norm_backward_validate", a, change, ws, ws_bytes)


@pytest.mark.parametrize("change,code", [
    ({}, OK), ({"grad_sum": None}, OK), ({"weight_dtype": _lib.F16}, OK), ({"dtype": _lib.F32}, OK),
    ({"rows": 0, "x": None, "grad": None, "grad_x": None, "grad_sum": None}, OK),
    ({"dtype": _lib.I8}, DTYPE), ({"weight_dtype": _lib.BF16}, DTYPE), ({"H": 0}, SHAPE), ({"H": 16385}, SHAPE),
    ({"rows": -1}, SHAPE), ({"eps": 0.0}, VALUE), ({"x": None}, VALUE), ({"grad": None}, VALUE), ({"grad_x": None}, VALUE),
    ({"weight": None}, VALUE), ({"grad_weight": None}, VALUE), ({"grad_x": AT["grad"]}, VALUE),
    ({"grad_weight": AT["ws"]}, VALUE), ({"grad_x": AT["grad_x"] + 1}, MISALIGNED), ({"grad_weight": AT["x"] + 2}, MISALIGNED),
])
def test_norm_backward_checks(change, code):
    assert norm_backward(change) == code


def test_norm_backward_workspace():
    L = _lib.load()
    for rows, H in ((1, 1), (8, 256), (100000, 100), (100000, 16384), (0, 64)):
        need = L.mrr_rms_norm_backward_workspace_size(rows, H)
        assert 0 < need <= 256 + 4 * H * 2048 + 256
    need = L.mrr_rms_norm_backward_workspace_size(8, 256)
    assert norm_backward({}, ws_bytes=need) == OK and norm_backward({}, ws_bytes=need - 1) == SMALL
    assert norm_backward({}, ws=None) == VALUE and norm_backward({}, ws=AT["ws"] + 8) == MISALIGNED
    for bad in ((-1, 64), (1 << 31, 64), (8, 0), (8, 16385)):
        assert L.mrr_rms_norm_backward_workspace_size(*bad) == 0


ROUTER = dict(dtype=_lib.F32, T=8, E=64, top_k=4, renormalize=1)
ROUTER_BAD = [
    ({}, OK), ({"dtype": _lib.BF16}, OK), ({"renormalize": 0}, OK), ({"E": 1024, "top_k": 16}, OK), ({"E": 1, "top_k": 1}, OK),
    ({"T": 0, "logits": None, "expert_weight": None, "expert_ids": None}, OK),
    ({"dtype": _lib.I8}, DTYPE), ({"T": -1}, SHAPE), ({"T": 1 << 31}, SHAPE), ({"E": 0}, SHAPE), ({"E": 1025}, SHAPE),
    ({"top_k": 0}, SHAPE), ({"top_k": 17}, SHAPE), ({"E": 3}, SHAPE), ({"renormalize": 2}, VALUE), ({"expert_ids": None}, VALUE),
    ({"expert_weight": None}, VALUE), ({"logits": AT["logits"] + 2}, MISALIGNED), ({"expert_ids": AT["expert_ids"] + 2}, MISALIGNED),
]


@pytest.mark.parametrize("change,code", ROUTER_BAD + [
    ({"logits": None}, VALUE), ({"expert_ids": AT["expert_weight"] + 4}, VALUE), ({"expert_weight": AT["logits"]}, VALUE)])
def test_router_checks(change, code):
    assert check("mrr_router_validate", filled(_lib.MrrRouterArgs, ROUTER), change) == code


@pytest.mark.parametrize("change,code", ROUTER_BAD + [
    ({"logits": None}, OK), ({"logits": None, "renormalize": 0}, VALUE), ({"grad_weight": None}, VALUE),
    ({"grad_logits": None}, VALUE), ({"grad_logits": AT["logits"]}, VALUE), ({"grad_logits": AT["grad_logits"] + 2}, MISALIGNED)])
def test_router_backward_checks(change, code):
    assert check("mrr_router_backward_validate", filled(_lib.MrrRouterBackwardArgs, ROUTER), change) == code


def permute(change, ws=AT["ws"], ws_bytes=1 << 30):
    a = filled(_lib.MrrTokenPermuteArgs, dict(tokens_dtype=_lib.I8, T=8, H=256, top_k=4, E=64, scales_dtype=_lib.F32,
                                              scales_ndim=1, expert_token_num_type=1))
    a.scales_dims[0] = 8
    return check("mrr_token_permute_validate", a, change, ws, ws_bytes)


NO_SCALES = {"per_token_scales": None, "permute_per_token_scales": None}


@pytest.mark.parametrize("change,code", [
    ({}, OK), (NO_SCALES, OK), ({"scales_ndim": 2, "scales_dims": (8, 7, 0)}, OK), ({"tokens_dtype": _lib.F32}, OK),
    ({"scales_dtype": _lib.F8_E8M0, "scales_ndim": 3, "scales_dims": (8, 4, 2)}, OK), ({"tokens_dtype": _lib.F4_E1M2}, OK),
    ({"expert_weight": None, "permute_topk_weight": None}, OK), ({"E": 4096, "top_k": 16, "H": 65536}, OK),
    ({"T": 0, "tokens": None, "expert_ids": None, "permute_tokens": None, "permute_token_idx": None, "scales_dims": (0, 0, 0)}, OK),
    ({**NO_SCALES, "scales_dtype": 99}, OK), ({"expert_token_num_type": 0}, OK),
    ({"tokens_dtype": _lib.I32}, DTYPE), ({"scales_dtype": _lib.F16}, DTYPE), ({"T": -1}, SHAPE),
    ({"T": (1 << 31) // 4}, SHAPE), ({"top_k": 0}, SHAPE), ({"top_k": 17}, SHAPE), ({"E": 0}, SHAPE), ({"E": 4097}, SHAPE),
    ({"H": 0}, SHAPE), ({"H": 65537}, SHAPE), ({"tokens_dtype": _lib.F4_E2M1, "H": 33}, SHAPE), ({"scales_ndim": 0}, SHAPE),
    ({"scales_ndim": 3}, SHAPE), ({"scales_dims": (7, 0, 0)}, SHAPE), ({"scales_ndim": 2, "scales_dims": (8, 0, 0)}, SHAPE),
    ({"scales_dtype": _lib.F8_E8M0, "scales_ndim": 3, "scales_dims": (8, 5, 2)}, SHAPE), ({"expert_token_num_type": 2}, VALUE),
    ({"tokens": None}, VALUE), ({"expert_ids": None}, VALUE), ({"permute_tokens": None}, VALUE),
    ({"permute_token_idx": None}, VALUE), ({"expert_token_num": None}, VALUE), ({"per_token_scales": None}, VALUE),
    ({"permute_per_token_scales": None}, VALUE), ({"expert_weight": None}, VALUE), ({"permute_topk_weight": None}, VALUE),
    ({"permute_tokens": AT["tokens"] + 8}, VALUE), ({"permute_token_idx": AT["expert_ids"] + 4}, VALUE),
    ({"permute_topk_weight": AT["permute_tokens"] + 4 * 8 * 256 - 4}, VALUE),
    ({"expert_ids": AT["expert_ids"] + 2}, MISALIGNED), ({"per_token_scales": AT["x"] + 2}, MISALIGNED),
    ({"tokens_dtype": _lib.F16, "tokens": AT["tokens"] + 1}, MISALIGNED), ({"tokens": AT["tokens"] + 1}, OK),
])
def test_permute_checks(change, code):
    assert permute(change) == code


def test_permute_workspace():
    L = _lib.load()
    for T, k, E in ((0, 1, 1), (8, 4, 64), (100000, 16, 4096), (1 << 27, 8, 256)):
        need = L.mrr_token_permute_workspace_size(T, k, E)
        assert 0 < need <= 256 + 4 * 64 * (E + 1) + 256
    many = {"T": 4097, "scales_dims": (4097, 0, 0)}
    need = L.mrr_token_permute_workspace_size(4097, 4, 64)
    assert permute(many, ws_bytes=need) == OK and permute(many, ws_bytes=need - 1) == SMALL
    assert permute(many, ws=None, ws_bytes=0) == VALUE and permute(many, ws=AT["ws"] + 4) == MISALIGNED
    assert permute({**many, "expert_token_num": AT["ws"]}) == VALUE
    alone = {"T": 4096, "scales_dims": (4096, 0, 0)}  # few choices use none
    assert permute(alone, ws=None, ws_bytes=0) == OK and permute({}, ws=None, ws_bytes=0) == OK
    for bad in ((-1, 4, 64), (1 << 30, 4, 64), (8, 0, 64), (8, 17, 64), (8, 4, 0), (8, 4, 4097)):
        assert L.mrr_token_permute_workspace_size(*bad) == 0


SUM = dict(dtype=_lib.BF16, R=32, H=256, T=8, top_k=4)
SUM_BAD = [
    ({}, OK), ({"dtype": _lib.F32}, OK), ({"H": 65536, "top_k": 16, "T": 1}, OK), ({"dtype": _lib.I8}, DTYPE),
    ({"R": -1}, SHAPE), ({"R": 1 << 31}, SHAPE), ({"H": 0}, SHAPE), ({"H": 65537}, SHAPE), ({"T": -1}, SHAPE),
    ({"T": 1 << 29}, SHAPE), ({"top_k": 0}, SHAPE), ({"top_k": 17}, SHAPE), ({"rows": None}, VALUE),
    ({"permute_token_idx": None}, VALUE), ({"rows": AT["rows"] + 1}, MISALIGNED),
    ({"permute_token_idx": AT["permute_token_idx"] + 1}, MISALIGNED), ({"expert_weight": AT["expert_weight"] + 2}, MISALIGNED),
]


@pytest.mark.parametrize("change,code", SUM_BAD + [
    ({"expert_weight": None}, OK), ({"row_values": None, "choice_values": None}, OK), ({"R": 0, "rows": None, "row_values": None}, OK),
    ({"T": 0, "permute_token_idx": None, "y": None, "choice_values": None}, OK), ({"y": None}, VALUE),
    ({"row_values": None}, VALUE), ({"choice_values": None}, VALUE), ({"y": AT["rows"]}, VALUE),
    ({"choice_values": AT["row_values"]}, VALUE), ({"y": AT["y"] + 1}, MISALIGNED)])
def test_unpermute_checks(change, code):
    assert check("mrr_token_unpermute_validate", filled(_lib.MrrTokenUnpermuteArgs, SUM), change) == code


@pytest.mark.parametrize("change,code", SUM_BAD + [
    ({"expert_weight": None, "grad_weight": None, "rows": None}, OK), ({"R": 0, "rows": None, "grad_rows": None}, OK),
    ({"T": 0, "grad": None, "permute_token_idx": None, "grad_weight": None}, OK), ({"grad": None}, VALUE),
    ({"grad_rows": None}, VALUE), ({"grad_weight": None}, VALUE), ({"expert_weight": None}, VALUE),
    ({"grad_rows": AT["rows"]}, VALUE), ({"grad_weight": AT["permute_token_idx"]}, VALUE), ({"grad": AT["grad"] + 1}, MISALIGNED)])
def test_unpermute_backward_checks(change, code):
    assert check("mrr_token_unpermute_backward_validate", filled(_lib.MrrTokenUnpermuteBackwardArgs, SUM), change) == code


def test_no_arguments_at_all():
    L = _lib.load()
    for name in ("rms_norm", "router", "router_backward", "token_unpermute", "token_unpermute_backward"):
        assert getattr(L, f"mrr_{name}_validate")(None) == VALUE and getattr(L, f"mrr_{name}")(None, None) == VALUE
    for name in ("rms_norm_backward", "token_permute"):
        assert getattr(L, f"mrr_{name}_validate")(None, None, 0) == VALUE
        assert getattr(L, f"mrr_{name}")(None, None, 0, None) == VALUE


def test_launching_calls_refuse_before_any_launch():
    """The checks come first: these return without a GPU."""
    L = _lib.load()
    for name, struct, sizes in (("rms_norm", _lib.MrrRmsNormArgs, NORM), ("router", _lib.MrrRouterArgs, ROUTER),
                                ("router_backward", _lib.MrrRouterBackwardArgs, ROUTER),
                                ("token_unpermute", _lib.MrrTokenUnpermuteArgs, SUM),
                                ("token_unpermute_backward", _lib.MrrTokenUnpermuteBackwardArgs, SUM)):
        a = filled(struct, sizes)
        a.dtype = _lib.I64
        assert getattr(L, f"mrr_{name}")(ctypes.byref(a), None) == DTYPE
    a = filled(_lib.MrrTokenPermuteArgs, dict(tokens_dtype=_lib.I64))
    assert L.mrr_token_permute(ctypes.byref(a), None, 0, None) == DTYPE
    a = filled(_lib.MrrRmsNormBackwardArgs, dict(dtype=_lib.I64))
    assert L.mrr_rms_norm_backward(ctypes.byref(a), None, 0, None) == DTYPE


def test_python_refuses_cpu_tensors():
    x, i = torch.zeros(2, 64), torch.zeros(2, 1, dtype=torch.int32)
    w = torch.ones(64)
    for call in (lambda: moe.rms_norm(x, w), lambda: moe.rms_norm_backward(x, x, w), lambda: moe.moe_router_top_k(x, 2),
                 lambda: moe.moe_router_top_k_backward(x, x, x, i), lambda: moe.moe_token_permute(x, i, 4),
                 lambda: moe.moe_token_permute_backward(x, i), lambda: moe.moe_token_unpermute(x, i),
                 lambda: moe.moe_token_unpermute_backward(x, x, i)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: moe.rms_norm([1.0], w), lambda: moe.moe_router_top_k(None, 2)):
        with pytest.raises(TypeError):
            call()


def test_binding_leaves_cpu_tensors_alone():
    b = _lib.binding()
    x, i = torch.zeros(2, 64), torch.zeros(2, 1, dtype=torch.int32)
    w = torch.ones(64)
    assert b.rms_norm(x, w, None, 1e-6, None) is None and b.rms_norm_backward(x, x, w, None, 1e-6) is None
    assert b.router(x, 2, True) is None and b.router_backward(x, x, x, i, True) is None
    assert b.permute(x, i, 4, None, None, 1) is None and b.unpermute(x, i, None) is None
    assert b.unpermute_backward(x, x, i, None) is None and b.permute_backward(x, i, None) is None
    for call in (b.rms_norm, b.rms_norm_backward, b.router, b.router_backward, b.permute, b.permute_backward, b.unpermute,
                 b.unpermute_backward):
        for n in range(8):
            assert call(*[None] * n) is None
