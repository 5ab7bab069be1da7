"""The experts' operators on the host, without a GPU: the library's checks of
their arguments (pointers are fake addresses, compared and tested for alignment
but never dereferenced), the workspace's size, and the Python binding's
refusals of CPU tensors."""
import ctypes
import os

import pytest
import torch

from moe_token_re_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="library not built")

AT = {n: (i + 1) << 40 for i, n in enumerate(
    ("tokens", "token_scales", "weight", "weight_scales", "num", "row_weight", "out", "ws", "x", "logits", "ids",
     "expert_weight", "gate_up", "gate_up_scales", "down", "down_scales", "y"))}
OK, VALUE, SHAPE, DTYPE = _lib.SUCCESS, _lib.ERROR_INVALID_VALUE, _lib.ERROR_INVALID_SHAPE, _lib.ERROR_UNSUPPORTED_DTYPE
MISALIGNED, SMALL = _lib.ERROR_MISALIGNED, _lib.ERROR_WORKSPACE_TOO_SMALL


def grouped(ws=None, ws_bytes=0, **change):
    a = _lib.MrrGroupedMmArgs(AT["tokens"], AT["token_scales"], 64, 256, AT["weight"], AT["weight_scales"], 4, 96,
                              AT["num"], _lib.I32, 1, 0, AT["row_weight"], AT["out"], _lib.BF16)
    for k, v in change.items():
        setattr(a, k, v)
    return _lib.load().mrr_grouped_mm_validate(ctypes.byref(a), ws, ws_bytes)


@pytest.mark.parametrize("change,code", [
    ({}, OK), ({"gated": 1}, OK), ({"row_weight": None}, OK), ({"counts_dtype": _lib.I64}, OK),
    ({"expert_token_num_type": 0}, OK), ({"out_dtype": _lib.F32}, OK), ({"out_dtype": _lib.F16}, OK),
    ({"A": 0, "tokens": None, "token_scales": None, "out": None}, OK),
    ({"A": 0, "E": 0, "expert_token_num": None}, OK), ({"K": 32}, OK), ({"N": 1}, OK),
    ({"out_dtype": _lib.I8}, DTYPE), ({"counts_dtype": _lib.F32}, DTYPE),
    ({"gated": 2}, VALUE), ({"expert_token_num_type": 2}, VALUE), ({"tokens": None}, VALUE),
    ({"token_scales": None}, VALUE), ({"weight": None}, VALUE), ({"weight_scales": None}, VALUE),
    ({"out": None}, VALUE), ({"expert_token_num": None}, VALUE), ({"out": AT["tokens"]}, VALUE),
    ({"out": AT["weight"] + 64 * 4 * 96}, VALUE), ({"out": AT["row_weight"] + 4}, VALUE),
    ({"A": -1}, SHAPE), ({"A": 1 << 31}, SHAPE), ({"K": 0}, SHAPE), ({"K": 48}, SHAPE), ({"K": 1 << 20}, SHAPE),
    ({"N": 0}, SHAPE), ({"N": 97, "gated": 1}, SHAPE), ({"N": 1 << 20}, SHAPE), ({"E": -1}, SHAPE),
    ({"E": 4097}, SHAPE), ({"E": 0}, SHAPE),
    ({"tokens": AT["tokens"] + 8}, MISALIGNED), ({"weight": AT["weight"] + 4}, MISALIGNED),
    ({"expert_token_num": AT["num"] + 2}, MISALIGNED), ({"row_weight": AT["row_weight"] + 2}, MISALIGNED),
    ({"out": AT["out"] + 1}, MISALIGNED),
])
def test_grouped_mm_checks(change, code):
    assert grouped(**change) == code


def test_grouped_mm_workspace_checks():
    assert grouped(AT["ws"], 256) == OK
    assert grouped(AT["ws"], 255) == SMALL
    assert grouped(AT["ws"], 0) == VALUE
    assert grouped(None, 256) == VALUE
    assert grouped(AT["ws"] + 8, 256) == MISALIGNED
    assert grouped(AT["out"] + 256, 256) == VALUE
    assert _lib.load().mrr_grouped_mm_validate(None, None, 0) == VALUE


def few(ws=AT["ws"], ws_bytes=1 << 30, **change):
    a = _lib.MrrFewTokensArgs(AT["x"], _lib.BF16, 8, 128, 16, 64, 4, AT["logits"], 1, None, None, _lib.BF16,
                              AT["gate_up"], None, AT["down"], None, AT["y"])
    for k, v in change.items():
        setattr(a, k, v)
    return _lib.load().mrr_few_tokens_validate(ctypes.byref(a), ws, ws_bytes)


GIVEN = {"router_logits": None, "expert_ids": AT["ids"], "expert_weight": AT["expert_weight"]}
MX = {"weights_dtype": _lib.F4_E2M1, "gate_up_scales": AT["gate_up_scales"], "down_scales": AT["down_scales"]}


@pytest.mark.parametrize("change,code", [
    ({}, OK), (GIVEN, OK), (MX, OK), ({**MX, **GIVEN}, OK), ({"dtype": _lib.F16, "weights_dtype": _lib.F16}, OK),
    ({"T": 0, "x": None, "y": None, "router_logits": None}, OK), ({"T": 128}, OK), ({"E": 1024, "top_k": 16}, OK),
    ({"dtype": _lib.F32}, DTYPE), ({"weights_dtype": _lib.F16}, DTYPE), ({"dtype": _lib.F16, **MX}, DTYPE),
    ({"weights_dtype": _lib.F4_E1M2}, DTYPE),
    ({"renormalize": 2}, VALUE), ({"router_logits": None}, VALUE), ({"expert_ids": AT["ids"]}, VALUE),
    ({"expert_weight": AT["expert_weight"]}, VALUE), ({**GIVEN, "expert_weight": None}, VALUE),
    ({"gate_up": None}, VALUE), ({"down": None}, VALUE), ({"x": None}, VALUE), ({"y": None}, VALUE),
    ({"gate_up_scales": AT["gate_up_scales"]}, VALUE), ({**MX, "down_scales": None}, VALUE),
    ({"y": AT["x"] + 16}, VALUE), ({"y": AT["logits"]}, VALUE), ({"y": AT["down"] + 2 * 16 * 128 * 64 - 2}, VALUE),
    ({"T": -1}, SHAPE), ({"T": 129}, SHAPE), ({"H": 0}, SHAPE), ({"H": 40}, SHAPE), ({"H": 65568}, SHAPE),
    ({"I": 0}, SHAPE), ({"I": 48}, SHAPE), ({"I": 65568}, SHAPE), ({"E": 0}, SHAPE), ({"E": 1025}, SHAPE),
    ({"top_k": 0}, SHAPE), ({"top_k": 17}, SHAPE), ({"E": 3}, SHAPE),
    ({"x": AT["x"] + 2}, MISALIGNED), ({"gate_up": AT["gate_up"] + 8}, MISALIGNED),
    ({"down": AT["down"] + 2}, MISALIGNED), ({"router_logits": AT["logits"] + 1}, MISALIGNED),
    ({"y": AT["y"] + 1}, MISALIGNED), ({**GIVEN, "expert_ids": AT["ids"] + 2}, MISALIGNED),
])
def test_few_tokens_checks(change, code):
    assert few(**change) == code


def test_few_tokens_workspace():
    L = _lib.load()
    need = L.mrr_few_tokens_workspace_size(8, 4, 64)
    assert need >= 4 * 8 * 4 + 2 * 8 * 4 * 64
    assert few(ws_bytes=need) == OK and few(ws_bytes=need - 1) == SMALL
    assert few(ws=None) == VALUE and few(ws=AT["ws"] + 4) == MISALIGNED and few(ws=AT["y"] + 256) == VALUE
    for bad in ((-1, 4, 64), (129, 4, 64), (8, 0, 64), (8, 17, 64), (8, 4, 0), (8, 4, 1 << 17)):
        assert L.mrr_few_tokens_workspace_size(*bad) == 0
    assert L.mrr_few_tokens_validate(None, None, 0) == VALUE


@pytest.mark.parametrize("change,code", [
    ({"wide_dtype": _lib.I8}, DTYPE), ({"rows": -1}, SHAPE), ({"H": 0}, SHAPE), ({"H": 33}, SHAPE),
    ({"H": 1 << 24}, SHAPE), ({"rows": 1 << 60}, SHAPE), ({"wide": None}, VALUE), ({"packed": None}, VALUE),
    ({"scales": None}, VALUE), ({"wide": AT["x"] + 1}, MISALIGNED), ({"packed": AT["x"] + 256}, VALUE),
    ({"rows": 0}, OK),
])
def test_conversions_refuse_before_any_launch(change, code):
    """Both directions make the same checks first; without rows nothing is launched."""
    a = _lib.MrrMxArgs(AT["x"], _lib.BF16, 4, 64, AT["tokens"], AT["token_scales"])
    for k, v in change.items():
        setattr(a, k, v)
    L = _lib.load()
    assert L.mrr_mx_quantize(ctypes.byref(a), None) == code
    assert L.mrr_mx_dequantize(ctypes.byref(a), None) == code
    assert L.mrr_mx_quantize(None, None) == VALUE


def test_python_refuses_cpu_tensors():
    import moe_token_re_amd as moe

    x = torch.zeros(2, 64)
    p, s = torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 1, 2, dtype=torch.uint8)
    for call in (lambda: moe.mx_quantize(x), lambda: moe.mx_dequantize(p, s),
                 lambda: moe.mx_grouped_mm(p, s, p[None], s[None], torch.tensor([2])),
                 lambda: moe.moe_few_tokens(x, x, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        moe.mx_quantize([1.0])


@pytest.mark.parametrize("change,code", [
    ({**GIVEN, "E": 4, "top_k": 6}, OK), ({**GIVEN, "E": 1, "top_k": 16}, OK), ({**MX, **GIVEN, "E": 3, "top_k": 8}, OK),
    ({**GIVEN, "E": 4, "top_k": 17}, SHAPE), ({**GIVEN, "E": 0, "top_k": 1}, SHAPE),
    ({"E": 4, "top_k": 5}, SHAPE), ({"E": 4, "top_k": 4}, OK),
    ({"T": 0, "x": None, "y": None, "router_logits": None, "E": 4, "top_k": 6}, OK),
])
def test_few_tokens_more_choices_than_experts(change, code):
    """A token names experts of all ranks, and this one may have fewer; the
    largest logits are chosen among its own."""
    assert few(**change) == code
