"""Python binding of the experts' operators on MI355X: microscaled 4-bit rows
(mx_quantize, mx_dequantize), the experts' product over expert-major rows
(mx_grouped_mm) and the whole layer for a few tokens (moe_few_tokens).

Argument marshalling only, as in api.py: torch provides device memory and the
current stream; every step runs in the HIP kernels of libmoe_rerouting_v2.so,
and there is no CPU fallback. A plain call goes by the native binding
(csrc/mrr_torch.cpp), which launches it or returns None; the code here makes
every other call (all of them, by ctypes, where the binding is not built) and
raises every error. The operators serve inference: their
results carry no gradient.

The microscaled format is the one moe_re_routing moves: a row of H values is a
row of float4_e2m1fn_x2 [H/2] (two values a byte, the first in the low nibble)
and a row of float8_e8m0fnu scales [ceil(H/64), 2], one for 32 values.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from .api import _check_tensor, _ptr, _raise

_WIDE = {torch.float16: _lib.F16, torch.bfloat16: _lib.BF16, torch.float32: _lib.F32}
_COUNTS = {torch.int32: _lib.I32, torch.int64: _lib.I64}
_PACKED = (torch.float4_e2m1fn_x2, torch.uint8)
_SCALES = (torch.float8_e8m0fnu, torch.uint8)
FEW_TOKENS_MAX = 128  # MRR_FEW_TOKENS_MAX
GROUPED_MM_WORKSPACE_BYTES = 256  # MRR_GROUPED_MM_WORKSPACE_BYTES


# The current stream's handle by device index, without a Stream object around it
# (0.1 us against 1.8 us, of a call of about 8).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _gpu(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device (there is no CPU path)")
    return t.device


def _call(fn, where, dev, *args):
    """Calls a library entry point on dev's current stream."""
    index = dev.index
    if index == torch.cuda.current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(index))
    if st != _lib.SUCCESS:
        _raise(st, where)


def _check_mx(name, packed, scales, dev, lead=None):
    """Checks a pair of packed rows and scales; returns (leading shape, values per row)."""
    _check_tensor(name, packed, dev)
    _check_tensor(name, scales, dev)
    if packed.dtype not in _PACKED:
        raise TypeError(f"{name} must be float4_e2m1fn_x2 (or its bytes as uint8), got {packed.dtype}")
    if scales.dtype not in _SCALES:
        raise TypeError(f"{name} scales must be float8_e8m0fnu (or uint8), got {scales.dtype}")
    shape = tuple(packed.shape)
    if len(shape) != (lead + 1 if lead is not None else max(1, len(shape))):
        raise ValueError(f"{name} has shape {shape}" + (f", expected {lead + 1} dimensions" if lead else ""))
    values = 2 * shape[-1]
    rows = shape[:-1]
    if scales.shape != rows + ((values + 63) // 64, 2):
        raise ValueError(f"{name} scales have shape {tuple(scales.shape)}, expected {rows + ((values + 63) // 64, 2)}")
    return rows, values


def _mx_args(wide, packed, scales):
    H = wide.shape[-1]
    return _lib.MrrMxArgs(wide.data_ptr(), _WIDE[wide.dtype], wide.numel() // H if H else 0, H, packed.data_ptr(),
                          scales.data_ptr())


def mx_quantize(x: torch.Tensor, *, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """Rounds rows x [..., H] (float16, bfloat16 or float32, H even) to
    microscaled 4-bit rows. Returns (packed, scales): float4_e2m1fn_x2
    [..., H/2] and float8_e8m0fnu [..., ceil(H/64), 2], as moe_re_routing takes
    them for tokens and per_token_scales. Each 32 values share the scale
    2^(floor(log2(max |x|)) - 2); values are rounded to nearest, ties to even,
    and saturate at 6 times the scale. A block that holds a NaN or an infinity
    becomes NaN as a whole."""
    if out is None:
        done = _lib.plain_calls().quantize(x)
        if done is not None:
            return done
    dev = _gpu("x", x)
    _check_tensor("x", x, dev)
    if x.dtype not in _WIDE:
        raise TypeError(f"x must be float16, bfloat16 or float32, got {x.dtype}")
    if x.dim() < 1 or x.shape[-1] == 0 or x.shape[-1] % 2:
        raise ValueError(f"x must hold rows of an even number of values, got shape {tuple(x.shape)}")
    *lead, H = x.shape
    lead = tuple(lead)
    if out is None:
        packed = torch.empty(lead + (H // 2,), dtype=torch.float4_e2m1fn_x2, device=dev)
        scales = torch.empty(lead + ((H + 63) // 64, 2), dtype=torch.float8_e8m0fnu, device=dev)
    else:
        packed, scales = out
        if _check_mx("out", packed, scales, dev) != (lead, H):
            raise ValueError(f"out holds rows {tuple(packed.shape)}, expected {lead + (H // 2,)}")
    _call(_lib.load().mrr_mx_quantize, "mrr_mx_quantize", dev, ctypes.byref(_mx_args(x, packed, scales)))
    return packed, scales


def mx_dequantize(packed: torch.Tensor, scales: torch.Tensor, *, dtype: torch.dtype = torch.bfloat16,
                  out: Optional[torch.Tensor] = None):
    """The values of microscaled 4-bit rows (as mx_quantize returns them), rounded
    once to `dtype` (float16, bfloat16 or float32): [..., H]."""
    if out is None:
        done = _lib.plain_calls().dequantize(packed, scales, dtype)
        if done is not None:
            return done
    dev = _gpu("packed", packed)
    lead, H = _check_mx("packed", packed, scales, dev)
    if H == 0:
        raise ValueError("packed holds rows without values")
    if out is None:
        if dtype not in _WIDE:
            raise TypeError(f"dtype must be float16, bfloat16 or float32, got {dtype}")
        out = torch.empty(lead + (H,), dtype=dtype, device=dev)
    else:
        _check_tensor("out", out, dev)
        if out.dtype not in _WIDE:
            raise TypeError(f"out must be float16, bfloat16 or float32, got {out.dtype}")
        if tuple(out.shape) != lead + (H,):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {lead + (H,)}")
    _call(_lib.load().mrr_mx_dequantize, "mrr_mx_dequantize", dev, ctypes.byref(_mx_args(out, packed, scales)))
    return out


def mx_grouped_mm(tokens: torch.Tensor, scales: torch.Tensor, weight: torch.Tensor, weight_scales: torch.Tensor,
                  expert_token_num: torch.Tensor, *, gated: bool = False, row_weight: Optional[torch.Tensor] = None,
                  expert_token_num_type: int = 1, dtype: torch.dtype = torch.bfloat16,
                  out: Optional[torch.Tensor] = None, check: bool = False,
                  workspace: Optional[torch.Tensor] = None):
    """The experts' product over expert-major rows, as moe_re_routing returns
    them: out[r] = weight[e(r)] @ tokens[r], times row_weight[r] where given
    (permute_topk_weight). All operands are microscaled 4-bit rows: tokens
    [A, K/2] with scales [A, ceil(K/64), 2], and weight [E, N, K/2] with
    weight_scales [E, N, ceil(K/64), 2]; K is a multiple of 32. expert_token_num
    [E] says how many rows each expert has (or, with expert_token_num_type=0,
    their running sum). With gated=True the first N/2 rows of a weight are its
    gate and the others its up projection, and out[r] = silu(gate) * up.

    Returns out [A, N] (or [A, N/2]) of `dtype`; sums are kept in 32 bits. The
    counts are checked on the device: where they are negative or do not sum to
    A nothing is written, and with check=True the call waits for the stream and
    raises MrrValueError."""
    if out is None and workspace is None and not check:
        done = _lib.plain_calls().grouped_mm(tokens, scales, weight, weight_scales, expert_token_num, gated, row_weight,
                                         expert_token_num_type, dtype)
        if done is not None:
            return done
    dev = _gpu("tokens", tokens)
    (A,), K = _check_mx("tokens", tokens, scales, dev, 1)
    (E, N), wk = _check_mx("weight", weight, weight_scales, dev, 2)
    if wk != K:
        raise ValueError(f"weight has rows of {wk} values, tokens of {K}")
    _check_tensor("expert_token_num", expert_token_num, dev)
    if expert_token_num.dtype not in _COUNTS:
        raise TypeError(f"expert_token_num must be int32 or int64, got {expert_token_num.dtype}")
    if expert_token_num.shape != (E,):
        raise ValueError(f"expert_token_num has shape {tuple(expert_token_num.shape)}, expected {(E,)}")
    if row_weight is not None:
        _check_tensor("row_weight", row_weight, dev)
        if row_weight.dtype != torch.float32:
            raise TypeError("row_weight must be float32")
        if row_weight.numel() != A or row_weight.dim() > 2:
            raise ValueError(f"row_weight has shape {tuple(row_weight.shape)}, expected [{A}] or [{A}, 1]")
    cols = N // 2 if gated else N
    if out is None:
        if dtype not in _WIDE:
            raise TypeError(f"dtype must be float16, bfloat16 or float32, got {dtype}")
        out = torch.empty((A, cols), dtype=dtype, device=dev)
    else:
        _check_tensor("out", out, dev)
        if out.dtype not in _WIDE:
            raise TypeError(f"out must be float16, bfloat16 or float32, got {out.dtype}")
        if tuple(out.shape) != (A, cols):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(A, cols)}")
    if workspace is not None:
        _check_tensor("workspace", workspace, dev)
    elif check:
        workspace = torch.empty((GROUPED_MM_WORKSPACE_BYTES,), dtype=torch.uint8, device=dev)
    args = _lib.MrrGroupedMmArgs(tokens.data_ptr(), scales.data_ptr(), A, K, weight.data_ptr(),
                                 weight_scales.data_ptr(), E, N, expert_token_num.data_ptr(),
                                 _COUNTS[expert_token_num.dtype], int(expert_token_num_type), int(gated),
                                 _ptr(row_weight), out.data_ptr(), _WIDE[out.dtype])
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _call(_lib.load().mrr_mx_grouped_mm, "mrr_mx_grouped_mm", dev, ctypes.byref(args), _ptr(workspace), ws_bytes)
    if check:
        with torch.cuda.device(dev):
            st = _lib.load().mrr_get_device_status(workspace.data_ptr(), _raw_stream(dev.index))
        if st != _lib.SUCCESS:
            _raise(st, "device count check")
    return out


def few_tokens_workspace_size(T: int, top_k: int, I: int) -> int:
    """Bytes of workspace moe_few_tokens needs for T tokens of top_k experts of I values."""
    return int(_lib.load().mrr_few_tokens_workspace_size(T, top_k, I))


def moe_few_tokens(x: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor, *,
                   router_logits: Optional[torch.Tensor] = None, top_k: Optional[int] = None,
                   renormalize: bool = True, expert_ids: Optional[torch.Tensor] = None,
                   expert_weight: Optional[torch.Tensor] = None, gate_up_scales: Optional[torch.Tensor] = None,
                   down_scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """A whole mixture-of-experts layer for a few tokens (at most 128), in two or
    three kernels: y[t] = sum over the chosen experts of p * down @ (silu(gate @ x[t]) * (up @ x[t])).

    x is [T, H] float16 or bfloat16. gate_up [E, 2 I, H] (the gate's rows, then
    up's) and down [E, H, I] have x's dtype, or are microscaled 4-bit rows
    ([E, 2 I, H/2] and [E, H, I/2] with gate_up_scales and down_scales, as
    mx_quantize makes them; x is then bfloat16). H and I are multiples of 32.

    Routing: router_logits [T, E] float32 with top_k (the largest logits, ties
    to the lowest expert, weighted by the softmax over all experts, or with
    renormalize=True over the chosen ones; an expert of logit -inf is never
    chosen), or expert_ids [T, k] int32 with expert_weight [T, k] float32 (an id
    outside [0, E) chooses nothing, and k may be more than E: experts of other ranks). Returns y [T, H] of x's dtype; a token
    without experts gives zeros."""
    if out is None and workspace is None:
        done = _lib.plain_calls().few_tokens(x, gate_up, down, router_logits, top_k, renormalize, expert_ids,
                                         expert_weight, gate_up_scales, down_scales)
        if done is not None:
            return done
    dev = _gpu("x", x)
    _check_tensor("x", x, dev)
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"x must be float16 or bfloat16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    T, H = x.shape
    mx = gate_up_scales is not None or down_scales is not None
    if mx:
        if gate_up_scales is None or down_scales is None:
            raise ValueError("gate_up_scales and down_scales come together")
        (E, rows), h = _check_mx("gate_up", gate_up, gate_up_scales, dev, 2)
        (e2, h2), inner = _check_mx("down", down, down_scales, dev, 2)
        weights = _lib.F4_E2M1
    else:
        _check_tensor("gate_up", gate_up, dev)
        _check_tensor("down", down, dev)
        if gate_up.dtype != x.dtype or down.dtype != x.dtype:
            raise TypeError(f"the weights must have x's dtype {x.dtype}, or be 4-bit rows with scales; "
                            f"got {gate_up.dtype} and {down.dtype}")
        if gate_up.dim() != 3 or down.dim() != 3:
            raise ValueError("gate_up and down must be 3-D")
        E, rows, h = gate_up.shape
        e2, h2, inner = down.shape
        weights = _WIDE[x.dtype]
    if h != H or h2 != H or e2 != E or rows != 2 * inner:
        raise ValueError(f"gate_up [{E}, {rows}, {h}] and down [{e2}, {h2}, {inner}] do not fit x [{T}, {H}]")
    if (router_logits is None) == (expert_ids is None):
        raise ValueError("give either router_logits or expert_ids")
    if router_logits is not None:
        _check_tensor("router_logits", router_logits, dev)
        if router_logits.dtype != torch.float32:
            raise TypeError("router_logits must be float32")
        if router_logits.shape != (T, E):
            raise ValueError(f"router_logits have shape {tuple(router_logits.shape)}, expected {(T, E)}")
        if expert_weight is not None:
            raise ValueError("expert_weight goes with expert_ids")
        if top_k is None:
            raise ValueError("router_logits need top_k")
        if top_k > E:  # without tokens the library gets no logits to see it by
            _raise(_lib.ERROR_INVALID_SHAPE, "mrr_few_tokens")
    else:
        _check_tensor("expert_ids", expert_ids, dev)
        if expert_weight is None:
            raise ValueError("expert_ids need expert_weight")
        _check_tensor("expert_weight", expert_weight, dev)
        if expert_ids.dtype != torch.int32 or expert_weight.dtype != torch.float32:
            raise TypeError("expert_ids must be int32 and expert_weight float32")
        if expert_ids.dim() != 2 or expert_ids.shape[0] != T or expert_weight.shape != expert_ids.shape:
            raise ValueError(f"expert_ids {tuple(expert_ids.shape)} and expert_weight {tuple(expert_weight.shape)} "
                             f"must both be [{T}, k]")
        if top_k is not None and top_k != expert_ids.shape[1]:
            raise ValueError(f"top_k is {top_k}, expert_ids have {expert_ids.shape[1]}")
        top_k = expert_ids.shape[1]
    if out is None:
        out = torch.empty_like(x)
    else:
        _check_tensor("out", out, dev)
        if out.dtype != x.dtype or out.shape != x.shape:
            raise ValueError(f"out must be {x.dtype} {tuple(x.shape)}, got {out.dtype} {tuple(out.shape)}")
    lib = _lib.load()
    if workspace is None:
        workspace = torch.empty((lib.mrr_few_tokens_workspace_size(T, top_k, inner),), dtype=torch.uint8, device=dev)
    else:
        _check_tensor("workspace", workspace, dev)
    # an empty tensor has no address: a call without tokens passes no routing
    args = _lib.MrrFewTokensArgs(x.data_ptr(), _WIDE[x.dtype], T, H, E, inner, int(top_k), _ptr(router_logits),
                                 int(renormalize), _ptr(expert_ids), _ptr(expert_weight), weights, gate_up.data_ptr(),
                                 _ptr(gate_up_scales), down.data_ptr(), _ptr(down_scales), out.data_ptr())
    _call(lib.mrr_few_tokens, "mrr_few_tokens", dev, ctypes.byref(args), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return out
