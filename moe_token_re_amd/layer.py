"""Python binding of the operators around an expert layer on MI355X: the norm
before it with the residual's addition and 8-bit or microscaled rows as output
(rms_norm), the router's choice of experts (moe_router_top_k), a rank's tokens
sorted by expert (moe_token_permute) and the experts' rows summed back by token
(moe_token_unpermute).

Argument marshalling only, as in experts.py: a plain call goes by the native
binding (csrc/mrr_torch.cpp), the code here makes every other call and raises
every error, and there is no CPU path. The results carry no autograd graph:
each operator's gradient is a function of its own (*_backward), which can be
called, and captured into a graph, like any other operator here, or stand in
the backward of a torch.autograd.Function. While autograd records, an operator
refuses inputs that require a gradient, which would be lost: it is called under
torch.no_grad(), or in the forward of such a Function, where nothing is recorded.
The gradients take any tensors, and what they return leads no further.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from .api import _FP4, _TAGGED, _TOKEN_DTYPES, _check_tensor, _ptr, _raise
from .experts import _WIDE, _call, _gpu

_SCALE_F32, _SCALE_MX = (torch.float32,), (torch.float8_e8m0fnu, torch.uint8)
# quantize -> (y's dtypes, its code, the scales' dtypes, their code)
_QUANTIZE = {
    "int8": ((torch.int8,), _lib.I8, _SCALE_F32, _lib.F32),
    "fp8": ((torch.float8_e4m3fn,), _lib.F8_E4M3FN, _SCALE_F32, _lib.F32),
    "mxfp8": ((torch.float8_e4m3fn,), _lib.F8_E4M3FN, _SCALE_MX, _lib.F8_E8M0),
    "mxfp4": ((torch.float4_e2m1fn_x2, torch.uint8), _lib.F4_E2M1, _SCALE_MX, _lib.F8_E8M0),
}
_MOVED = {**_TOKEN_DTYPES, torch.float32: _lib.F32}


def _wide(name, t, dev):
    _check_tensor(name, t, dev)
    if t.dtype not in _WIDE:
        raise TypeError(f"{name} must be float16, bfloat16 or float32, got {t.dtype}")


def _is(name, t, dev, dtypes, shape):
    """Checks one tensor's device, dtype and shape."""
    _check_tensor(name, t, dev)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _no_graph(where, *tensors):
    """Refuses to lose a gradient."""
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in tensors):
        raise ValueError(f"{where} records no gradient, and one of its inputs requires one: call it under torch.no_grad(), "
                         f"or in a torch.autograd.Function with {where}_backward as its backward")


def _outputs(out, dev, *want):
    """The outputs: new ones, or those of `out` checked. want: (name, dtypes, shape), or None for one that is absent."""
    if out is None:
        return tuple(None if w is None else torch.empty(w[2], dtype=w[1][0], device=dev) for w in want)
    if not isinstance(out, (tuple, list)) or len(out) != len(want):
        raise ValueError(f"out must be a tuple of {len(want)} like the result")
    for t, w in zip(out, want):
        if w is None:
            if t is not None:
                raise ValueError("out holds a tensor where the result has None")
        else:
            _is("out " + w[0], t, dev, w[1], w[2])
    return tuple(out)


def _workspace(workspace, need, dev, where):
    if workspace is None:
        if need == 0:
            _raise(_lib.ERROR_INVALID_SHAPE, where)
        return torch.empty((need,), dtype=torch.uint8, device=dev)
    _check_tensor("workspace", workspace, dev)
    return workspace


def _norm_weight(weight, x, dev):
    _is("weight", weight, dev, (x.dtype, torch.float32), x.shape[-1:])


def rms_norm(x: torch.Tensor, weight: torch.Tensor, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             quantize: Optional[str] = None, out=None):
    """Root-mean-square norm of rows x [..., H] (float16, bfloat16 or float32, H up
    to 16384) with weight [H] of x's dtype or float32: with s = x + residual,
    rounded to x's dtype (x itself without a residual), y = weight * s / sqrt(mean(s^2) + eps).

    Returns (y, scales, s). s is None without a residual. `quantize` says what y is:
      None     x's dtype; scales is None
      "int8", "fp8"  int8 or float8_e4m3fn rows, scales [...] float32: max |y| / 127
               or / 448 of a row; values y / scale rounded to nearest even. The scale
               of a row that is not finite is NaN.
      "mxfp8", "mxfp4"  microscaled float8_e4m3fn or float4_e2m1fn_x2 [..., H/2] rows,
               scales [..., ceil(H/64), 2] float8_e8m0fnu, as mx_quantize makes them.
    These are tokens and per_token_scales as moe_token_permute and moe_re_routing
    take them; "mxfp4" rows are mx_grouped_mm's. `out` is a tuple like the result.
    Up to 256 rows add their squares in another order than more do: the last place of a
    wide value, or of a scale, may differ between the same row in a small and a large batch."""
    if out is None:
        done = _lib.plain_calls().rms_norm(x, weight, residual, eps, quantize)
        if done is not None:
            return done
    _no_graph("rms_norm", x, weight, residual)
    dev = _gpu("x", x)
    _wide("x", x, dev)
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError(f"x must hold rows, got shape {tuple(x.shape)}")
    _norm_weight(weight, x, dev)
    *lead, H = x.shape
    if residual is not None:
        _is("residual", residual, dev, (x.dtype,), x.shape)
    scales = None
    if quantize is None:
        y, code, scale_code = ("y", (x.dtype,), x.shape), _WIDE[x.dtype], _lib.F32
    else:
        if quantize not in _QUANTIZE:
            raise ValueError(f"quantize must be None or one of {sorted(_QUANTIZE)}, got {quantize!r}")
        dtypes, code, scale_dtypes, scale_code = _QUANTIZE[quantize]
        if code == _lib.F4_E2M1 and H % 2:
            raise ValueError(f"mxfp4 rows hold an even number of values, got {H}")
        y = ("y", dtypes, (*lead, H // 2 if code == _lib.F4_E2M1 else H))
        scales = ("scales", scale_dtypes, lead if scale_code == _lib.F32 else (*lead, (H + 63) // 64, 2))
    total = None if residual is None else ("sum", (x.dtype,), x.shape)
    y, scales, total = out = _outputs(out, dev, y, scales, total)
    args = _lib.MrrRmsNormArgs(x.data_ptr(), _WIDE[x.dtype], x.numel() // H, H, _ptr(residual), weight.data_ptr(),
                               _WIDE[weight.dtype], float(eps), y.data_ptr(), code, _ptr(scales), scale_code,
                               _ptr(total))
    _call(_lib.load().mrr_rms_norm, "mrr_rms_norm", dev, ctypes.byref(args))
    return out


def rms_norm_backward_workspace_size(rows: int, H: int) -> int:
    """Bytes of workspace rms_norm_backward needs for rows of H values."""
    return int(_lib.load().mrr_rms_norm_backward_workspace_size(rows, H))


def rms_norm_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, *,
                      grad_residual: Optional[torch.Tensor] = None, eps: float = 1e-6, out=None,
                      workspace: Optional[torch.Tensor] = None):
    """The gradient of rms_norm with y of x's dtype. grad [..., H] is y's, x what was
    normalised: rms_norm's s where it added a residual. grad_residual is the gradient
    that reaches s by itself (from what reads the residual later), added to the result.

    Returns (grad_x, grad_weight) of x's and weight's dtypes: grad_x is the gradient of
    x and of the residual alike, grad_weight [H] is summed over all rows in float32. grad *
    weight is to lie between 2^-70 and 2^100, or be 0."""
    if out is None and workspace is None:
        done = _lib.plain_calls().rms_norm_backward(grad, x, weight, grad_residual, eps)
        if done is not None:
            return done
    dev = _gpu("grad", grad)
    _wide("x", x, dev)
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError(f"x must hold rows, got shape {tuple(x.shape)}")
    _is("grad", grad, dev, (x.dtype,), x.shape)
    _norm_weight(weight, x, dev)
    if grad_residual is not None:
        _is("grad_residual", grad_residual, dev, (x.dtype,), x.shape)
    H = x.shape[-1]
    rows = x.numel() // H
    grad_x, grad_weight = out = _outputs(out, dev, ("grad_x", (x.dtype,), x.shape),
                                         ("grad_weight", (weight.dtype,), weight.shape))
    lib = _lib.load()
    workspace = _workspace(workspace, lib.mrr_rms_norm_backward_workspace_size(rows, H), dev, "mrr_rms_norm_backward")
    args = _lib.MrrRmsNormBackwardArgs(grad.data_ptr(), x.data_ptr(), _WIDE[x.dtype], rows, H, weight.data_ptr(),
                                       _WIDE[weight.dtype], float(eps), _ptr(grad_residual), grad_x.data_ptr(),
                                       grad_weight.data_ptr())
    _call(lib.mrr_rms_norm_backward, "mrr_rms_norm_backward", dev, ctypes.byref(args), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return out


def _logits(t, dev):
    _wide("router_logits", t, dev)
    if t.dim() != 2:
        raise ValueError(f"router_logits must be [T, E], got shape {tuple(t.shape)}")
    return t.shape


def moe_router_top_k(router_logits: torch.Tensor, top_k: int, *, renormalize: bool = True, out=None):
    """The router's choice of experts, as moe_few_tokens makes it: of logits [T, E]
    (float16, bfloat16 or float32, E up to 1024) the top_k (at most 16) largest of each
    row, in falling order, ties to the lowest expert, weighted by the softmax over the
    chosen ones, or with renormalize=False over all experts.

    Returns (expert_weight [T, top_k] float32, expert_ids [T, top_k] int32). An expert of
    logit -inf is never chosen: where fewer than top_k are left the id is -1 and the
    weight 0. A NaN or +inf in a row makes its weights NaN."""
    if out is None:
        done = _lib.plain_calls().router(router_logits, top_k, renormalize)
        if done is not None:
            return done
    _no_graph("moe_router_top_k", router_logits)
    dev = _gpu("router_logits", router_logits)
    T, E = _logits(router_logits, dev)
    if not 1 <= top_k <= min(E, 16):  # without tokens the library gets no address to see it by
        _raise(_lib.ERROR_INVALID_SHAPE, "mrr_router")
    weight, ids = out = _outputs(out, dev, ("expert_weight", (torch.float32,), (T, top_k)),
                                 ("expert_ids", (torch.int32,), (T, top_k)))
    args = _lib.MrrRouterArgs(router_logits.data_ptr(), _WIDE[router_logits.dtype], T, E, int(top_k), int(renormalize),
                              weight.data_ptr(), ids.data_ptr())
    _call(_lib.load().mrr_router, "mrr_router", dev, ctypes.byref(args))
    return out


def moe_router_top_k_backward(grad_weight: torch.Tensor, router_logits: torch.Tensor, expert_weight: torch.Tensor,
                              expert_ids: torch.Tensor, *, renormalize: bool = True,
                              out: Optional[torch.Tensor] = None):
    """The gradient of moe_router_top_k: grad_weight [T, top_k] float32 is
    expert_weight's; router_logits are its input, expert_weight and expert_ids its
    results, renormalize as there. Returns grad_logits [T, E] of the logits' dtype."""
    if out is None:
        done = _lib.plain_calls().router_backward(grad_weight, router_logits, expert_weight, expert_ids, renormalize)
        if done is not None:
            return done
    dev = _gpu("grad_weight", grad_weight)
    T, E = _logits(router_logits, dev)
    if expert_ids.dim() != 2:
        raise ValueError(f"expert_ids must be [T, top_k], got shape {tuple(expert_ids.shape)}")
    shape = (T, expert_ids.shape[1])
    _is("expert_ids", expert_ids, dev, (torch.int32,), shape)
    _is("expert_weight", expert_weight, dev, (torch.float32,), shape)
    _is("grad_weight", grad_weight, dev, (torch.float32,), shape)
    (out,) = _outputs(None if out is None else (out,), dev,
                      ("grad_logits", (router_logits.dtype,), router_logits.shape))
    args = _lib.MrrRouterBackwardArgs(grad_weight.data_ptr(), router_logits.data_ptr(), _WIDE[router_logits.dtype], T, E,
                                      shape[1], int(renormalize), expert_weight.data_ptr(), expert_ids.data_ptr(),
                                      out.data_ptr())
    _call(_lib.load().mrr_router_backward, "mrr_router_backward", dev, ctypes.byref(args))
    return out


def token_permute_workspace_size(T: int, top_k: int, num_experts: int) -> int:
    """Bytes of workspace moe_token_permute needs for T tokens of top_k experts each."""
    return int(_lib.load().mrr_token_permute_workspace_size(T, top_k, num_experts))


def moe_token_permute(tokens: torch.Tensor, expert_ids: torch.Tensor, num_experts: int, *,
                      per_token_scales: Optional[torch.Tensor] = None, expert_weight: Optional[torch.Tensor] = None,
                      expert_token_num_type: int = 1, tokens_dtype: Optional[str] = None, out=None,
                      workspace: Optional[torch.Tensor] = None):
    """Sorts a rank's tokens by expert: a token's row is copied to one row for each of
    its experts, in the order of a stable sort of all choices (t, j) by expert.

    tokens [T, H] is of any dtype that moe_re_routing moves (uint8 with its tokens_dtype
    tag), or float32; expert_ids [T, top_k] int32 (top_k at most 16) number the experts
    [0, num_experts), of all ranks if the rows go through an all-to-all. per_token_scales
    [T], [T, S] float32 or [T, ceil(H/64), 2] float8_e8m0fnu and expert_weight [T, top_k]
    float32 move along.

    Returns, with A = T top_k, (permute_tokens [A, H], permute_per_token_scales [A, ...] or
    None, permute_token_idx [T, top_k] int32: the row of each choice, expert_token_num
    [num_experts] int32: rows of each expert, or with expert_token_num_type=0 their running
    sum, permute_topk_weight [A, 1] or None). Choices whose id is outside [0, num_experts)
    get the rows behind the experts' ones, filled with zeros, and the index -1 - row."""
    if out is None and workspace is None and tokens_dtype is None:
        done = _lib.plain_calls().permute(tokens, expert_ids, num_experts, per_token_scales, expert_weight,
                                          expert_token_num_type)
        if done is not None:
            return done
    _no_graph("moe_token_permute", tokens, per_token_scales, expert_weight)
    dev = _gpu("tokens", tokens)
    _check_tensor("tokens", tokens, dev)
    if tokens.dim() != 2:
        raise ValueError(f"tokens must be [T, H], got shape {tuple(tokens.shape)}")
    if tokens_dtype is not None:
        if tokens.dtype not in (torch.uint8, torch.int8) or tokens_dtype not in _TAGGED:
            raise TypeError(f"tokens_dtype={tokens_dtype!r} needs uint8 storage and one of {sorted(_TAGGED)}")
        code = _TAGGED[tokens_dtype]
    elif tokens.dtype in _MOVED:
        code = _MOVED[tokens.dtype]
    else:
        raise TypeError(f"unsupported tokens dtype {tokens.dtype}")
    T = tokens.shape[0]
    H = tokens.shape[1] * (2 if code in _FP4 else 1)
    _check_tensor("expert_ids", expert_ids, dev)
    if expert_ids.dtype != torch.int32:
        raise TypeError(f"expert_ids must be int32, got {expert_ids.dtype}")
    if expert_ids.dim() != 2 or expert_ids.shape[0] != T:
        raise ValueError(f"expert_ids has shape {tuple(expert_ids.shape)}, expected {(T, 'top_k')}")
    k = expert_ids.shape[1]
    a = _lib.MrrTokenPermuteArgs()
    if not 1 <= k <= 16 or not 1 <= num_experts <= 4096 or H == 0:
        _raise(_lib.ERROR_INVALID_SHAPE, "mrr_token_permute")
    A = T * k
    scales = weight = None
    if per_token_scales is not None:
        s = per_token_scales
        _check_tensor("per_token_scales", s, dev)
        if s.dtype not in _SCALE_F32 + _SCALE_MX:
            raise TypeError(f"unsupported per_token_scales dtype {s.dtype}")
        if not 1 <= s.dim() <= 3 or s.shape[0] != T:
            raise ValueError(f"per_token_scales has shape {tuple(s.shape)}, expected {T} rows")
        if s.dtype != torch.float32 and tuple(s.shape) != (T, (H + 63) // 64, 2):
            raise ValueError(f"per_token_scales has shape {tuple(s.shape)}, expected {(T, (H + 63) // 64, 2)}")
        if s.dtype == torch.float32 and (s.dim() > 2 or s.numel() == 0 < T):
            raise ValueError(f"per_token_scales has shape {tuple(s.shape)}, expected {(T,)} or {(T, 'S')}")
        a.scales_dtype = _lib.F32 if s.dtype == torch.float32 else _lib.F8_E8M0
        a.scales_ndim = s.dim()
        for i in range(s.dim()):
            a.scales_dims[i] = s.shape[i]
        scales = ("permute_per_token_scales", (s.dtype,), (A, *s.shape[1:]))
    if expert_weight is not None:
        _is("expert_weight", expert_weight, dev, (torch.float32,), expert_ids.shape)
        weight = ("permute_topk_weight", (torch.float32,), (A, 1))
    out = _outputs(out, dev, ("permute_tokens", (tokens.dtype,), (A, tokens.shape[1])), scales,
                   ("permute_token_idx", (torch.int32,), (T, k)),
                   ("expert_token_num", (torch.int32,), (num_experts,)), weight)
    lib = _lib.load()
    workspace = _workspace(workspace, lib.mrr_token_permute_workspace_size(T, k, num_experts), dev, "mrr_token_permute")
    a.tokens, a.tokens_dtype, a.T, a.H = tokens.data_ptr(), code, T, H
    a.expert_ids, a.top_k, a.E = expert_ids.data_ptr(), k, num_experts
    a.per_token_scales, a.expert_weight = _ptr(per_token_scales), _ptr(expert_weight)
    a.permute_tokens, a.permute_per_token_scales = out[0].data_ptr(), _ptr(out[1])
    a.permute_token_idx, a.expert_token_num, a.permute_topk_weight = out[2].data_ptr(), out[3].data_ptr(), _ptr(out[4])
    a.expert_token_num_type = int(expert_token_num_type)
    _call(lib.mrr_token_permute, "mrr_token_permute", dev, ctypes.byref(a), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return out


def _rows(name, t, dev):
    _wide(name, t, dev)
    if t.dim() != 2 or t.shape[1] == 0:
        raise ValueError(f"{name} must be [rows, H], got shape {tuple(t.shape)}")
    return t.shape


def _index(t, dev):
    _check_tensor("permute_token_idx", t, dev)
    if t.dtype != torch.int32:
        raise TypeError(f"permute_token_idx must be int32, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"permute_token_idx must be [T, top_k], got shape {tuple(t.shape)}")
    if not 1 <= t.shape[1] <= 16:
        _raise(_lib.ERROR_INVALID_SHAPE, "mrr_token_unpermute")
    return t.shape


def _unpermute(rows, idx, expert_weight, y, row_values, choice_values, dev):
    (R, H), (T, k) = rows.shape, idx.shape
    args = _lib.MrrTokenUnpermuteArgs(rows.data_ptr(), _WIDE[rows.dtype], R, H, idx.data_ptr(), T, k,
                                      _ptr(expert_weight), y.data_ptr(), _ptr(row_values), _ptr(choice_values))
    _call(_lib.load().mrr_token_unpermute, "mrr_token_unpermute", dev, ctypes.byref(args))


def moe_token_unpermute(rows: torch.Tensor, permute_token_idx: torch.Tensor, *,
                        expert_weight: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """The experts' rows summed back by token: y[t] = sum over j of
    expert_weight[t, j] * rows[permute_token_idx[t, j]], in float32 in the order of j and
    rounded once. rows [R, H] are float16, bfloat16 or float32, permute_token_idx
    [T, top_k] is moe_token_permute's, expert_weight [T, top_k] float32 (every weight 1
    without it). An index outside [0, R) adds nothing. Returns y [T, H] of rows' dtype."""
    if out is None:
        done = _lib.plain_calls().unpermute(rows, permute_token_idx, expert_weight)
        if done is not None:
            return done
    _no_graph("moe_token_unpermute", rows, expert_weight)
    dev = _gpu("rows", rows)
    _, H = _rows("rows", rows, dev)
    T, k = _index(permute_token_idx, dev)
    if expert_weight is not None:
        _is("expert_weight", expert_weight, dev, (torch.float32,), (T, k))
    (out,) = _outputs(None if out is None else (out,), dev, ("y", (rows.dtype,), (T, H)))
    _unpermute(rows, permute_token_idx, expert_weight, out, None, None, dev)
    return out


def moe_token_permute_backward(grad_rows: torch.Tensor, permute_token_idx: torch.Tensor, *,
                               grad_topk_weight: Optional[torch.Tensor] = None, out=None):
    """The gradient of moe_token_permute: grad_rows [A, H] is permute_tokens', and
    grad_topk_weight [A, 1] or [A] float32 permute_topk_weight's. Returns (grad_tokens
    [T, H]: the sum of a token's rows, grad_expert_weight [T, top_k] or None); choices
    that were not here have no part in either."""
    if out is None:
        done = _lib.plain_calls().permute_backward(grad_rows, permute_token_idx, grad_topk_weight)
        if done is not None:
            return done
    dev = _gpu("grad_rows", grad_rows)
    R, H = _rows("grad_rows", grad_rows, dev)
    T, k = _index(permute_token_idx, dev)
    if grad_topk_weight is not None:
        _is("grad_topk_weight", grad_topk_weight, dev, (torch.float32,),
            (R,) if grad_topk_weight.dim() == 1 else (R, 1))
    grad, weight = out = _outputs(out, dev, ("grad_tokens", (grad_rows.dtype,), (T, H)),
                                  None if grad_topk_weight is None else
                                  ("grad_expert_weight", (torch.float32,), (T, k)))
    _unpermute(grad_rows, permute_token_idx, None, grad, grad_topk_weight, weight, dev)
    return out


def moe_token_unpermute_backward(grad: torch.Tensor, rows: torch.Tensor, permute_token_idx: torch.Tensor, *,
                                 expert_weight: Optional[torch.Tensor] = None, out=None):
    """The gradients of moe_token_unpermute: grad [T, H] is y's; rows, permute_token_idx
    (as moe_token_permute returns it: no row twice) and expert_weight as there.

    Returns (grad_rows [R, H], grad_expert_weight [T, top_k] float32, None without
    expert_weight). The rows that moe_token_permute gave to choices that were not here get
    zeros; rows that no index names are left as they were (a new grad_rows holds anything
    there; moe_token_permute's indices name every row)."""
    if out is None:
        done = _lib.plain_calls().unpermute_backward(grad, rows, permute_token_idx, expert_weight)
        if done is not None:
            return done
    dev = _gpu("grad", grad)
    R, H = _rows("rows", rows, dev)
    T, k = _index(permute_token_idx, dev)
    _is("grad", grad, dev, (rows.dtype,), (T, H))
    if expert_weight is not None:
        _is("expert_weight", expert_weight, dev, (torch.float32,), (T, k))
    grad_rows, weight = out = _outputs(out, dev, ("grad_rows", (rows.dtype,), (R, H)),
                                       None if expert_weight is None else
                                       ("grad_expert_weight", (torch.float32,), (T, k)))
    args = _lib.MrrTokenUnpermuteBackwardArgs(grad.data_ptr(), rows.data_ptr(), _WIDE[rows.dtype], R, H,
                                              permute_token_idx.data_ptr(), T, k, _ptr(expert_weight),
                                              grad_rows.data_ptr(), _ptr(weight))
    _call(_lib.load().mrr_token_unpermute_backward, "mrr_token_unpermute_backward", dev, ctypes.byref(args))
    return out
