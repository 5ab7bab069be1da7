"""MoE re-routing (MoeReRoutingV2) for MI355X: hand-written HIP kernels behind a C ABI.

`moe_re_routing` is the Python entry point (`moe_re_routing_inverse` runs the
moves backwards). Beside it stand the experts' operators: `mx_quantize` and
`mx_dequantize` (microscaled 4-bit rows), `mx_grouped_mm` (the experts' product
over re-routed rows) and `moe_few_tokens` (a whole layer for a few tokens), and the
operators around a layer, with their gradients: `rms_norm` (with the residual's
addition and 8-bit rows as output), `moe_router_top_k`, `moe_token_permute` and
`moe_token_unpermute` (a rank's tokens sorted by expert, and back). The in-tree
HIP library is loaded on first use, and a missing build raises an error: there
is no CPU fallback.
"""

_API = ("moe_re_routing", "moe_re_routing_inverse", "workspace_size", "get_device_status", "MrrError")
_EXPERTS = ("mx_quantize", "mx_dequantize", "mx_grouped_mm", "moe_few_tokens", "few_tokens_workspace_size")
_LAYER = ("rms_norm", "rms_norm_backward", "rms_norm_backward_workspace_size", "moe_router_top_k",
          "moe_router_top_k_backward", "moe_token_permute", "moe_token_permute_backward",
          "token_permute_workspace_size", "moe_token_unpermute", "moe_token_unpermute_backward")


def __getattr__(name):
    if name in _API:
        from . import api

        return getattr(api, name)
    if name in _EXPERTS:
        from . import experts

        value = globals()[name] = getattr(experts, name)
        return value
    if name in _LAYER:
        from . import layer

        value = globals()[name] = getattr(layer, name)
        return value
    raise AttributeError(name)
