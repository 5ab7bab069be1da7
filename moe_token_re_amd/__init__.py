"""MoE re-routing (MoeReRoutingV2) for MI355X: hand-written HIP kernels behind a C ABI.

`moe_re_routing` is the Python entry point (`moe_re_routing_inverse` runs the
moves backwards). Beside it stand the experts' operators: `mx_quantize` and
`mx_dequantize` (microscaled 4-bit rows), `mx_grouped_mm` (the experts' product
over re-routed rows) and `moe_few_tokens` (a whole layer for a few tokens). The
in-tree HIP library is loaded on first use, and a missing build raises an
error: there is no CPU fallback.
"""

_API = ("moe_re_routing", "moe_re_routing_inverse", "workspace_size", "get_device_status", "MrrError")
_EXPERTS = ("mx_quantize", "mx_dequantize", "mx_grouped_mm", "moe_few_tokens", "few_tokens_workspace_size")


def __getattr__(name):
    if name in _API:
        from . import api

        return getattr(api, name)
    if name in _EXPERTS:
        from . import experts

        value = globals()[name] = getattr(experts, name)
        return value
    raise AttributeError(name)
