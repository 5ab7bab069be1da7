"""A mixture-of-experts layer of 4-bit experts, the ways a server runs it.

A layer on one device: rms_norm adds the residual and makes 4-bit rows,
moe_router_top_k chooses experts, moe_token_permute sorts the tokens by them,
mx_grouped_mm multiplies, and moe_token_unpermute sums the rows back by token.

A batch: the rows that the all-to-all brought (ordered by source rank, then by
expert) are microscaled 4-bit rows; moe_re_routing makes them expert-major,
mx_grouped_mm multiplies them with the experts (gate and up, then down with the
top-k weights, mx_quantize in between), and moe_re_routing_inverse puts them
back in the order in which they came.

A decode step: moe_few_tokens takes a few tokens and the router's logits through
the whole layer.

    python examples/expert_layer.py [--rows 4096] [--hidden 2048] [--inner 1024] [--experts 16] [--ranks 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_token_re_amd as moe  # noqa: E402


def batch(rows, scales, counts, topk_weight, w):
    """One batch of re-routed rows: rows [A, H/2] as they arrived, back in that order as bfloat16."""
    tokens, token_scales, _, expert_num, weight = moe.moe_re_routing(
        rows, counts, per_token_scales=scales, expert_topk_weight=topk_weight)
    h = moe.mx_grouped_mm(tokens, token_scales, w["gate_up"], w["gate_up_scales"], expert_num, gated=True)
    h, h_scales = moe.mx_quantize(h)
    y = moe.mx_grouped_mm(h, h_scales, w["down"], w["down_scales"], expert_num, row_weight=weight)
    return moe.moe_re_routing_inverse(y, counts)[0]


def layer(x, residual, norm_weight, router, top_k, w):
    """One layer's output for x [T, H] bfloat16, and the residual stream behind it."""
    rows, scales, residual = moe.rms_norm(x, norm_weight, residual=residual, quantize="mxfp4")
    logits = moe.mx_dequantize(rows, scales) @ router
    weight, ids = moe.moe_router_top_k(logits, top_k)
    tokens, token_scales, index, expert_num, _ = moe.moe_token_permute(rows, ids, router.shape[1], per_token_scales=scales)
    h = moe.mx_grouped_mm(tokens, token_scales, w["gate_up"], w["gate_up_scales"], expert_num, gated=True)
    y = moe.mx_grouped_mm(*moe.mx_quantize(h), w["down"], w["down_scales"], expert_num)
    return moe.moe_token_unpermute(y, index, expert_weight=weight), residual, (rows, scales, weight, ids)


def plain(x, w, expert, weight):
    """The layer in plain operations, row by row's expert, from the 4-bit weights' values."""
    y = torch.zeros_like(x)
    for e in range(w["down"].shape[0]):
        at = (expert == e).nonzero()[:, 0]
        up = moe.mx_dequantize(w["gate_up"][e], w["gate_up_scales"][e], dtype=torch.float32)
        down = moe.mx_dequantize(w["down"][e], w["down_scales"][e], dtype=torch.float32)
        gate, up = (x[at] @ up.t()).chunk(2, dim=1)
        y[at] = (torch.nn.functional.silu(gate) * up) @ down.t() * weight[at, None]
    return y


def relative(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def main():
    p = argparse.ArgumentParser()
    for name, default in (("rows", 4096), ("hidden", 2048), ("inner", 1024), ("experts", 16), ("ranks", 8)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(0)

    def weights(*shape):
        v = torch.empty(shape, device=dev).normal_(0, shape[-1] ** -0.5, generator=g).to(torch.bfloat16)
        return moe.mx_quantize(v)

    w = {}
    w["gate_up"], w["gate_up_scales"] = weights(a.experts, 2 * a.inner, a.hidden)
    w["down"], w["down_scales"] = weights(a.experts, a.hidden, a.inner)

    # a layer on one device
    x, residual = (torch.empty(a.rows, a.hidden, device=dev).normal_(generator=g).to(torch.bfloat16) for _ in range(2))
    router = torch.empty(a.hidden, a.experts, device=dev).normal_(0, a.hidden ** -0.5, generator=g).to(torch.bfloat16)
    top_k = min(2, a.experts)
    y, _, (rows, scales, weight, ids) = layer(x, residual, torch.ones(a.hidden, device=dev), router, top_k, w)
    rows = moe.mx_dequantize(rows, scales, dtype=torch.float32)
    want = sum(plain(rows, w, ids[:, j], weight[:, j]) for j in range(top_k))
    print(f"layer of {a.rows} tokens: {relative(y, want):.3f} off the plain layer (its inner rows are 4-bit values)")

    # a batch: every row has come for one expert from one rank
    cell = torch.randint(a.ranks * a.experts, (a.rows,), device=dev, generator=g).sort()[0]
    counts = torch.bincount(cell, minlength=a.ranks * a.experts).reshape(a.ranks, a.experts).to(torch.int32)
    x = torch.empty(a.rows, a.hidden, device=dev).normal_(generator=g).to(torch.bfloat16)
    topk_weight = torch.rand(a.rows, 1, device=dev, generator=g)
    rows, scales = moe.mx_quantize(x)
    y = batch(rows, scales, counts, topk_weight, w)
    want = plain(moe.mx_dequantize(rows, scales, dtype=torch.float32), w, cell % a.experts, topk_weight[:, 0])
    print(f"batch of {a.rows} rows: {relative(y, want):.3f} off the plain layer (its inner rows are 4-bit values)")

    # a decode step: eight tokens, two experts each
    x = x[:8].contiguous()
    logits = torch.randn(8, a.experts, device=dev, generator=g)
    y = moe.moe_few_tokens(x, w["gate_up"], w["down"], router_logits=logits, top_k=2,
                           gate_up_scales=w["gate_up_scales"], down_scales=w["down_scales"])
    top, ids = logits.topk(2, dim=1)
    share = torch.softmax(top, dim=1)
    want = sum(plain(x.float(), w, ids[:, j], share[:, j]) for j in range(2))
    print(f"decode step of 8 tokens: {relative(y, want):.4f} off the plain layer")


if __name__ == "__main__":
    main()
