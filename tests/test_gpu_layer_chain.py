"""The operators around an expert layer as they are used together, with the
re-routing and the experts' operators: a whole layer of 4-bit experts for a
batch, the way over several ranks, a training step's gradients, and the calls
that are refused."""
import os
import sys
import zlib

import layer_reference as ref
import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import _dev

pytestmark = pytest.mark.gpu


def gen(*parts):
    return torch.Generator().manual_seed(zlib.crc32(repr(parts).encode()))


def mx_values(rows, scales):
    return moe.mx_dequantize(rows, scales, dtype=torch.float32).double().cpu()


@pytest.mark.parametrize("T,E,k", [(5, 4, 2), (300, 12, 3), (1500, 6, 4)])
def test_a_layer_of_4_bit_experts(T, E, k):
    """Norm to 4-bit rows, router, rows by expert, products, back by token; from the 4-bit values on against the
    definition in 64 bits. h is read back after its own quantisation, so that only the products' 32-bit sums and
    one rounding to bf16 lie between."""
    dev = _dev()
    g = gen("layer", T, E, k)
    H, inner = 256, 128
    x, r = (torch.randn(T, H, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    up = moe.mx_quantize((torch.randn(E, 2 * inner, H, generator=g) / H ** 0.5).to(dev))
    down = moe.mx_quantize((torch.randn(E, H, inner, generator=g) / inner ** 0.5).to(dev))
    logits = torch.randn(T, E, generator=g).to(dev)
    rows, scales, s = moe.rms_norm(x, torch.ones(H, device=dev), residual=r, quantize="mxfp4")
    weight, ids = moe.moe_router_top_k(logits, k)
    tokens, token_scales, index, num, row_weight = moe.moe_token_permute(rows, ids, E, per_token_scales=scales,
                                                                         expert_weight=weight)
    h = moe.mx_quantize(moe.mx_grouped_mm(tokens, token_scales, *up, num, gated=True, check=True))
    y = moe.mx_grouped_mm(*h, *down, num, row_weight=row_weight, check=True)
    out = moe.moe_token_unpermute(y, index)
    also = moe.moe_token_unpermute(moe.mx_grouped_mm(*h, *down, num), index, expert_weight=weight)

    assert torch.equal(s, ref.norm_sum(x, r))
    want_weight, want_ids = ref.router(logits.cpu(), k, True)
    assert torch.equal(ids.cpu(), want_ids)
    v, hv, dv = mx_values(rows, scales), mx_values(*h), mx_values(*down)
    assert torch.equal(mx_values(tokens, token_scales), ref.place(v, index.cpu()))
    want = torch.zeros(T, H, dtype=torch.float64)
    size = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            row = hv[int(index[t, j])]
            want[t] += want_weight[t, j] * (dv[e] @ row)
            size[t] += want_weight[t, j] * (dv[e].abs() @ row.abs())
    # each expert's row rounded to bf16 (half a step is 2^-8 of it at most), the sum once more, and 32-bit sums
    most = 2 ** -7 * size * 1.01
    for got in (out, also):
        assert ((got.double().cpu() - want).abs() <= most).all()


@pytest.mark.parametrize("ranks,local,k", [(2, 3, 2), (4, 4, 5)])
def test_over_ranks(ranks, local, k):
    """Every rank sorts its tokens by the experts of all, the all-to-all moves the rows (here by slices), each
    rank re-routes what it received, and everything goes back the same way: each expert adds its number."""
    dev = _dev()
    g = gen("ranks", ranks, local, k)
    H, E = 96, ranks * local
    sent = []
    for rank in range(ranks):
        x = torch.randint(-20, 20, (50 + 13 * rank, H), generator=g).to(torch.bfloat16).to(dev)
        weight, ids = moe.moe_router_top_k(torch.randn(x.shape[0], E, generator=g).to(dev), k)
        rows, _, index, num, row_weight = moe.moe_token_permute(x, ids, E, expert_weight=weight)
        sent.append((x, weight, ids, rows, index, num.view(ranks, local), row_weight))
    back = [[None] * ranks for _ in range(ranks)]
    for rank in range(ranks):
        # what arrives here, ordered by source rank, then by local expert
        counts = torch.stack([s[5][rank] for s in sent])
        parts, weights = [], []
        for s in sent:
            at = int(s[5][:rank].sum())
            parts.append(s[3][at:at + int(s[5][rank].sum())])
            weights.append(s[6][at:at + int(s[5][rank].sum())])
        rows, _, _, etn, w = moe.moe_re_routing(torch.cat(parts), counts, expert_topk_weight=torch.cat(weights), check=True)
        expert = rank * local + torch.repeat_interleave(torch.arange(local, device=dev), etn.long())
        y = (rows.float() + expert[:, None]).to(torch.bfloat16)
        y, *_ = moe.moe_re_routing_inverse(y, counts, check=True)
        for source, part in enumerate(y.split([int(c) for c in counts.sum(1)])):
            back[source][rank] = part
    for rank, (x, weight, ids, _, index, _, _) in enumerate(sent):
        y = moe.moe_token_unpermute(torch.cat(back[rank]), index, expert_weight=weight)
        want = (weight.double()[..., None] * (x.double()[:, None] + ids.double()[..., None])).sum(1)
        size = (weight.double()[..., None] * (x.double()[:, None] + ids.double()[..., None]).abs()).sum(1)
        # one rounding to bf16, of 8 significant bits: half a step is 2^(e - 8) of a value from 2^e on, 2^-8 of it;
        # and 32-bit products and sums, 2 k roundings of 2^-24 of the terms
        assert ((y.double() - want).abs() <= want.abs() * 2 ** -8 + size * 2 ** -20 + 1e-30).all()


@pytest.mark.parametrize("renormalize", [True, False])
def test_gradients_of_a_training_step(renormalize):
    """Residual and norm, router, rows by expert, experts (plain products here), back by token, in fp32: the
    functions' gradients against autograd's of the same layer in 64 bits."""
    dev = _dev()
    g = gen("step", renormalize)
    T, H, E, k = 70, 64, 5, 2
    x, r = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)
    w, router = torch.randn(H, generator=g), torch.randn(E, H, generator=g) / 8
    experts, up = torch.randn(E, H, H, generator=g) / 8, torch.randn(T, H, generator=g)

    # the layer in 64 bits by elementary operations
    leaves = [t.double().requires_grad_() for t in (x, r, w, router, experts)]
    x64, r64, w64, router64, experts64 = leaves
    s64 = x64 + r64
    n64 = s64 / torch.sqrt(s64.square().mean(1, keepdim=True) + 1e-5) * w64
    logits64 = n64 @ router64.t()
    top, ids64 = torch.sort(logits64, dim=1, descending=True, stable=True)
    p = torch.softmax(top[:, :k], 1) if renormalize else torch.softmax(top, 1)[:, :k]
    picked = experts64[ids64[:, :k]]
    y64 = s64 + (p[..., None] * (picked @ n64[:, None, :, None])[..., 0]).sum(1)
    (y64 * up.double()).sum().backward()

    x, r, w, router, experts, up = (t.to(dev) for t in (x, r, w, router, experts, up))
    n, _, s = moe.rms_norm(x, w, residual=r, eps=1e-5)
    logits = n @ router.t()
    weight, ids = moe.moe_router_top_k(logits, k, renormalize=renormalize)
    rows, _, index, num, _ = moe.moe_token_permute(n, ids, E)
    parts = list(zip(rows.split(num.tolist()), range(E)))
    out = torch.cat([part @ experts[e].t() for part, e in parts])
    y = s + moe.moe_token_unpermute(out, index, expert_weight=weight)

    d_out, d_weight = moe.moe_token_unpermute_backward(up, out, index, expert_weight=weight)
    d_rows = torch.cat([d @ experts[e] for d, e in zip(d_out.split(num.tolist()), range(E))])
    d_experts = torch.stack([d.t() @ part for d, (part, _) in zip(d_out.split(num.tolist()), parts)])
    d_n, _ = moe.moe_token_permute_backward(d_rows, index)
    d_logits = moe.moe_router_top_k_backward(d_weight, logits, weight, ids, renormalize=renormalize)
    d_n = d_n + d_logits @ router
    d_x, d_w = moe.rms_norm_backward(d_n.contiguous(), s, w, grad_residual=up, eps=1e-5)

    assert torch.equal(ids.cpu().long(), ids64[:, :k])
    # a dozen products and sums of at most 128 terms, each off by 2^-24 of terms of about the result's size:
    # 2^-14 of the largest result covers 1024 of them
    for got, want in ((y, y64), (d_x, x64.grad), (d_x, r64.grad), (d_w, w64.grad), (d_logits.t() @ n, router64.grad),
                      (d_experts, experts64.grad)):
        assert ((got.double().cpu() - want).abs() <= 2 ** -14 * want.abs().max()).all()


def test_refusals():
    dev = _dev()
    f = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device=dev)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    x, w, bf = f(4, 64), f(64), f(4, 64, dtype=torch.bfloat16)
    value = [
        lambda: moe.rms_norm(x.t(), f(4)), lambda: moe.rms_norm(x[:, ::2], f(32)), lambda: moe.rms_norm(x, f(63)),
        lambda: moe.rms_norm(x, f(1, 64)), lambda: moe.rms_norm(x, w, residual=f(3, 64)), lambda: moe.rms_norm(x, w, eps=0.0),
        lambda: moe.rms_norm(x, w, eps=-1.0), lambda: moe.rms_norm(x, w, eps=float("nan")), lambda: moe.rms_norm(x, w, quantize="int4"),
        lambda: moe.rms_norm(f(4, 63), f(63), quantize="mxfp4"), lambda: moe.rms_norm(f(4, 0), f(0)), lambda: moe.rms_norm(f(1), f(64)),
        lambda: moe.rms_norm(f(2, 16385), f(16385)), lambda: moe.rms_norm(x, w, out=(x, None, None)),
        lambda: moe.rms_norm(x, w, out=(f(4, 64), f(4), None)), lambda: moe.rms_norm(x, w, out=f(4, 64)),
        lambda: moe.rms_norm(x, w, residual=x.clone().cpu()), lambda: moe.rms_norm(f(), w),
        lambda: moe.rms_norm_backward(f(4, 63), x, w), lambda: moe.rms_norm_backward(x, f(4, 64).t(), f(4)),
        lambda: moe.rms_norm_backward(x, x.clone(), w, grad_residual=f(64)),
        lambda: moe.rms_norm_backward(x, x.clone(), w, workspace=f(4)),
        lambda: moe.rms_norm_backward(x, x.clone(), w, out=(x, f(64))),
        lambda: moe.moe_router_top_k(f(4), 1), lambda: moe.moe_router_top_k(x, 0), lambda: moe.moe_router_top_k(x, 17),
        lambda: moe.moe_router_top_k(f(4, 3), 4), lambda: moe.moe_router_top_k(f(4, 1025), 4),
        lambda: moe.moe_router_top_k(f(0, 3), 4), lambda: moe.moe_router_top_k(x, 2, out=(f(4, 2), i(4, 3))),
        lambda: moe.moe_router_top_k_backward(f(4, 2), x, f(4, 2), i(4, 3)),
        lambda: moe.moe_router_top_k_backward(f(4, 2), x, f(3, 2), i(4, 2)),
        lambda: moe.moe_router_top_k_backward(f(4, 2), x, f(4, 2), i(4)),
        lambda: moe.moe_token_permute(f(64), i(4, 2), 8), lambda: moe.moe_token_permute(x, i(3, 2), 8),
        lambda: moe.moe_token_permute(x, i(4), 8), lambda: moe.moe_token_permute(x, i(4, 17), 8), lambda: moe.moe_token_permute(x, i(4, 0), 8),
        lambda: moe.moe_token_permute(x, i(4, 2), 0), lambda: moe.moe_token_permute(x, i(4, 2), 4097),
        lambda: moe.moe_token_permute(f(4, 0), i(4, 2), 8), lambda: moe.moe_token_permute(x, i(4, 2), 8, per_token_scales=f(3)),
        lambda: moe.moe_token_permute(x, i(4, 2), 8, per_token_scales=f(4, 0)),
        lambda: moe.moe_token_permute(x, i(4, 2), 8, per_token_scales=f(4, 2, 2)),
        lambda: moe.moe_token_permute(x, i(4, 2), 8, per_token_scales=f(4, 2, 2, dtype=torch.uint8)),
        lambda: moe.moe_token_permute(x, i(4, 2), 8, expert_weight=f(4, 3)),
        lambda: moe.moe_token_permute(x, i(4, 2), 8, expert_token_num_type=2),
        lambda: moe.moe_token_permute(x, i(4, 2), 8, out=(f(8, 64), None, i(4, 2), i(8), f(8, 1))),
        lambda: moe.moe_token_permute(x, i(4, 2), 8, out=(f(7, 64), None, i(4, 2), i(8), None)),
        lambda: moe.moe_token_unpermute(f(8, 64), i(8)), lambda: moe.moe_token_unpermute(f(64), i(4, 2)),
        lambda: moe.moe_token_unpermute(f(8, 64), i(4, 17)), lambda: moe.moe_token_unpermute(f(8, 64), i(4, 2), expert_weight=f(4, 1)),
        lambda: moe.moe_token_unpermute(f(8, 64).t(), i(4, 2)), lambda: moe.moe_token_unpermute(f(8, 64), i(4, 2), out=f(3, 64)),
        lambda: moe.moe_token_unpermute_backward(f(3, 64), f(8, 64), i(4, 2)),
        lambda: moe.moe_token_unpermute_backward(x, f(8, 64), i(4, 2), expert_weight=f(4, 3)),
        lambda: moe.moe_token_permute_backward(f(8, 64), i(4, 2), grad_topk_weight=f(7, 1)),
    ]
    kind = [
        lambda: moe.rms_norm(x.double(), w.double()), lambda: moe.rms_norm(bf, w.half()), lambda: moe.rms_norm(x, w.bfloat16()),
        lambda: moe.rms_norm(x, w, residual=f(4, 64), out=(f(4, 64), None, None)), lambda: moe.rms_norm(x, w, residual=bf), lambda: moe.rms_norm(x, w, out=(bf, None, None)),
        lambda: moe.rms_norm_backward(bf, x, w), lambda: moe.moe_router_top_k(i(4, 4), 1),
        lambda: moe.moe_router_top_k_backward(f(4, 2), x, f(4, 2), f(4, 2)),
        lambda: moe.moe_token_permute(x, i(4, 2).long(), 8), lambda: moe.moe_token_permute(x.double(), i(4, 2), 8),
        lambda: moe.moe_token_permute(f(4, 64, dtype=torch.uint8), i(4, 2), 8),
        lambda: moe.moe_token_permute(x, i(4, 2), 8, tokens_dtype="int8"),
        lambda: moe.moe_token_permute(x, i(4, 2), 8, per_token_scales=f(4).half()),
        lambda: moe.moe_token_permute(x, i(4, 2), 8, expert_weight=f(4, 2).half()),
        lambda: moe.moe_token_unpermute(f(8, 64).to(torch.int8), i(4, 2)), lambda: moe.moe_token_unpermute(f(8, 64), f(4, 2)),
        lambda: moe.moe_token_unpermute(f(8, 64), i(4, 2), expert_weight=f(4, 2).bfloat16()),
        lambda: moe.moe_token_unpermute_backward(bf, f(8, 64), i(4, 2)),
    ]
    for n, call in enumerate(value):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"value {n}")
    for n, call in enumerate(kind):
        with pytest.raises(TypeError):
            call()
            pytest.fail(f"type {n}")
    torch.cuda.synchronize()


@pytest.mark.parametrize("sizes", [[], ["--rows", "37", "--experts", "3", "--hidden", "64", "--inner", "32"]])
def test_the_example_runs(sizes, monkeypatch, capsys):
    _dev()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    monkeypatch.syspath_prepend(os.path.join(root, "examples"))
    monkeypatch.setattr(sys, "argv", ["expert_layer.py", *sizes])
    import expert_layer

    expert_layer.main()
    assert capsys.readouterr().out.count("off the plain layer") == 3
