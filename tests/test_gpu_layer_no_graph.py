"""Inputs that require a gradient: refused while autograd records, by both
bindings, and taken in the forward and backward of torch.autograd.Functions,
which make a training step of the operators."""
import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import _dev
from moe_token_re_amd import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["native", "python"])
def binding(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(_lib, "_plain_calls", _lib._NoBinding)


def tensors(dev, T=12, H=64, E=4, k=2):
    g = torch.Generator().manual_seed(3)
    x, w, logits = torch.randn(T, H, generator=g), torch.randn(H, generator=g), torch.randn(T, E, generator=g)
    return x.to(dev), w.to(dev), logits.to(dev)


def test_refused_while_autograd_records(binding):
    dev = _dev()
    x, w, logits = tensors(dev)
    weight, ids = moe.moe_router_top_k(logits, 2)
    rows, _, index, _, _ = moe.moe_token_permute(x, ids, 4)
    lead = lambda t: t.detach().clone().requires_grad_()  # noqa: E731
    param = torch.nn.Parameter(w.clone())
    scales = torch.rand(12, device=dev)
    calls = [lambda: moe.rms_norm(lead(x), w), lambda: moe.rms_norm(x, param), lambda: moe.rms_norm(x, w, residual=lead(x)),
             lambda: moe.rms_norm(x, param, quantize="fp8"), lambda: moe.rms_norm(lead(x) * 2, w),
             lambda: moe.moe_router_top_k(lead(logits), 2), lambda: moe.moe_token_permute(lead(x), ids, 4),
             lambda: moe.moe_token_permute(x, ids, 4, expert_weight=lead(weight)),
             lambda: moe.moe_token_permute(x, ids, 4, per_token_scales=lead(scales)),
             lambda: moe.moe_token_unpermute(lead(rows), index),
             lambda: moe.moe_token_unpermute(rows, index, expert_weight=lead(weight))]
    for n, call in enumerate(calls):
        with pytest.raises(ValueError, match="records no gradient"):
            call()
            pytest.fail(f"call {n}")
        with torch.no_grad():
            out = call()
        assert not any(t is not None and t.requires_grad for t in (out if isinstance(out, tuple) else (out,))), n
    # the gradients take them: nothing reads a graph there
    assert not moe.rms_norm_backward(lead(x), lead(x), param)[1].requires_grad
    assert not moe.moe_router_top_k_backward(lead(weight), lead(logits), lead(weight), ids).requires_grad
    assert not moe.moe_token_unpermute_backward(lead(x), lead(rows), index, expert_weight=lead(weight))[1].requires_grad
    assert not moe.moe_token_permute_backward(lead(rows), index)[0].requires_grad


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        ctx.save_for_backward(x, w)
        return moe.rms_norm(x, w, eps=1e-5)[0]

    @staticmethod
    def backward(ctx, grad):
        return moe.rms_norm_backward(grad.contiguous(), *ctx.saved_tensors, eps=1e-5)


class Router(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k):
        weight, ids = moe.moe_router_top_k(logits, k)
        ctx.save_for_backward(logits, weight, ids)
        ctx.mark_non_differentiable(ids)
        return weight, ids

    @staticmethod
    def backward(ctx, grad, _):
        return moe.moe_router_top_k_backward(grad.contiguous(), *ctx.saved_tensors), None


class There(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ids, E):
        rows, _, index, num, _ = moe.moe_token_permute(x, ids, E)
        ctx.save_for_backward(index)
        ctx.mark_non_differentiable(index, num)
        return rows, index, num

    @staticmethod
    def backward(ctx, grad, *_):
        return moe.moe_token_permute_backward(grad.contiguous(), *ctx.saved_tensors)[0], None, None


class Back(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, index, weight):
        ctx.save_for_backward(rows, index, weight)
        return moe.moe_token_unpermute(rows, index, expert_weight=weight)

    @staticmethod
    def backward(ctx, grad):
        rows, index, weight = ctx.saved_tensors
        d, dw = moe.moe_token_unpermute_backward(grad.contiguous(), rows, index, expert_weight=weight)
        return d, None, dw


def test_in_the_functions_of_a_training_step(binding):
    """Norm, router, rows by expert, a factor an expert, and back: autograd's gradients through the Functions against
    those of the same step in 64 bits."""
    dev = _dev()
    E, k = 4, 2
    x, w, logits = (t.requires_grad_() for t in tensors(dev, E=E))
    factor = torch.tensor([1.0, -2.0, 0.5, 3.0], device=dev, requires_grad=True)
    n = Norm.apply(x, w)
    weight, ids = Router.apply(logits, k)
    rows, index, num = There.apply(n, ids, E)
    y = Back.apply(rows * factor.repeat_interleave(num.long())[:, None], index, weight)
    (y * y).sum().backward()

    leaves = [t.detach().double().cpu().requires_grad_() for t in (x, w, logits, factor)]
    x64, w64, logits64, factor64 = leaves
    n64 = x64 / torch.sqrt(x64.square().mean(1, keepdim=True) + 1e-5) * w64
    top, ids64 = torch.sort(logits64, dim=1, descending=True, stable=True)
    y64 = n64 * (torch.softmax(top[:, :k], 1) * factor64[ids64[:, :k]]).sum(1, keepdim=True)
    (y64 * y64).sum().backward()
    assert torch.equal(ids.cpu().long(), ids64[:, :k])
    # sums of at most 64 x 12 terms of some ten roundings each, off by 2^-24 of terms of about the largest's size
    for got, want in zip((x, w, logits, factor), leaves):
        assert ((got.grad.double().cpu() - want.grad).abs() <= 2.0 ** -14 * want.grad.abs().max()).all()
