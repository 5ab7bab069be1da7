"""The norm's gradient over its range: values, weights and gradients of any size
whose products of gradient and weight lie between 2^-70 and 2^100, and rows
without a gradient or without values."""
import layer_reference as ref
import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import _dev

pytestmark = pytest.mark.gpu

BF16, F16, FP32 = torch.bfloat16, torch.float16, torch.float32


def check(up, x, w, eps, more=None):
    dev = _dev()
    there = [None if t is None else t.to(dev) for t in (up, x, w, more)]
    d, dw = moe.rms_norm_backward(*there[:3], grad_residual=there[3], eps=eps)
    want, want_w = ref.norm_backward(up, x, w, eps, more)
    r = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + eps)
    gw, n = up.double() * w.double(), x.double() * r
    size = r * (gw.abs() + n.abs() * (gw * n).abs().mean(-1, keepdim=True)) + (0 if more is None else more.double().abs())
    info = torch.finfo(x.dtype)
    # a rounding to the type, 2^-17 of the terms (128 roundings of 2^-24) as in the other tests, and where numbers lie
    # below 2^-126 roundings by half of 2^-149: of the mean (twice) and so of n by it, and of g w - n mean, which the root
    # multiplies then; and of the result
    most = want.abs() * info.eps / 2 + size * 2.0 ** -17 + info.tiny * info.eps
    most = most + r.clamp(min=1) * (n.abs() + 2) * 2.0 ** -149
    got = d.double().cpu()
    # a row with a term beyond the type's range may become infinite, or none
    inside = ((r * gw.abs()).amax(-1, keepdim=True) * 2 < info.max) & (size * 2 < info.max)
    assert ((got - want).abs() <= most)[inside].all(), float(((got - want).abs() / most)[inside].max())
    size_w = (up.double() * n).abs().sum(0)
    info = torch.finfo(w.dtype)  # its smallest step, 2^-133 of bf16, among them
    most_w = want_w.abs() * info.eps / 2 + size_w * 2.0 ** -17 + 2.0 ** -140 + info.tiny * info.eps
    inside = size_w * 2 < info.max
    assert ((dw.double().cpu() - want_w).abs() <= most_w)[inside].all()


@pytest.mark.parametrize("eps", [1e-6, 1e-30])
@pytest.mark.parametrize("product", [2.0 ** -62, 1e-9, 1.0, 1e10, 1e20, 2.0 ** 96])
@pytest.mark.parametrize("ws", [1e-20, 1e-8, 1.0, 1e8, 1e20])
@pytest.mark.parametrize("T,H", [(3, 64), (2, 3000), (300, 5), (2, 7168), (2, 9001)])
def test_gradients_and_weights_of_any_size(T, H, ws, product, eps):
    gs = product / ws
    g = torch.Generator().manual_seed(H)
    for dtype in (FP32, BF16):
        for xs in (1e-30, 1e-20, 1e-12, 1.0, 1e10, 1e19, 1e30):
            x, w, up = (torch.randn(*s, generator=g).double() for s in ((T, H), (H,), (T, H)))
            w = 1 + 0.3 * w.clamp(-2, 2)
            up = up.sign() * up.abs().clamp(2.0 ** -7, 4)  # with the weights from 2^-70 to 2^100
            check((up * gs).to(dtype), (x * xs).to(dtype), (w * ws).to(dtype), eps)


@pytest.mark.parametrize("eps", [1e-38 * 1.2, 1e-6, 1e4, 1e30])
@pytest.mark.parametrize("dtype", [FP32, BF16, F16])
@pytest.mark.parametrize("T,H", [(4, 64), (3, 3000), (300, 700), (2, 16384)])
def test_rows_without_a_gradient(T, H, dtype, eps):
    """Rows of a padded batch: no gradient, or no values, or neither; the others as without them."""
    dev = _dev()
    g = torch.Generator().manual_seed(H)
    x, up, more = (torch.randn(T, H, generator=g).to(dtype) for _ in range(3))
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(dtype)
    up[0], x[1] = 0, 0
    up[T - 1] = -0.0
    check(up, x, w, eps, more)
    d, _ = moe.rms_norm_backward(up.to(dev), x.to(dev), w.to(dev), eps=eps)
    assert (d[0] == 0).all() and (d[T - 1] == 0).all()
    x[T - 1] = 0
    check(up, x, w, eps)
