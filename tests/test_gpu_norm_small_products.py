"""Rows whose products with the weight are nothing in 32 bits, and whose norm is
not: the scale of an 8-bit row is that of the exact largest value, and 0 for a
row of zeros alone."""
import layer_reference as ref
import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import _dev

pytestmark = pytest.mark.gpu

BF16, F16, FP32 = torch.bfloat16, torch.float16, torch.float32


# sizes of the values, the weights and eps: products of 1e-46 to 1e-62, values of the norm of 1e-30 to 1e-38
@pytest.mark.parametrize("size,by,eps", [(1e-15, 1e-31, 1.2e-38), (1e-20, 1e-30, 1.2e-38), (1e-25, 1e-35, 1.2e-38),
                                         (1e-13, 1e-34, 1e-30), (1e-20, 1e-27, 1e-18)])
@pytest.mark.parametrize("T,H", [(3, 64), (3, 3000), (300, 700), (2, 16384)])
def test_products_below_32_bits(T, H, size, by, eps):
    dev = _dev()
    g = torch.Generator().manual_seed(H)
    for xt, wt in ((BF16, BF16), (BF16, FP32), (FP32, FP32)):
        x = (torch.randn(T, H, generator=g).double() * size).to(xt)
        w = ((1 + 0.3 * torch.randn(H, generator=g).double()) * by).to(wt)
        x[1] = 0
        want, p = ref.norm(x, w, eps)
        top = want.abs().amax(1)
        for q, most, rounder in (("int8", 127, torch.round), ("fp8", 448, ref.e4m3)):
            y, scales, _ = moe.rms_norm(x.to(dev), w.to(dev), eps=eps, quantize=q)
            # one rounding of a 32-bit number, subnormal ones among them
            assert ((scales.double().cpu() - top / most).abs() <= top / most * 2.0 ** -24 + 2.0 ** -149).all()
            assert scales[1] == 0 and (y[1].float() == 0).all()
            exact = most * p / p.abs().amax(1, keepdim=True).clamp(min=1e-300)
            lo, hi = rounder(exact * (1 - 2.0 ** -42)), rounder(exact * (1 + 2.0 ** -42))  # 64-bit numbers' errors
            got = y.double().cpu()
            assert ((got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi))).all()


@pytest.mark.parametrize("H", [64, 3000])
def test_zeros(H):
    """Rows of zeros of either sign, and weights of zeros."""
    dev = _dev()
    x = torch.zeros(4, H, device=dev)
    x[1] = -0.0
    x[2:] = torch.randn(2, H, generator=torch.Generator().manual_seed(H)).to(dev)
    for w in (torch.ones(H, device=dev), torch.zeros(H, device=dev)):
        for q in ("int8", "fp8"):
            y, scales, _ = moe.rms_norm(x, w, quantize=q)
            zero = (w == 0).all()
            assert (y[:2].float() == 0).all() and (scales[:2] == 0).all()
            assert bool((scales[2:] == 0).all()) == bool(zero) and bool((y[2:].float() == 0).all()) == bool(zero)
