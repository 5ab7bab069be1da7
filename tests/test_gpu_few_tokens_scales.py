"""The few-token layer's 4-bit weights with scale bytes from one end of their
range to the other, 2^-127 to 2^127: tokens (or weights of the choice) are scaled
inversely, so that every block matters in its result. Against 64 bits, within
the bounds that experts_reference.py derives."""
import numpy as np
import pytest
import torch

import experts_reference as ref
from gpu_helpers import _dev
from moe_token_re_amd import experts

pytestmark = pytest.mark.gpu

I = 64


def _codes(gen, *shape):
    return torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, generator=gen)


def _plain_scales(rows, n):
    return torch.full((1, rows, (n + 63) // 64, 2), 124, dtype=torch.uint8)


def _run(x, up, ups, down, downs, p, dev):
    """(y, want, bound) of T tokens of one expert."""
    ids = torch.zeros(x.shape[0], 1, dtype=torch.int32)
    y = experts.moe_few_tokens(x.to(dev), up.to(dev), down.to(dev), expert_ids=ids.to(dev), expert_weight=p.to(dev),
                               gate_up_scales=ups.to(dev), down_scales=downs.to(dev))
    want, bound = ref.few_tokens(x.double().numpy(), ref.unpack(up.numpy(), ups.numpy()),
                                 ref.unpack(down.numpy(), downs.numpy()), ids.numpy(), p.double().numpy(), torch.bfloat16)
    return y, want, bound


def _layer(T, H, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    return (x, _codes(gen, 1, 2 * I, H), _plain_scales(2 * I, H), _codes(gen, 1, H, I), _plain_scales(H, I),
            torch.ones(T, 1))


@pytest.mark.parametrize("scales", [(0,), (1,), (126,), (251,), (252,), (253,), (254,), (254, 0, 127, 253),
                                    (3, 254, 252, 20, 253)])
@pytest.mark.parametrize("T,H", [(3, 160), (9, 288), (20, 1056)])
def test_scales_of_the_first_product(T, H, scales):
    """The gate takes a row's first block, the up projection the others, whose
    scales differ and whose tokens' values are as much smaller or larger."""
    x, up, ups, down, downs, p = _layer(T, H, 900 + H + sum(scales))
    up[0, :I, 16:] = 0
    up[0, I:, :16] = 0
    for b in range(1, H // 32):
        s = scales[b % len(scales)]
        ups[0, I:, b // 2, b % 2] = s
        x[:, 32 * b:32 * b + 32] = (x[:, 32 * b:32 * b + 32].double() * 2.0 ** (124 - s)).to(torch.bfloat16)
    y, want, bound = _run(x, up, ups, down, downs, p, _dev())
    assert torch.isfinite(y).all()
    ref.assert_close(y, want, bound, f"{T} tokens, H {H}, scales {scales}")


@pytest.mark.parametrize("scale", [0, 1, 126, 251, 252, 253, 254])
@pytest.mark.parametrize("T,H", [(3, 64), (9, 96), (20, 4160)])
def test_scales_of_the_second_product(T, H, scale):
    """Every other row's second block has the scale, all other blocks plain ones."""
    x, up, ups, down, downs, p = _layer(T, H, 950 + H + scale)
    downs[0, ::2, 0, 1] = scale
    down[0, 0, 16:] = 0  # no value under the scale in this row
    p[:] = 2.0 ** min(max(124 - scale, -110), 100)
    y, want, bound = _run(x, up, ups, down, downs, p, _dev())
    assert torch.isfinite(y).all()
    ref.assert_close(y, want, bound, f"{T} tokens, H {H}, scale {scale}")


def test_large_scales_beside_a_nan():
    """A row with a NaN scale gives NaN, also where another block's scale is
    large, and the other rows what they give."""
    x, up, ups, down, downs, p = _layer(5, 96, 970)
    downs[0, :, 0, 1] = 254
    p[:] = 2.0 ** -110
    y, want, bound = _run(x, up, ups, down, downs, p, _dev())
    ref.assert_close(y, want, bound, "large scales")
    downs[0, 7, 0, 0] = 255
    bad, want, bound = _run(x, up, ups, down, downs, p, _dev())
    assert torch.isnan(bad[:, 7]).all()
    ref.assert_close(bad, want, bound, "beside a NaN")
    rest = [i for i in range(96) if i != 7]
    assert torch.equal(bad[:, rest], y[:, rest])


def test_large_scales_and_infinite_tokens():
    """An infinity in a token gives what the definition gives, in that token alone."""
    x, up, ups, down, downs, p = _layer(5, 96, 980)
    ups[0, :, 1, 0] = 254
    x[:, 64:] = (x[:, 64:].double() * 2.0 ** -130).to(torch.bfloat16)
    y, want, bound = _run(x, up, ups, down, downs, p, _dev())
    ref.assert_close(y, want, bound, "large scales")
    x[2, 3] = float("inf")
    bad = _run(x, up, ups, down, downs, p, _dev())[0]
    rest = [0, 1, 3, 4]
    assert not torch.isfinite(bad[2]).any() and torch.equal(bad[rest], y[rest])
