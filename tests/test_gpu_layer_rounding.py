"""The norm's 8-bit rows of 32-bit values against exact fractions: what lies
halfway between two of them is rounded to the even one."""
import random
from fractions import Fraction

import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import _dev

pytestmark = pytest.mark.gpu


def exact(x, w):
    """127 p / max |p| of every row, rounded to even, in fractions."""
    x, w = x.tolist(), [Fraction(v) for v in w.tolist()]
    out = []
    for row in x:
        p = [Fraction(v) * u for v, u in zip(row, w)]
        top = max(map(abs, p))
        out.append([round(127 * v / top) for v in p])
    return torch.tensor(out)


@pytest.mark.parametrize("few", [True, False])
def test_halves_of_the_largest_value(few):
    """Where the largest product is a row's only one of its size, its half is 63.5 and becomes 64."""
    dev = _dev()
    rng = random.Random(11)
    T, H = (200, 40) if few else (300, 600)
    x = torch.zeros(T, H)
    # a column of weights 2^-3 to 2^3 times one that fills 24 bits, another one in every call
    for call in range(4):
        base = 1 + rng.randrange(1, 1 << 23) / 2 ** 23
        w = torch.tensor([base * 2.0 ** rng.randrange(-3, 4) for _ in range(H)])
        for t in range(T):
            s = 1 + rng.randrange(1, 1 << 23) / 2 ** 23
            for n, c in enumerate(rng.sample(range(H), 8)):
                x[t, c] = (-1) ** n * s * 2.0 ** -n * base / float(w[c])
        q, _, _ = moe.rms_norm(x.to(dev), w.to(dev), quantize="int8")
        want = exact(x, w)
        assert (want == -64).any() and torch.equal(q.cpu().long(), want)
        x.zero_()


def test_every_border_between_two_values():
    """Rows of (k + 0.5) u under a largest of 127 u, for numbers u and weights that fill their bits."""
    dev = _dev()
    rng = random.Random(12)
    k = torch.arange(-127, 127).double() + 0.5
    x = torch.stack([torch.cat([torch.tensor([127.0], dtype=torch.float64), k]) * rng.randrange(1 << 15, 1 << 16)
                     for _ in range(60)]).float()
    want = torch.cat([torch.tensor([127.0]), torch.round(k.float())]).expand(60, -1)
    for _ in range(5):
        w = torch.full((x.shape[1],), rng.randrange(1 << 23, 1 << 24) / 2 ** 23)
        q, _, _ = moe.rms_norm(x.to(dev), w.to(dev), quantize="int8")
        assert torch.equal(q.cpu().float(), want)


@pytest.mark.parametrize("H", [64, 1500])
def test_rows_of_any_values(H):
    dev = _dev()
    g = torch.Generator().manual_seed(H)
    x, w = torch.randn(30, H, generator=g), 1 + 0.3 * torch.randn(H, generator=g)
    q, _, _ = moe.rms_norm(x.to(dev), w.to(dev), quantize="int8")
    assert torch.equal(q.cpu().long(), exact(x, w))
