"""Rows that go past the caches against the same rows that do not, bit for bit.

What does, of rows that begin and end at multiples of 16 bytes: the norm's of 16 bits
from 24 MiB of them on, its gradient's of 16 bits from 64 MiB, the rows that are
written by expert and the sums and their gradients always, and the rows that are
read for these from 256 MiB. Rows of 32 bits of the norm never do. A tensor that
begins elsewhere has all of a call's rows go by way of the caches."""
import os
import re
import zlib

import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import _dev

pytestmark = pytest.mark.gpu

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")
BF16, F16, FP32 = torch.bfloat16, torch.float16, torch.float32


def threshold(source, name):
    found = re.search(rf"constexpr int64_t {name} = int64_t\((\d+)\) << 20;", open(os.path.join(CSRC, source)).read())
    return int(found[1]) << 20


def gen(dev, *parts):
    return torch.Generator(dev).manual_seed(zlib.crc32(repr(parts).encode()))


def same(a, b):
    return (a is None and b is None) or torch.equal(a.contiguous().view(-1).view(torch.uint8),
                                                    b.contiguous().view(-1).view(torch.uint8))


def odd(t):
    """The same values one element past an aligned address."""
    buf = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    buf[1:t.numel() + 1] = t.reshape(-1)
    got = buf[1:t.numel() + 1].view(t.shape)
    assert t.data_ptr() % 16 == 0 and got.data_ptr() % 16 != 0
    return got


def aligned(*tensors):
    return all(t is None or (t.data_ptr() % 16 == 0 and t.shape[-1] * t.element_size() % 16 == 0) for t in tensors)


@pytest.mark.parametrize("T,H,dtype,weight", [
    (4000, 4096, BF16, FP32), (2000, 7168, F16, F16), (30000, 512, BF16, BF16), (14000, 1000, F16, FP32),
    (900, 16384, BF16, BF16), (26000, 488, BF16, FP32)])
def test_norm(T, H, dtype, weight):
    dev = _dev()
    g = gen(dev, T, H)
    least, size = threshold("mrr_rms_norm.hip", "kStreamBytes"), T * H * 2
    x, r = (torch.randn(T, H, device=dev, generator=g).to(dtype) for _ in range(2))
    w = (1 + 0.3 * torch.randn(H, device=dev, generator=g)).to(weight)
    x[3] = 0
    assert aligned(x, r)
    assert size >= least  # the whole goes past the caches, and no piece does
    pieces = -(-3 * size // (2 * least))
    for quantize in (None, "int8", "fp8", "mxfp8", "mxfp4"):
        for residual in (r, None):
            out = moe.rms_norm(x, w, residual=residual, quantize=quantize)
            elsewhere = moe.rms_norm(odd(x), w, residual=residual, quantize=quantize)
            assert all(same(a, b) for a, b in zip(out, elsewhere)), quantize
            for a in range(0, T, -(-T // pieces)):
                b = min(T, a - (-T // pieces))
                assert (b - a) * H * 2 < least and b - a > 256  # up to 256 rows would lie on more lanes, with other sums
                part = moe.rms_norm(x[a:b], w, residual=None if residual is None else residual[a:b], quantize=quantize)
                assert all(p is None or same(o[a:b], p) for p, o in zip(part, out)), (quantize, a)


@pytest.mark.parametrize("T,H,dtype,weight", [
    (8400, 4096, BF16, FP32), (5000, 7168, F16, F16), (70000, 512, BF16, BF16), (2100, 16384, BF16, FP32)])
def test_norm_backward(T, H, dtype, weight):
    dev = _dev()
    g = gen(dev, T, H)
    assert T * H * 2 >= threshold("mrr_rms_norm_backward.hip", "kStreamBytes")
    x, r, up = (torch.randn(T, H, device=dev, generator=g).to(dtype) for _ in range(3))
    w = (1 + 0.3 * torch.randn(H, device=dev, generator=g)).to(weight)
    assert aligned(x, r, up)
    for more in (r, None):
        out = moe.rms_norm_backward(up, x, w, grad_residual=more)
        for elsewhere in (moe.rms_norm_backward(odd(up), x, w, grad_residual=more),
                          moe.rms_norm_backward(up, odd(x), w, grad_residual=more)):
            assert all(same(a, b) for a, b in zip(out, elsewhere))


# bytes of the choices' rows on either side of what has them read past the caches
@pytest.mark.parametrize("T,k,H,dtype,reads", [
    (700, 8, 2048, BF16, False), (8300, 8, 2056, BF16, True), (900, 3, 1032, F16, False), (3000, 12, 2004, FP32, True),
    (1100, 15, 4096, BF16, False), (70000, 2, 1032, F16, True)])
def test_rows_by_expert_and_back(T, k, H, dtype, reads):
    dev = _dev()
    g = gen(dev, T, k, H)
    E = 24
    assert (T * k * H * dtype.itemsize >= threshold("mrr_token_unpermute.hip", "kPastBytes")) == reads
    x, up = (torch.randn(T, H, device=dev, generator=g).to(dtype) for _ in range(2))
    ids = torch.randint(-2, E + 1, (T, k), device=dev, generator=g, dtype=torch.int32)
    weight = torch.randn(T, k, device=dev, generator=g)
    rows, _, index, num, _ = moe.moe_token_permute(x, ids, E)
    assert aligned(rows, x)
    there = odd(torch.zeros_like(rows))
    moe.moe_token_permute(x, ids, E, out=(there, None, index.clone(), num.clone(), None))
    assert same(rows, there)
    for w in (weight, None):
        y = moe.moe_token_unpermute(rows, index, expert_weight=w)
        d, dw = moe.moe_token_unpermute_backward(up, rows, index, expert_weight=w)
        assert aligned(y, d)
        out = odd(torch.zeros_like(y)), odd(torch.zeros_like(d)), None if dw is None else torch.zeros_like(dw)
        moe.moe_token_unpermute(there, index, expert_weight=w, out=out[0])
        moe.moe_token_unpermute_backward(odd(up), there, index, expert_weight=w, out=out[1:])
        assert same(y, out[0]) and same(d, out[1]) and same(dw, out[2])
