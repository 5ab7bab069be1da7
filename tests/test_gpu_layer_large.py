"""Calls whose rows go past the caches (from 64 MiB of them, and from 256 MiB
where they are read): bit for bit what the same call in parts gives, whose rows
do not, and which the small tests compare with the definitions."""
import zlib

import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import Guarded, _dev

pytestmark = pytest.mark.gpu


def gen(dev, *parts):
    return torch.Generator(dev).manual_seed(zlib.crc32(repr(parts).encode()))


def same(a, b):
    return (a is None and b is None) or torch.equal(a.contiguous().view(-1).view(torch.uint8),
                                                    b.contiguous().view(-1).view(torch.uint8))


def guarded(outs):
    guard = Guarded()
    return guard, tuple(None if t is None else guard.like(str(i), t) for i, t in enumerate(outs))


@pytest.mark.parametrize("T,H,dtype,weight", [
    (8200, 4096, torch.bfloat16, torch.float32), (5000, 7168, torch.float16, torch.float16),
    (70000, 512, torch.bfloat16, torch.bfloat16), (34000, 1000, torch.float16, torch.float32),
    (2100, 16384, torch.bfloat16, torch.bfloat16), (9000, 2044, torch.float32, torch.float32)])
def test_norm_and_its_gradient(T, H, dtype, weight):
    dev = _dev()
    g = gen(dev, T, H)
    x, r, up = (torch.randn(T, H, device=dev, generator=g).to(dtype) for _ in range(3))
    w = (1 + 0.3 * torch.randn(H, device=dev, generator=g)).to(weight)
    x[3], x[T - 1, 5] = 0, float("inf")
    assert x.numel() * x.element_size() >= 64 << 20
    half = [(0, T // 3), (T // 3, 2 * T // 3), (2 * T // 3, T)]
    for quantize in (None, "int8", "fp8", "mxfp8", "mxfp4"):
        for residual in (r, None):
            out = moe.rms_norm(x, w, residual=residual, quantize=quantize)
            guard, outs = guarded(out)
            moe.rms_norm(x, w, residual=residual, quantize=quantize, out=outs)
            torch.cuda.synchronize()
            guard.check()
            for a, b in half:
                part = moe.rms_norm(x[a:b], w, residual=None if residual is None else residual[a:b], quantize=quantize)
                assert all((p is None and o is None) or (same(o[a:b], p) and same(q[a:b], p))
                           for p, o, q in zip(part, out, outs)), (quantize, a)
    x[T - 1, 5] = 1
    for more in (r, None):
        out = moe.rms_norm_backward(up, x, w, grad_residual=more)
        guard, outs = guarded(out)
        moe.rms_norm_backward(up, x, w, grad_residual=more, out=outs)
        torch.cuda.synchronize()
        guard.check()
        assert same(out[0], outs[0]) and same(out[1], outs[1])
        sums = torch.zeros(H, device=dev, dtype=torch.float64)
        for a, b in half:
            d, dw = moe.rms_norm_backward(up[a:b], x[a:b], w.float() if dtype == torch.float32 else w,
                                          grad_residual=None if more is None else more[a:b])
            assert same(out[0][a:b], d), (a, more is None)
            sums += dw.double()
        n = x.double() / torch.sqrt(x.double().square().mean(1, keepdim=True) + 1e-6)
        want = (up.double() * n).sum(0)
        size = (up.double() * n).abs().sum(0)
        # a rounding to the weight's type, and at most 70000 / 2048 + 2048 / 64 + 16 additions of 2^-24 each
        most = want.abs() * torch.finfo(weight).eps / 2 + size * 2.0 ** -17
        assert ((out[1].double() - want).abs() <= most).all()


@pytest.mark.parametrize("T,k,H,dtype", [
    (4096, 8, 1040, torch.bfloat16), (9000, 8, 2048, torch.bfloat16), (3000, 12, 2000, torch.float32),
    (70000, 2, 1032, torch.float16), (2000, 16, 4096, torch.float32)])
def test_rows_by_expert_and_back(T, k, H, dtype):
    """Some choices are not here; some indices are no rows."""
    dev = _dev()
    g = gen(dev, T, k, H)
    E = 24
    x, up = (torch.randn(T, H, device=dev, generator=g).to(dtype) for _ in range(2))
    ids = torch.randint(-2, E + 1, (T, k), device=dev, generator=g, dtype=torch.int32)
    weight = torch.randn(T, k, device=dev, generator=g)
    rows, _, index, num, _ = out = moe.moe_token_permute(x, ids, E)
    assert rows.numel() * rows.element_size() >= 64 << 20
    guard, outs = guarded(out)
    moe.moe_token_permute(x, ids, E, out=outs)
    torch.cuda.synchronize()
    guard.check()
    assert all(same(a, b) for a, b in zip(out, outs))
    flat = torch.where((ids < 0) | (ids >= E), E, ids).flatten().long()
    order = torch.sort(flat, stable=True)[1]
    assert torch.equal(num.long(), torch.bincount(flat, minlength=E + 1)[:E])
    for a in range(0, T * k, 20000):
        at = order[a:a + 20000]
        assert torch.equal(rows[a:a + 20000], torch.where((flat[at] < E)[:, None], x[at // k], 0))
    index[5, 0] = T * k  # no row: nothing is added, and no gradient written
    part = 60_000_000 // (k * H * x.element_size())
    for w in (weight, None):
        y = moe.moe_token_unpermute(rows, index, expert_weight=w)
        d, dw = out = moe.moe_token_unpermute_backward(up, rows, index, expert_weight=w)
        guard, outs = guarded((y, d, dw))
        moe.moe_token_unpermute(rows, index, expert_weight=w, out=outs[0])
        moe.moe_token_unpermute_backward(up, rows, index, expert_weight=w, out=outs[1:])
        torch.cuda.synchronize()
        guard.check()
        lost = (order == 5 * k).nonzero()[0, 0]  # the row that no index names any more
        for t in (d, outs[1]):
            t[lost] = 0
        assert same(y, outs[0]) and same(d, outs[1]) and same(dw, outs[2])
        parts = torch.zeros_like(d)
        for a in range(0, T, part):
            b = min(T, a + part)
            small = None if w is None else w[a:b]
            assert same(y[a:b], moe.moe_token_unpermute(rows, index[a:b], expert_weight=small))
            own = parts if w is None else torch.zeros_like(d)
            dw_part = None if w is None else torch.empty(b - a, k, device=dev)
            moe.moe_token_unpermute_backward(up[a:b], rows, index[a:b], expert_weight=small, out=(own, dw_part))
            if w is not None:
                assert same(dw[a:b], dw_part)
                parts += own
        parts[lost] = 0
        assert torch.equal(d, parts)
