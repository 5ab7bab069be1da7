"""Calls of more tokens than a launch holds."""
import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import _dev

pytestmark = pytest.mark.gpu


def test_gradient_of_more_sums_than_a_launch_holds():
    """2^23 and some tokens of one choice, rows of 4112 bytes by eight waves each: three launches, 103 GB."""
    dev = _dev()
    T, H = (1 << 23) + 3, 2056
    need = 3 * T * H * 2 + T * 12 + (4 << 30)
    if torch.cuda.mem_get_info(dev)[0] < need:
        pytest.skip("less free memory than the call takes")
    g = torch.Generator(dev).manual_seed(5)
    grad, rows = (torch.empty(T, H, dtype=torch.bfloat16, device=dev).uniform_(-1, 1, generator=g) for _ in range(2))
    weight = torch.rand(T, 1, device=dev, generator=g)
    index = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=dev)[:, None]
    index[::1001] = -1 - index[::1001]  # choices that are not here
    d, dw = moe.moe_token_unpermute_backward(grad, rows, index, expert_weight=weight)
    torch.cuda.synchronize()
    step = 1 << 20
    for a in range(0, T, step):
        b = min(T, a + 4096)  # 4096 tokens of each 2^20, and all next to a launch's end
        for lo, hi in ((a, b), (max(0, a - 64), a)):
            w = torch.where(index[lo:hi] >= 0, weight[lo:hi], 0.0)
            want = (grad[lo:hi].float() * w).bfloat16()
            assert torch.equal(d[T - hi:T - lo].flip(0), want), lo
            p = grad[lo:hi].double() * rows[T - hi:T - lo].flip(0).double() * (index[lo:hi] >= 0)
            # at most 2056 products of 24 bits and additions, as in the small tests: 2^-17 of the terms
            assert ((dw[lo:hi, 0].double() - p.sum(1)).abs() <= p.abs().sum(1) * 2.0 ** -17).all(), lo
    del grad, rows, d
    torch.cuda.empty_cache()
