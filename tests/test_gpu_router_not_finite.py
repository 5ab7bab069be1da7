"""The router's gradient where no logit of a row is a number: a NaN stays one."""
import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E", [5, 64, 100, 256, 300, 1000])
def test_gradient_of_rows_of_nan(E, dtype):
    dev = _dev()
    nan, inf = float("nan"), float("inf")
    logits = torch.zeros(7, E)
    logits[0] = nan
    logits[1] = -inf
    logits[1, E - 1] = nan  # the only expert that can be chosen
    logits[2] = -inf  # none can
    logits[3, 1:] = -inf
    logits[4] = nan
    logits[4, E // 2] = -inf
    logits[5, 2], logits[5, 3:] = nan, -inf
    logits = logits.to(dtype).to(dev)
    up = torch.randn(7, 3, generator=torch.Generator().manual_seed(E)).to(dev)
    for renormalize in (True, False):
        weight, ids = moe.moe_router_top_k(logits, 3, renormalize=renormalize)
        assert ids[[0, 1, 2, 3, 5]].tolist() == [[0, 1, 2], [E - 1, -1, -1], [-1] * 3, [0, -1, -1], [2, 0, 1]]
        assert torch.isnan(weight[0]).all() and torch.isnan(weight[1, 0]) and weight[1, 1:].tolist() == [0, 0]
        d = moe.moe_router_top_k_backward(up, logits, weight, ids, renormalize=renormalize)
        assert (d[2] == 0).all() and (d[3] == 0).all() and torch.isfinite(d[6]).all()
        for row in (0, 1, 4, 5):
            chosen = ids[row][ids[row] >= 0].long()
            assert torch.isnan(d[row][chosen]).all(), row
            if renormalize:  # the others have no part
                rest = torch.ones(E, dtype=torch.bool, device=dev).scatter_(0, chosen, False)
                assert (d[row][rest] == 0).all(), row
            else:  # a softmax over a NaN is nothing else
                assert torch.isnan(d[row]).all(), row
