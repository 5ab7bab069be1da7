"""Weights of experts whose logits lie far below the largest: down to the
smallest numbers of 32 bits, and 0 below them alone."""
import layer_reference as ref
import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E,k", [(16, 2), (60, 8), (300, 16)])
def test_small_weights(E, k, dtype, renormalize):
    dev = _dev()
    gaps = torch.tensor([0.5, 80, 86, 86.6, 87, 87.3, 87.4, 88, 90, 95, 100, 103, 103.9, 104.5, 110, 1000, 30000])
    logits = torch.zeros(len(gaps), E)
    logits[:, 1:] = -gaps[:, None] - torch.arange(E - 1) * (0.01 if dtype == torch.float32 else 0.0)
    logits = (logits + 3.25).to(dtype)
    weight, ids = moe.moe_router_top_k(logits.to(dev), k, renormalize=renormalize)
    want, want_ids = ref.router(logits, k, renormalize)
    assert torch.equal(ids.cpu(), want_ids)
    # 2^-17 of a weight, as in the other tests, and two roundings to a multiple of 2^-149
    assert ((weight.double().cpu() - want).abs() <= want * 2.0 ** -17 + 2.0 ** -149).all()
    assert ((want > 2.0 ** -148) <= (weight.cpu() > 0)).all() and (weight[-1, 1:] == 0).all()
    lowest = logits.clone()
    lowest[:, 1:] = torch.finfo(dtype).min  # a mask of the type's lowest value
    weight, ids = moe.moe_router_top_k(lowest.to(dev), k, renormalize=renormalize)
    assert (weight[:, 0] == 1).all() and (weight[:, 1:] == 0).all() and ids[0].tolist() == list(range(k))
