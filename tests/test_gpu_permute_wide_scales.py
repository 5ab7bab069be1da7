"""Few choices whose tokens have scale rows of more units than a workgroup has
threads: the last turn of them fills a few lanes, fewer than a token has choices."""
import layer_reference as ref
import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import Guarded, _dev

pytestmark = pytest.mark.gpu


# floats a scale row: 4 make a unit, 256 units a turn
CASES = [(T, k, S) for T, k in ((1, 8), (3, 16), (37, 8), (5, 1), (256, 16), (9, 3))
         for S in (1024, 1025, 1028, 1040, 1100, 2051, 5000)] + [(2, 16, 65536), (3, 5, 65535)]


@pytest.mark.parametrize("T,k,S", CASES)
def test_wide_scale_rows(T, k, S):
    dev = _dev()
    g = torch.Generator().manual_seed(1000 * T + k + S)
    E = 24
    tokens = torch.randint(-128, 128, (T, 40), generator=g, dtype=torch.int8)
    scales = torch.rand(T, S, generator=g)
    ids = torch.randint(-2, E + 1, (T, k), generator=g, dtype=torch.int32)
    index, num = ref.plan(ids, E)
    out = moe.moe_token_permute(tokens.to(dev), ids.to(dev), E, per_token_scales=scales.to(dev))
    guard = Guarded()
    outs = tuple(None if t is None else guard.like(str(i), t) for i, t in enumerate(out))
    moe.moe_token_permute(tokens.to(dev), ids.to(dev), E, per_token_scales=scales.to(dev), out=outs)
    torch.cuda.synchronize()
    guard.check()
    for got in (out, outs):
        assert torch.equal(got[0].cpu(), ref.place(tokens, index)) and torch.equal(got[1].cpu(), ref.place(scales, index))
        assert torch.equal(got[2].cpu(), index) and torch.equal(got[3].cpu(), num)
