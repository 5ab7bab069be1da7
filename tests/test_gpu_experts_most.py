"""The experts' operators with as many experts as they take: 1024 of a few-token
layer, 4096 of a grouped product. Against 64 bits, within the bounds that
experts_reference.py derives."""
import numpy as np
import pytest
import torch

import experts_reference as ref
from gpu_helpers import _dev
from moe_token_re_amd import experts

pytestmark = pytest.mark.gpu


def _mx(gen, *shape):
    return (torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, generator=gen),
            torch.randint(119, 124, shape[:-1] + ((shape[-1] + 63) // 64, 2), dtype=torch.uint8, generator=gen))


@pytest.mark.parametrize("kind", ["mx", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,k", [(1, 16), (3, 8), (70, 16), (128, 16)])
def test_few_tokens_of_1024_experts(T, k, renorm, kind):
    dev, E, H, I = _dev(), 1024, 64, 32
    gen = torch.Generator().manual_seed(1200 + T + k)
    if kind == "mx":
        (u, us), (d, ds) = _mx(gen, E, 2 * I, H), _mx(gen, E, H, I)
        w = dict(gate_up=u.to(dev), gate_up_scales=us.to(dev), down=d.to(dev), down_scales=ds.to(dev))
        up, down = ref.unpack(u.numpy(), us.numpy()), ref.unpack(d.numpy(), ds.numpy())
    else:
        u = (torch.randn(E, 2 * I, H, generator=gen) * H ** -0.5).to(torch.bfloat16)
        d = (torch.randn(E, H, I, generator=gen) * I ** -0.5).to(torch.bfloat16)
        w, up, down = dict(gate_up=u.to(dev), down=d.to(dev)), u.double().numpy(), d.double().numpy()
    x = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen) * 2
    logits[0, [1023, 0, 512]] = 9.0  # the first and the last expert, alike
    ids, weights = ref.route(logits.double().numpy(), k, renorm)
    assert {0, 512, 1023} <= set(ids[0].tolist())
    want, bound = ref.few_tokens(x.double().numpy(), up, down, ids, weights, torch.bfloat16)
    y = experts.moe_few_tokens(x.to(dev), router_logits=logits.to(dev), top_k=k, renormalize=renorm, **w)
    ref.assert_close(y, want, bound, f"logits, {T} tokens")
    y = experts.moe_few_tokens(x.to(dev), expert_ids=torch.tensor(ids, dtype=torch.int32, device=dev),
                               expert_weight=torch.tensor(weights, dtype=torch.float32, device=dev), **w)
    want, bound = ref.few_tokens(x.double().numpy(), up, down, ids, weights.astype(np.float32).astype(np.float64),
                                 torch.bfloat16)
    ref.assert_close(y, want, bound, f"ids, {T} tokens")


@pytest.mark.parametrize("counts_dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("running", [False, True])
@pytest.mark.parametrize("A", [1, 3000, 20000])
def test_grouped_mm_of_4096_experts(A, running, counts_dtype):
    dev, E, K, N = _dev(), 4096, 64, 40
    gen = torch.Generator().manual_seed(1300 + A)
    (xp, xs), (wp, ws) = _mx(gen, A, K), _mx(gen, E, N, K)
    # all sizes: many experts without rows, some with more than a tile, the last one among those that have some
    of_row = (torch.rand(A, generator=gen) ** 6 * E).long()
    of_row[0] = E - 1
    counts = torch.bincount(of_row, minlength=E)
    num = (counts.cumsum(0) if running else counts).to(counts_dtype)
    y = experts.mx_grouped_mm(xp.to(dev), xs.to(dev), wp.to(dev), ws.to(dev), num.to(dev),
                              expert_token_num_type=0 if running else 1, dtype=torch.float32, check=True)
    want, bound = ref.grouped(ref.unpack(xp.numpy(), xs.numpy()), ref.unpack(wp.numpy(), ws.numpy()), counts.tolist(),
                              False, None, torch.float32)
    ref.assert_close(y, want, bound, f"{A} rows of {E} experts")
