"""The few-token layer where a rank has fewer experts than a token chooses of
all ranks' (expert_ids): against 64 bits, within the bounds that
experts_reference.py derives, by the native binding and by the Python code."""
import pytest
import torch

import experts_reference as ref
from gpu_helpers import Guarded, _dev
from moe_token_re_amd import api, experts

pytestmark = pytest.mark.gpu

# T, E, k, H, I
CASES = [(1, 1, 2, 64, 32), (1, 1, 16, 64, 32), (3, 4, 6, 96, 160), (16, 4, 6, 288, 96), (20, 2, 8, 64, 64),
         (70, 3, 16, 96, 32), (128, 1, 16, 64, 32), (128, 15, 16, 64, 64)]


@pytest.mark.parametrize("kind", ["mx", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_fewer_experts_than_choices(case, kind):
    dev = _dev()
    T, E, k, H, I = CASES[case]
    gen = torch.Generator().manual_seed(1000 + case)
    dtype = torch.float16 if kind == "f16" else torch.bfloat16
    if kind == "mx":
        def rows(*shape):
            return (torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, generator=gen),
                    torch.randint(119, 124, shape[:-1] + ((shape[-1] + 63) // 64, 2), dtype=torch.uint8, generator=gen))
        (u, us), (d, ds) = rows(E, 2 * I, H), rows(E, H, I)
        w = dict(gate_up=u.to(dev), gate_up_scales=us.to(dev), down=d.to(dev), down_scales=ds.to(dev))
        up, down = ref.unpack(u.numpy(), us.numpy()), ref.unpack(d.numpy(), ds.numpy())
    else:
        u = (torch.randn(E, 2 * I, H, generator=gen) * H ** -0.5).to(dtype)
        d = (torch.randn(E, H, I, generator=gen) * I ** -0.5).to(dtype)
        w, up, down = dict(gate_up=u.to(dev), down=d.to(dev)), u.double().numpy(), d.double().numpy()
    x = torch.randn(T, H, generator=gen).to(dtype)
    # experts of all ranks, this one's own among them, each named once; one token names an own expert twice
    ids = torch.stack([torch.randperm(max(k, 2 * E) + 2, generator=gen)[:k] for _ in range(T)]).to(torch.int32) - 1
    ids[T // 2, :2] = E - 1
    weight = torch.randn(T, k, generator=gen)
    want, bound = ref.few_tokens(x.double().numpy(), up, down, ids.numpy(), weight.double().numpy(), dtype)
    call = dict(expert_ids=ids.to(dev), expert_weight=weight.to(dev), **w)
    ref.assert_close(experts.moe_few_tokens(x.to(dev), **call), want, bound, f"{CASES[case]} {kind}")
    g = Guarded()
    y = g.like("y", torch.empty(T, H, dtype=dtype, device=dev))
    ws = g.bytes("workspace", experts.few_tokens_workspace_size(T, k, I), dev)
    experts.moe_few_tokens(x.to(dev), out=y, workspace=ws, **call)
    torch.cuda.synchronize()
    g.check(f"{CASES[case]} {kind}")
    ref.assert_close(y, want, bound, f"{CASES[case]} {kind}, out given")


@pytest.mark.parametrize("T", [0, 2])
def test_logits_choose_among_the_experts_there_are(T):
    dev = _dev()
    x = torch.zeros(T, 64, dtype=torch.bfloat16, device=dev)
    up, down = torch.zeros(3, 64, 64, dtype=x.dtype, device=dev), torch.zeros(3, 64, 32, dtype=x.dtype, device=dev)
    for out in (None, torch.empty_like(x)):
        with pytest.raises(api.MrrValueError):
            experts.moe_few_tokens(x, up, down, router_logits=torch.zeros(T, 3, device=dev), top_k=4, out=out)
        y = experts.moe_few_tokens(x, up, down, expert_ids=torch.zeros(T, 4, dtype=torch.int32, device=dev),
                                   expert_weight=torch.zeros(T, 4, device=dev), out=out)
        assert y.shape == (T, 64)
