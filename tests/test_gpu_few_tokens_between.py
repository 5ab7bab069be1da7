"""What the few-token layer holds between its two products, p silu(g) u: two bf16
values, whatever the tokens' type, which have the range of 32 bits. The first is
the next bf16 towards zero, so the second has at most 2^-7 of the value, and is
rounded by at most 2^-8 of itself: together they are off by at most 2^-15.
Against 64 bits, within bounds that have that and the result's own rounding."""
import numpy as np
import pytest
import torch

import experts_reference as ref
from gpu_helpers import _dev
from moe_token_re_amd import experts

pytestmark = pytest.mark.gpu

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "mx": torch.bfloat16}


def _weights(gen, E, H, I, kind, dev):
    """(arguments, float64 gate_up, float64 down)."""
    if kind == "mx":
        def rows(*shape):
            p = torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, generator=gen)
            s = torch.randint(119, 124, shape[:-1] + ((shape[-1] + 63) // 64, 2), dtype=torch.uint8, generator=gen)
            return p, s
        (u, us), (d, ds) = rows(E, 2 * I, H), rows(E, H, I)
        return (dict(gate_up=u.to(dev), gate_up_scales=us.to(dev), down=d.to(dev), down_scales=ds.to(dev)),
                ref.unpack(u.numpy(), us.numpy()), ref.unpack(d.numpy(), ds.numpy()))
    u = (torch.randn(E, 2 * I, H, generator=gen) * H ** -0.5).to(DTYPES[kind])
    d = (torch.randn(E, H, I, generator=gen) * I ** -0.5).to(DTYPES[kind])
    return dict(gate_up=u.to(dev), down=d.to(dev)), u.double().numpy(), d.double().numpy()


def _want(x, up, down, ids, weights, dtype, h_eps):
    """(y, bound) in 64 bits: a relative h_eps and what 32 bits lose between the
    products, one rounding to dtype at the end."""
    y, err = ref.few_tokens(x, up, down, ids, weights, torch.float32)
    h = np.zeros_like(y)  # sum over j of |h| |down|
    for t in range(x.shape[0]):
        for e, p in zip(ids[t], weights[t]):
            if 0 <= e < up.shape[0]:
                one, _ = ref.gate(x[t:t + 1], up[e])
                h[t] += (np.abs(one * p) @ np.abs(down[e]).T)[0]
    return y, ref.rounding(y, err + h * h_eps, dtype)


# T, E, k, H, I: the second kernel with one workgroup a run of rows, with several, with four waves, with two
# groups of tokens, with more than 16 tokens an expert
CASES = [(1, 4, 2, 64, 32), (3, 8, 2, 288, 96), (20, 9, 4, 96, 160), (9, 4, 2, 800, 1056), (40, 2, 2, 64, 288),
         (70, 3, 2, 4160, 64), (128, 40, 5, 96, 96)]


@pytest.mark.parametrize("kind", ["mx", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_precision_between_the_products(case, kind):
    dev = _dev()
    T, E, k, H, I = CASES[case]
    gen = torch.Generator().manual_seed(700 + case)
    w, up, down = _weights(gen, E, H, I, kind, dev)
    x = torch.randn(T, H, generator=gen).to(DTYPES[kind])
    logits = torch.randn(T, E, generator=gen)
    y = experts.moe_few_tokens(x.to(dev), router_logits=logits.to(dev), top_k=k, **w)
    ids, weights = ref.route(logits.double().numpy(), k, True)
    want, bound = _want(x.double().numpy(), up, down, ids, weights, DTYPES[kind], 2.0 ** -15)
    ref.assert_close(y, want, bound, f"{CASES[case]} {kind}")


@pytest.mark.parametrize("kind", ["mx", "bf16", "f16"])
@pytest.mark.parametrize("power", [-60, -40, -24, -14, 12, 24, 60])
@pytest.mark.parametrize("T", [2, 9])
def test_range_between_the_products(T, power, kind):
    """p of 2^power and down rows of 2^-power: an intermediate that 16 bits
    cannot hold, and results that they can. (fp16 rows of that size only as far
    as fp16 goes; p u is what grows there.)"""
    dev = _dev()
    E, H, I = 2, 64, 96
    gen = torch.Generator().manual_seed(800 + power + T)
    x = torch.randn(T, H, generator=gen).to(DTYPES[kind])
    ids = (torch.arange(T, dtype=torch.int32) % E).reshape(T, 1)
    w, up, down = _weights(gen, E, H, I, kind, dev)
    if kind == "mx":
        s = w["down_scales"].cpu().int() - power
        w["down_scales"] = s.to(torch.uint8).to(dev)
        down = ref.unpack(w["down"].cpu().numpy(), w["down_scales"].cpu().numpy())
    else:
        shift = power if kind == "bf16" else max(min(power, 12), -12)
        w["down"] = (w["down"].double() * 2.0 ** -shift).to(DTYPES[kind])
        down = w["down"].cpu().double().numpy()
    p = 2.0 ** power
    if kind == "f16":  # down rows of fp16 have no more range: the result's size then follows p
        p = 2.0 ** max(min(power, 14), -24)
    weight = torch.rand(T, 1, generator=gen) * p + p
    y = experts.moe_few_tokens(x.to(dev), expert_ids=ids.to(dev), expert_weight=weight.to(dev), **w)
    want, bound = _want(x.double().numpy(), up, down, ids.numpy(), weight.double().numpy(), DTYPES[kind],
                        2.0 ** -15)
    ref.assert_close(y, want, bound, f"T {T} power {power} {kind}")
    assert torch.isfinite(y).all()


def test_large_fp16_intermediate():
    """silu(g) u of a few hundred thousand, past the largest fp16, and results
    that fp16 holds."""
    dev = _dev()
    T, E, H, I = 5, 1, 64, 32
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, generator=gen).half()
    up = (torch.randn(E, 2 * I, H, generator=gen) * 50).half()
    down = (torch.randn(E, H, I, generator=gen) * 2 ** -9).half()
    ids, weight = torch.zeros(T, 1, dtype=torch.int32), torch.full((T, 1), 4.0)
    h, _ = ref.gate(x.double().numpy(), up[0].double().numpy())
    assert (np.abs(h) * 4 > 65504).any()
    y = experts.moe_few_tokens(x.to(dev), up.to(dev), down.to(dev), expert_ids=ids.to(dev), expert_weight=weight.to(dev))
    want, bound = _want(x.double().numpy(), up.double().numpy(), down.double().numpy(), ids.numpy(),
                        weight.double().numpy(), torch.float16, 2.0 ** -15)
    assert np.abs(want).max() < 60000
    ref.assert_close(y, want, bound, "large fp16 intermediate")


@pytest.mark.parametrize("kind", ["mx", "bf16", "f16"])
def test_infinities_between_the_products(kind):
    """An infinite weight p gives what the definition gives: an infinity or a
    NaN in that token's results, and the other tokens' as they were."""
    dev = _dev()
    T, E, H, I = 6, 2, 96, 64
    gen = torch.Generator().manual_seed(82)
    w, up, down = _weights(gen, E, H, I, kind, dev)
    x = torch.randn(T, H, generator=gen).to(DTYPES[kind])
    ids = (torch.arange(T, dtype=torch.int32) % E).reshape(T, 1)
    weight = torch.ones(T, 1)
    run = lambda: experts.moe_few_tokens(x.to(dev), expert_ids=ids.to(dev), expert_weight=weight.to(dev), **w).cpu()
    clean = run()
    weight[2], weight[3] = float("inf"), float("nan")
    y = run()
    rest = [0, 1, 4, 5]
    assert torch.equal(y[rest], clean[rest])
    assert not torch.isfinite(y[2]).any() and torch.isnan(y[3]).all()
