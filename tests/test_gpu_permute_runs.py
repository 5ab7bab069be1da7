"""Choices that meet at one expert's next row again and again: a wave places 64
of them at a time, and the next 64 follow on from where it stands."""
import layer_reference as ref
import pytest
import torch

import moe_token_re_amd as moe
from gpu_helpers import _dev

pytestmark = pytest.mark.gpu


def pattern(kind, n, E, g):
    i = torch.arange(n)
    if kind == "one expert":
        return torch.full((n,), E - 1)
    if kind == "in turn":
        return i % min(E, 3)
    if kind == "runs of 64":
        return i // 64 % E
    if kind == "runs of 65":
        return i // 65 % E
    if kind == "the first and the last of 64":
        return torch.where((i % 64 == 0) | (i % 64 == 63), 0, 1 + i % max(E - 1, 1)).clamp(max=E - 1)
    return torch.where(torch.rand(n, generator=g) < 0.9, 0, torch.randint(-1, E, (n,), generator=g))  # mostly one


# blocks that count for themselves and those that share counts; 16, 4 and 1 of a block's waves place them
@pytest.mark.parametrize("T,k", [(4099, 1), (1025, 7), (2048, 8), (9000, 2), (20011, 3)])
@pytest.mark.parametrize("E", [1, 2, 700, 1300, 4096])
@pytest.mark.parametrize("kind", ["one expert", "in turn", "runs of 64", "runs of 65", "the first and the last of 64", "mostly one"])
def test_stable_within_a_wave(T, k, E, kind):
    dev = _dev()
    g = torch.Generator().manual_seed(T + E)
    ids = pattern(kind, T * k, E, g).view(T, k).to(torch.int32)
    tokens = torch.arange(T, dtype=torch.float32)[:, None].expand(T, 2).contiguous()
    weight = torch.arange(T * k, dtype=torch.float32).view(T, k)
    index, num = ref.plan(ids, E)
    rows, _, got, got_num, w = moe.moe_token_permute(tokens.to(dev), ids.to(dev), E, expert_weight=weight.to(dev))
    assert torch.equal(got.cpu(), index) and torch.equal(got_num.cpu(), num)
    assert torch.equal(rows.cpu(), ref.place(tokens, index))
    want = torch.zeros(T * k)
    flat = index.flatten().long()
    want[flat[flat >= 0]] = weight.flatten()[flat >= 0]
    assert torch.equal(w.cpu().flatten(), want)
