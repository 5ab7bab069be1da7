"""Where several workgroups share a run of output rows in the few-token layer's
second kernel: the last to arrive adds their sums in order, so repeated calls,
calls on one workspace and replays of a graph give the same bits. That a shape
takes this way is read from the counts of arrived workgroups, which the call
leaves in the workspace."""
import pytest
import torch

import experts_reference as ref
from gpu_helpers import Guarded, _dev
from moe_token_re_amd import experts

pytestmark = pytest.mark.gpu

# T, E, k, H, I: one tile of eight tokens; two and four tiles; two groups of 64 tokens
CASES = [(2, 8, 4, 64, 2048), (9, 64, 2, 256, 2048), (40, 3, 2, 64, 2048), (40, 12, 4, 512, 1024), (30, 9, 2, 96, 2048),
         (100, 8, 2, 128, 1024), (128, 24, 4, 96, 2048)]


def _arrived(ws, T, k, H):
    """The workgroups that each run of 16 or 32 rows had (0: one alone, which does not count)."""
    at = 3 * ((4 * T * k + 255) // 256 * 256)
    runs = H // 32 * (2 if T > 64 else 1)
    return ws[at:at + 4 * 512].view(torch.int32)[:runs].cpu()


def _case(case, kind, dev):
    T, E, k, H, I = CASES[case]
    gen = torch.Generator().manual_seed(1100 + case)
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
    logits = torch.randn(T, E, generator=gen)
    return gen, w, up, down, x, logits, dtype


@pytest.mark.parametrize("kind", ["mx", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_join_repeats_bit_for_bit(case, kind):
    dev = _dev()
    T, E, k, H, I = CASES[case]
    _, w, up, down, x, logits, dtype = _case(case, kind, dev)
    g = Guarded()
    ws = g.bytes("workspace", experts.few_tokens_workspace_size(T, k, I), dev)
    call = dict(router_logits=logits.to(dev), top_k=k, **w)
    xd, first = x.to(dev), None
    for _ in range(6):  # on one workspace, with what the call before left there
        y = g.like("y", torch.empty(T, H, dtype=dtype, device=dev))
        experts.moe_few_tokens(xd, out=y, workspace=ws, **call)
        first = y.clone() if first is None else first
        assert torch.equal(y, first)
    counts = _arrived(ws, T, k, H)
    assert counts.min() > 1 and (counts == counts[0]).all(), f"{CASES[case]} {kind}: {counts}"
    g.check(f"{CASES[case]} {kind}")
    ws.fill_(0xff)
    experts.moe_few_tokens(xd, out=y, workspace=ws, **call)
    assert torch.equal(y, first)
    for _ in range(3):
        assert torch.equal(experts.moe_few_tokens(xd, **call), first)
    ids, weights = ref.route(logits.double().numpy(), k, True)
    want, bound = ref.few_tokens(x.double().numpy(), up, down, ids, weights, dtype)
    ref.assert_close(first, want, bound, f"{CASES[case]} {kind}")


@pytest.mark.parametrize("case,kind", [(1, "mx"), (3, "bf16"), (4, "mx"), (5, "f16")])
def test_join_in_a_graph(case, kind):
    """One workspace, given, through a graph's replays and eager calls in turn."""
    dev = _dev()
    T, E, k, H, I = CASES[case]
    gen, w, _, _, x, logits, dtype = _case(case, kind, dev)
    xd, ld = x.to(dev), logits.to(dev)
    ws = torch.empty(experts.few_tokens_workspace_size(T, k, I), dtype=torch.uint8, device=dev)
    y = torch.empty(T, H, dtype=dtype, device=dev)
    side = torch.cuda.Stream(dev)

    def call(out):
        experts.moe_few_tokens(xd, router_logits=ld, top_k=k, out=out, workspace=ws, **w)

    with torch.cuda.stream(side):
        call(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(y)
    for replay in range(5):
        xd.copy_(torch.randn(T, H, generator=gen))
        ld.copy_(torch.randn(T, E, generator=gen))
        want = torch.empty_like(y)
        call(want)
        torch.cuda.synchronize()
        assert _arrived(ws, T, k, H).min() > 1
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), replay
        assert _arrived(ws, T, k, H).min() > 1
