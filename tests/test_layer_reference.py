"""The 64-bit definitions that the GPU tests of the operators around a layer
compare with, against differences and against each other. No GPU."""
import layer_reference as ref
import pytest
import torch


def difference(f, x, direction, h=1e-6):
    """The derivative of f at x along a direction, by central differences."""
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


@pytest.mark.parametrize("rows,H,with_sum", [(1, 1, False), (3, 7, True), (4, 64, False)])
def test_norm_backward_is_the_derivative(rows, H, with_sum):
    g = torch.Generator().manual_seed(rows * 100 + H)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, up, up_sum = rand(rows, H), rand(H), rand(rows, H), rand(rows, H)
    dx, dw = ref.norm_backward(up, x, w, 1e-3, up_sum if with_sum else None)
    loss = lambda x, w: (ref.norm(x, w, 1e-3)[0] * up).sum() + ((x * up_sum).sum() if with_sum else 0)  # noqa: E731
    for _ in range(3):
        d, e = rand(rows, H), rand(H)
        assert torch.allclose((dx * d).sum(), difference(lambda x: loss(x, w), x, d), rtol=1e-6, atol=1e-8)
        assert torch.allclose((dw * e).sum(), difference(lambda w: loss(x, w), w, e), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("renormalize", [True, False])
def test_router_backward_is_the_derivative(renormalize):
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(4, 9, generator=g, dtype=torch.float64)
    logits[1, 3] = float("-inf")
    up = torch.randn(4, 3, generator=g, dtype=torch.float64)
    _, ids = ref.router(logits, 3, renormalize)
    d = torch.randn(4, 9, generator=g, dtype=torch.float64)
    d[1, 3] = 0
    got = (ref.router_backward(up, logits, ids, renormalize) * d).sum()
    want = difference(lambda x: (ref.router(x, 3, renormalize)[0] * up).sum(), logits, d)
    assert torch.allclose(got, want, rtol=1e-6, atol=1e-9)


def test_combine_backward_is_the_derivative_and_the_transpose():
    g = torch.Generator().manual_seed(4)
    ids = torch.tensor([[2, 0], [5, 2], [-1, 1], [0, 0]], dtype=torch.int32)
    index, num = ref.plan(ids, 3)
    assert num.tolist() == [3, 1, 2] and sorted(i if i >= 0 else -1 - i for i in index.flatten().tolist()) == list(range(8))
    assert index.tolist() == [[4, 0], [-7, 5], [-8, 3], [1, 2]]
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    rows, w, up = rand(8, 5), rand(4, 2), rand(4, 5)
    d, dw, _ = ref.combine_backward(up, rows, index, w)
    e, f = rand(8, 5), rand(4, 2)
    assert torch.allclose((d * e).sum(), difference(lambda r: (ref.combine(r, index, w)[0] * up).sum(), rows, e))
    assert torch.allclose((dw * f).sum(), difference(lambda v: (ref.combine(rows, index, v)[0] * up).sum(), w, f))
    # moving rows out and adding them back are each other's transpose
    x = rand(4, 5)
    assert torch.allclose((ref.place(x, index) * rows).sum(), (x * ref.combine(rows, index)[0]).sum())


def test_roundings_to_few_bits():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    every = every[every.isfinite()]
    assert torch.equal(ref.e4m3(every), every)
    v = torch.randn(4096, generator=torch.Generator().manual_seed(0), dtype=torch.float64) * 100
    assert torch.equal(ref.e4m3(v), v.float().clamp(-448, 448).to(torch.float8_e4m3fn).double())
    assert ref.e4m3(torch.tensor([464.0, 1e9, -1e9, 17.0, 19.0, 2.0 ** -10], dtype=torch.float64)).tolist() == [
        448, 448, -448, 16, 20, 0]
    assert ref.e2m1(torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -9.0], dtype=torch.float64)).tolist() == [
        0, 1, 1, 2, 2, 4, 4, 6, -6]
