"""The experts' operators on the GPU at the sizes where another of their ways is
taken: the grouped product's large tiles, the few-token layer with many rows of
output, rows that end inside a chunk, scales that are NaN, and the native
binding beside the Python one. Against 64 bits, within the bounds that
experts_reference.py derives."""
import numpy as np
import pytest
import torch

import experts_reference as ref
from gpu_helpers import Guarded, _dev
from moe_token_re_amd import _lib, experts

pytestmark = pytest.mark.gpu

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def _u8(t):
    return t.view(torch.uint8).cpu().numpy()


def _mx(gen, *shape):
    packed = torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, generator=gen)
    scales = torch.randint(119, 124, shape[:-1] + ((shape[-1] + 63) // 64, 2), dtype=torch.uint8, generator=gen)
    return packed, scales


def _fp4(packed, scales, dev):
    return packed.to(dev).view(torch.float4_e2m1fn_x2), scales.to(dev).view(torch.float8_e8m0fnu)


def _unpack64(packed, scales, dev):
    """Packed rows and scales (bytes) as float64 on the GPU."""
    lut = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=dev)
    p = packed.to(dev).long()
    v = lut[torch.stack((p & 15, p >> 4), -1).flatten(-2)]
    f = torch.exp2(scales.to(dev).flatten(-2).double() - 127).repeat_interleave(32, -1)
    return v * f[..., :v.shape[-1]]


# The numbers of rows and columns are such that the large tiles cost least.
LARGE = [
    # A, counts, K, N, gated, dtype, row weight
    (4099, [2500, 0, 1599], 288, 8200, False, "f32", True),
    (4099, [1, 4000, 98], 544, 16400, True, "bf16", False),
    (6000, [300, 257, 256, 255, 1, 4931], 256, 8191, False, "f16", True),
    (9000, [9000], 64, 4098, True, "f32", False),
]


@pytest.mark.parametrize("case", range(len(LARGE)))
def test_grouped_mm_large_tiles(case):
    dev = _dev()
    A, counts, K, N, gated, kind, weighted = LARGE[case]
    gen = torch.Generator().manual_seed(500 + case)
    (xp, xs), (wp, ws) = _mx(gen, A, K), _mx(gen, len(counts), N, K)
    dtype = DTYPES[kind]
    rw = torch.randn(A, generator=gen) if weighted else None
    g = Guarded()
    out = g.like("out", torch.empty(A, N // 2 if gated else N, dtype=dtype, device=dev))
    experts.mx_grouped_mm(*_fp4(xp, xs, dev), *_fp4(wp, ws, dev), torch.tensor(counts, device=dev), gated=gated,
                          row_weight=None if rw is None else rw.to(dev), out=out, check=True)
    g.check(f"grouped {LARGE[case]}")
    x, f, at = _unpack64(xp, xs, dev), (K + 8) * 2.0 ** -23, 0
    fi = torch.finfo(dtype)
    for e, c in enumerate(counts):
        if c == 0:
            continue
        xe, w = x[at:at + c], _unpack64(wp[e], ws[e], dev)
        y, err = xe @ w.T.contiguous(), f * (xe.abs() @ w.abs().T.contiguous())
        if gated:  # as experts_reference.gate has it
            (gt, up), (eg, eu) = y.chunk(2, 1), err.chunk(2, 1)
            s = gt * torch.sigmoid(gt)
            y = s * up
            err = 1.1 * eg * (up.abs() + eu) + s.abs() * eu + y.abs() * (8 + gt.abs()) * 2.0 ** -22
        if rw is not None:
            r = rw[at:at + c].to(dev).double()[:, None]
            y, err = y * r, err * r.abs() + (y * r).abs() * 2.0 ** -23
        bound = err + (y.abs() + err) * (fi.eps / 2) + fi.tiny * (fi.eps / 2)
        off = ((out[at:at + c].double() - y).abs() - bound).max().item()
        assert off <= 0, f"{LARGE[case]} expert {e}: {off} beyond the bound"
        at += c


FEW = [
    # T, E, k, H, I: more than 256 runs of 16 output rows; rows of every ending
    (1, 3, 2, 4160, 64),
    (4, 4, 2, 4128, 288),
    (6, 5, 3, 4352, 320),
    (20, 2, 1, 4160, 96),
    (3, 4, 2, 992, 544),
    (9, 4, 2, 800, 1056),
    (70, 3, 2, 4160, 32),
]


@pytest.mark.parametrize("kind", ["mx", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(FEW)))
def test_few_tokens_many_rows(case, kind):
    dev = _dev()
    T, E, k, H, I = FEW[case]
    gen = torch.Generator().manual_seed(600 + case)
    dtype = torch.bfloat16 if kind == "mx" else DTYPES[kind]
    if kind == "mx":
        (u, us), (d, ds) = _mx(gen, E, 2 * I, H), _mx(gen, E, H, I)
        w = dict(zip(("gate_up", "gate_up_scales", "down", "down_scales"), _fp4(u, us, dev) + _fp4(d, ds, dev)))
        up, down = ref.unpack(u.numpy(), us.numpy()), ref.unpack(d.numpy(), ds.numpy())
    else:
        u = (torch.randn(E, 2 * I, H, generator=gen) * H ** -0.5).to(dtype)
        d = (torch.randn(E, H, I, generator=gen) * I ** -0.5).to(dtype)
        w, up, down = dict(gate_up=u.to(dev), down=d.to(dev)), u.double().numpy(), d.double().numpy()
    x = torch.randn(T, H, generator=gen).to(dtype)
    logits = torch.randn(T, E, generator=gen)
    g = Guarded()
    y = g.like("y", torch.empty(T, H, dtype=dtype, device=dev))
    ws = g.bytes("workspace", experts.few_tokens_workspace_size(T, k, I), dev)
    experts.moe_few_tokens(x.to(dev), router_logits=logits.to(dev), top_k=k, out=y, workspace=ws, **w)
    torch.cuda.synchronize()
    g.check(f"few {FEW[case]} {kind}")
    ids, weights = ref.route(logits.double().numpy(), k, True)
    want, bound = ref.few_tokens(x.double().numpy(), up, down, ids, weights, dtype)
    ref.assert_close(y, want, bound, f"few {FEW[case]} {kind}")


@pytest.mark.parametrize("T", [3, 7])
@pytest.mark.parametrize("H,I", [(96, 160), (288, 96), (544, 352)])
def test_few_tokens_scales(H, I, T):
    """A NaN scale reaches its own row's results and no other; the scale slot of
    no block may hold anything; scales of 0 and 254 are their powers."""
    dev = _dev()
    gen = torch.Generator().manual_seed(71 + H)
    E, k = 2, 1
    (u, us), (d, ds) = _mx(gen, E, 2 * I, H), _mx(gen, E, H, I)
    for s, n in ((us, H), (ds, I)):
        if n // 32 % 2:
            s[..., -1, 1] = 255
    us[0, 3, 0, 0] = 0  # a block that all but vanishes
    x = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    ids = (torch.arange(T, dtype=torch.int32) % 2).reshape(T, 1)
    weight = torch.rand(T, 1, generator=gen) + 0.5

    def run(us, ds):
        g, gs = _fp4(u, us, dev)
        dn, dns = _fp4(d, ds, dev)
        return experts.moe_few_tokens(x.to(dev), g, dn, expert_ids=ids.to(dev), expert_weight=weight.to(dev),
                                      gate_up_scales=gs, down_scales=dns)

    y = run(us, ds)
    want, bound = ref.few_tokens(x.double().numpy(), ref.unpack(u.numpy(), us.numpy()),
                                 ref.unpack(d.numpy(), ds.numpy()), ids.numpy(), weight.double().numpy(), torch.bfloat16)
    ref.assert_close(y, want, bound, "odd blocks")
    ds[1, 5, 0, 1] = 255
    bad = run(us, ds).cpu()
    nan = torch.zeros(T, H, dtype=torch.bool)
    nan[1::2, 5] = True
    assert torch.equal(torch.isnan(bad), nan) and torch.equal(bad[~nan], y.cpu()[~nan])
    ds[1, 5, 0, 1] = 120
    us[0, I + 2, -1, 0] = 255
    bad = run(us, ds).cpu()
    assert torch.isnan(bad[0::2]).all() and not torch.isnan(bad[1::2]).any()


def test_few_tokens_nonfinite_weights_stay_in_their_row():
    """16-bit weights whose rows end inside a chunk: an infinity gives its row's
    results alone."""
    dev = _dev()
    gen = torch.Generator().manual_seed(81)
    T, E, H, I = 6, 2, 96, 32
    gate_up = (torch.randn(E, 2 * I, H, generator=gen) * 0.1).to(torch.bfloat16)
    down = (torch.randn(E, H, I, generator=gen) * 0.1).to(torch.bfloat16)
    x = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    ids, weight = torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1)

    def run(down):
        return experts.moe_few_tokens(x.to(dev), gate_up.to(dev), down.to(dev), expert_ids=ids.to(dev),
                                      expert_weight=weight.to(dev)).cpu()

    y = run(down)
    down[0, 7, 0] = float("inf")
    down[0, 8, 31] = float("nan")
    bad = run(down)
    rest = [i for i in range(H) if i not in (7, 8)]
    assert torch.isinf(bad[:, 7]).all() and torch.isnan(bad[:, 8]).all()
    assert torch.equal(bad[:, rest], y[:, rest])


def test_binding_and_python_agree():
    """The native binding's calls give what the Python ones give, bit for bit; a
    call that is not plain goes the other way."""
    dev = _dev()
    gen = torch.Generator().manual_seed(91)
    fast = _lib.binding()
    x = torch.randn(3, 5, 1058, generator=gen).half().to(dev)
    p, s = fast.quantize(x)
    op = torch.empty(3, 5, 529, dtype=torch.float4_e2m1fn_x2, device=dev)
    os_ = torch.empty(3, 5, 17, 2, dtype=torch.float8_e8m0fnu, device=dev)
    experts.mx_quantize(x, out=(op, os_))
    assert np.array_equal(_u8(p), _u8(op)) and np.array_equal(_u8(s), _u8(os_))
    assert p.dtype == op.dtype and s.dtype == os_.dtype and p.device == x.device
    back = fast.dequantize(p, s, torch.float32)
    out = torch.empty(3, 5, 1058, device=dev)
    assert torch.equal(back, experts.mx_dequantize(p, s, out=out))
    (xp, xs), (wp, ws) = _fp4(*_mx(gen, 9, 96), dev), _fp4(*_mx(gen, 2, 40, 96), dev)
    num, rw = torch.tensor([4, 5], device=dev), torch.rand(9, 1, generator=gen).to(dev)
    y = fast.grouped_mm(xp, xs, wp, ws, num, True, rw, 1, torch.float16)
    assert torch.equal(y, experts.mx_grouped_mm(xp, xs, wp, ws, num, gated=True, row_weight=rw, dtype=torch.float16,
                                                check=True))
    t = torch.randn(6, 64, generator=gen).to(torch.bfloat16).to(dev)
    up, down = torch.randn(3, 64, 64, generator=gen).to(t.dtype).to(dev), torch.randn(3, 64, 32, generator=gen).to(t.dtype).to(dev)
    logits = torch.randn(6, 3, generator=gen).to(dev)
    y = fast.few_tokens(t, up, down, logits, 2, False, None, None, None, None)
    assert torch.equal(y, experts.moe_few_tokens(t, up, down, router_logits=logits, top_k=2, renormalize=False,
                                                 out=torch.empty_like(t)))
    # what it leaves to the Python code, which refuses or makes the call
    assert fast.quantize(x[:, :, ::2]) is None and fast.quantize(x.double()) is None and fast.quantize("x") is None
    assert fast.quantize() is None and fast.dequantize(p, s, torch.int8) is None and fast.dequantize(p, s) is None
    assert fast.dequantize(p, s[:1], torch.float32) is None
    assert fast.grouped_mm(xp, xs, wp, ws, num[:1], True, rw, 1, torch.float16) is None
    assert fast.grouped_mm(xp, xs, wp, ws, num, True, rw, 7, torch.float16) is None
    assert fast.few_tokens(t, up, down, logits, 9, False, None, None, None, None) is None
    assert fast.few_tokens(t, up, down, None, 2, False, None, None, None, None) is None
    assert fast.few_tokens(t, up, down, logits, 2 ** 70, False, None, None, None, None) is None


def test_quantize_on_a_side_stream():
    """The calls go to the current stream, by the binding and by the Python code."""
    dev = _dev()
    x = torch.zeros(2048, 4096, dtype=torch.bfloat16, device=dev)
    side = torch.cuda.Stream(dev)
    out = experts.mx_quantize(torch.ones_like(x))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        x.fill_(3.0)
        a = experts.mx_dequantize(*experts.mx_quantize(x))
        experts.mx_quantize(x, out=out)
        b = experts.mx_dequantize(*out)
    side.synchronize()
    assert (a == 3).all() and (b == 3).all()


def test_weights_past_32_bits():
    """More than 2^32 bytes of weights: the last expert's results are those of
    the same expert alone."""
    dev = _dev()
    g = torch.Generator(dev).manual_seed(101)
    E, N, K = 5, 65536, 32768
    wp = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=dev, generator=g)
    ws = torch.randint(119, 124, (E, N, K // 64, 2), dtype=torch.uint8, device=dev, generator=g)
    xp = torch.randint(0, 256, (6, K // 2), dtype=torch.uint8, device=dev, generator=g)
    xs = torch.randint(119, 124, (6, K // 64, 2), dtype=torch.uint8, device=dev, generator=g)
    y = experts.mx_grouped_mm(xp, xs, wp, ws, torch.tensor([1, 0, 0, 0, 5], device=dev))
    one = experts.mx_grouped_mm(xp[1:].clone(), xs[1:].clone(), wp[4:].clone(), ws[4:].clone(),
                                torch.tensor([5], device=dev))
    assert torch.equal(y[1:], one)
    del wp, ws
    E, H, I = 80, 4096, 4096
    up = torch.empty(E, 2 * I, H, dtype=torch.bfloat16, device=dev).normal_(0, 0.02, generator=g)
    down = torch.empty(E, H, I, dtype=torch.bfloat16, device=dev).normal_(0, 0.02, generator=g)
    x = torch.empty(7, H, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    last, first = torch.full((7, 1), E - 1, dtype=torch.int32, device=dev), torch.zeros(7, 1, dtype=torch.int32, device=dev)
    weight = torch.ones(7, 1, device=dev)
    y = experts.moe_few_tokens(x, up, down, expert_ids=last, expert_weight=weight)
    one = experts.moe_few_tokens(x, up[-1:].clone(), down[-1:].clone(), expert_ids=first, expert_weight=weight)
    assert torch.equal(y, one) and torch.isfinite(y).all() and (y != 0).any()
