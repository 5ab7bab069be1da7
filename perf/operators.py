"""Cases of the expert operators, for measuring them: microscaled 4-bit
quantisation and its inverse, the grouped product over expert-major rows, and
the whole mixture-of-experts layer for a few tokens.

`listed()` names the cases, `draw()` gives more of the same ranges,
`prepare()` makes a case's inputs on the GPU from a seed, and `run()` makes
one pass: through the library where `own` is true, else in plain torch
operations in 32 bits. `exact()` computes the same outputs in 64 bits from the
operators' definitions, and `work()` says what a pass has to move and compute.

The microscaled format (OCP MX, elements e2m1, scales e8m0): 32 values of a
row share the scale 2^(s - 127); s - 127 = floor(log2(max |x|)) - 2 of the
block, and each value divided by the scale is rounded to the nearest of
0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, ties to the even code, larger
ones to 6. Two values share a byte, the first in the low nibble. Scales of a
row of H values are [ceil(H / 64), 2] bytes.
"""
import math
from statistics import NormalDist

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------- cases

def listed():
    return [
        # quantise rows before they are sent or multiplied, and read them back:
        # the row of a single new token
        {"name": "quant_one_row", "op": "quant", "A": 1, "H": 7168, "dtype": "bf16"},
        # an odd row length (no whole number of 32-value blocks), half precision
        {"name": "quant_odd_f16", "op": "quant", "A": 777, "H": 1058, "dtype": "f16"},
        # an ordinary batch held in single precision
        {"name": "quant_f32", "op": "quant", "A": 4096, "H": 2048, "dtype": "f32"},
        # the re-routing operator's own row count and length
        {"name": "quant_16384", "op": "quant", "A": 16384, "H": 7168, "dtype": "bf16"},
        # experts' products over expert-major rows: a decode step, about four
        # rows an expert, bound by the weights
        {"name": "group_decode", "op": "group", "A": 64, "E": 16, "K": 2048, "N": 4096, "gated": True,
         "skew": 0.0, "row_weight": False, "dtype": "bf16"},
        # ragged everything: experts without rows, a row length of 33 blocks
        {"name": "group_ragged", "op": "group", "A": 1237, "E": 24, "K": 1056, "N": 1111, "gated": False,
         "skew": 1.2, "row_weight": True, "dtype": "f16"},
        # the down product of a long batch, rows scaled by their top-k weight
        {"name": "group_down", "op": "group", "A": 16384, "E": 16, "K": 2048, "N": 7168, "gated": False,
         "skew": 0.0, "row_weight": True, "dtype": "bf16"},
        # the gate and up products of the same batch, skewed over the experts
        {"name": "group_gate_up", "op": "group", "A": 16384, "E": 16, "K": 7168, "N": 4096, "gated": True,
         "skew": 0.6, "row_weight": False, "dtype": "bf16"},
        # the whole layer: one token through a small layer, where latency counts
        {"name": "few_one_small", "op": "few", "T": 1, "E": 16, "k": 2, "H": 1024, "I": 512, "weights": "bf16",
         "routing": "logits", "renorm": True},
        # one token through a large layer of 4-bit experts
        {"name": "few_one_large", "op": "few", "T": 1, "E": 64, "k": 8, "H": 7168, "I": 2048, "weights": "mx",
         "routing": "logits", "renorm": True},
        # a small batch, routed elsewhere; some of its experts live on other ranks
        {"name": "few_16_routed", "op": "few", "T": 16, "E": 64, "k": 6, "H": 2048, "I": 1408, "weights": "f16",
         "routing": "ids", "renorm": False},
        # the largest batch: several tokens for every 4-bit expert
        {"name": "few_64", "op": "few", "T": 64, "E": 32, "k": 4, "H": 4096, "I": 2048, "weights": "mx",
         "routing": "logits", "renorm": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["quant", "group", "few"])
    if op == "quant":
        H = 2 * _log_int(rng, 16, 8191)
        return {"op": op, "A": _log_int(rng, 1, min(65536, 16384 * 7168 // H)), "H": H,
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    if op == "group":
        gated = rng.random() < 0.5
        K = 32 * _log_int(rng, 2, 224)
        N = _log_int(rng, 32, 3584) * 2 - (0 if gated or rng.random() < 0.5 else 1)
        E = _log_int(rng, 1, max(1, min(128, 16 * 4096 * 7168 // (K * N))))
        A = _log_int(rng, 1, min(16384, 16384 * 4096 * 7168 // (K * N)))
        return {"op": op, "A": A, "E": E, "K": K, "N": N, "gated": gated, "skew": round(rng.uniform(0.0, 1.2), 2),
                "row_weight": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f16", "f32"])}
    H = 32 * _log_int(rng, 8, 224)
    intermediate = 32 * _log_int(rng, 2, 64)
    E = _log_int(rng, 4, max(4, min(256, 64 * 2048 * 7168 // (H * intermediate))))
    return {"op": op, "T": _log_int(rng, 1, 64), "E": E, "k": rng.randint(1, min(8, E)), "H": H, "I": intermediate,
            "weights": rng.choice(["mx", "bf16", "f16"]), "routing": rng.choice(["logits", "ids"]),
            "renorm": rng.random() < 0.5}


def _scale_bytes(n):
    return 2 * ((n + 63) // 64)


def work(case):
    if case["op"] == "quant":
        A, H = case["A"], case["H"]
        wide = A * H * _DTYPES[case["dtype"]].itemsize
        packed = A * (H // 2 + _scale_bytes(H))
        # the rows read, the 4-bit rows written and read back, the rows written
        return {"bytes": 2 * wide + 2 * packed, "flops": 4 * A * H}
    if case["op"] == "group":
        A, E, K, N = case["A"], case["E"], case["K"], case["N"]
        row = K // 2 + _scale_bytes(K)
        out = (N // 2 if case["gated"] else N) * _DTYPES[case["dtype"]].itemsize
        return {"bytes": A * (row + out + (4 if case["row_weight"] else 0)) + min(A, E) * N * row,
                "flops": 2 * A * N * K}
    T, E, k, H, n = case["T"], case["E"], case["k"], case["H"], case["I"]
    if case["weights"] == "mx":
        expert = 2 * n * (H // 2 + _scale_bytes(H)) + H * (n // 2 + _scale_bytes(n))
    else:
        expert = 3 * n * H * 2
    chosen = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token chooses, on average
    return {"bytes": chosen * expert + 2 * T * H * 2 + T * (4 * E if case["routing"] == "logits" else 8 * k),
            "flops": 2 * T * k * 3 * H * n}


# -------------------------------------------------------------------- inputs

def _e2m1_bytes(g, shape, device):
    """Packed 4-bit values as quantised normal values have them: nibble codes
    drawn by the quantiles of a normal variable of 2.3 units."""
    codes = []
    for i in range(256):
        z = 2.3 * NormalDist().inv_cdf((i + 0.5) / 256)
        code = min(range(8), key=lambda c: abs(_E2M1[c] - abs(z)))
        codes.append(code | (8 if z < 0 else 0))
    n = torch.tensor(codes, dtype=torch.uint8, device=device)
    pairs = (n[None, :] | (n[:, None] << 4)).reshape(-1)
    return pairs[torch.randint(0, 65536, shape, generator=g, device=device, dtype=torch.int32)]


def _mx_weights(g, shape, device):
    """4-bit weights [..., K] of variance about 1 / K: packed bytes and scales."""
    K = shape[-1]
    packed = _e2m1_bytes(g, shape[:-1] + (K // 2,), device)
    centre = 127 + round(math.log2(1.0 / (2.3 * math.sqrt(K))))
    scales = torch.randint(centre - 1, centre + 2, shape[:-1] + ((K + 63) // 64, 2), generator=g, device=device,
                           dtype=torch.uint8)
    return packed.view(torch.float4_e2m1fn_x2), scales.view(torch.float8_e8m0fnu)


def _rows(g, rows, n, dtype, device):
    """Activation rows: normal values, rows of different size, some channels larger."""
    x = torch.randn(rows, n, generator=g, device=device)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=device))
    x *= torch.where(torch.rand(n, generator=g, device=device) < 0.01, 8.0, 1.0)
    return x.to(dtype)


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"] == "quant":
        s["x"] = _rows(g, case["A"], case["H"], _DTYPES[case["dtype"]], device)
        return s
    if case["op"] == "group":
        A, E, K, N = case["A"], case["E"], case["K"], case["N"]
        # rows spread over the experts by a power law of their shuffled rank
        rank = torch.randperm(E, generator=g, device=device).double() + 1
        of_row = torch.multinomial(rank ** -case["skew"], A, replacement=True, generator=g)
        counts = torch.bincount(of_row, minlength=E)
        s["counts"] = counts.to(torch.int32)
        s["most"] = int(counts.max())
        packed, scales = _plain_pack(_rows(g, A, K, torch.bfloat16, device))
        s["tokens"], s["scales"] = packed, scales
        s["weight"], s["weight_scales"] = _mx_weights(g, (E, N, K), device)
        s["row_weight"] = torch.rand(A, 1, generator=g, device=device) if case["row_weight"] else None
        s["gated"], s["dtype"] = case["gated"], _DTYPES[case["dtype"]]
        return s
    T, E, k, H, n = case["T"], case["E"], case["k"], case["H"], case["I"]
    dtype = torch.bfloat16 if case["weights"] == "mx" else _DTYPES[case["weights"]]
    s["x"] = _rows(g, T, H, dtype, device)
    s["k"], s["renorm"] = k, case["renorm"]
    logits = 1.5 * torch.randn(T, E, generator=g, device=device)
    if case["routing"] == "logits":
        s["logits"] = logits
    else:
        top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
        away = torch.rand(T, k, generator=g, device=device) < 0.25  # experts of other ranks
        s["ids"] = torch.where(away, -1, ids[:, :k]).to(torch.int32).contiguous()
        s["weight"] = torch.softmax(top[:, :k], dim=1).contiguous()
    if case["weights"] == "mx":
        s["gate_up"], s["gate_up_scales"] = _mx_weights(g, (E, 2 * n, H), device)
        s["down"], s["down_scales"] = _mx_weights(g, (E, H, n), device)
    else:
        s["gate_up"] = torch.empty(E, 2 * n, H, dtype=dtype, device=device).normal_(0, H ** -0.5, generator=g)
        s["down"] = torch.empty(E, H, n, dtype=dtype, device=device).normal_(0, n ** -0.5, generator=g)
    return s


# --------------------------------------------------------------- plain forms

def _blocks(x):
    """[A, H] as [A, 2 ceil(H / 64), 32], zeros behind the row's end."""
    A, H = x.shape
    pairs = (H + 63) // 64
    return torch.nn.functional.pad(x, (0, 64 * pairs - H)).view(A, 2 * pairs, 32)


def _power(code):
    """2^(code - 127) by the bits of a float; the library's powers are not exact."""
    code = code.int()
    return (code.clamp(min=1) << 23).view(torch.float32) * torch.where(code == 0, 0.5, 1.0)


def _plain_quant(x):
    """(signed 4-bit codes [A, nb, 32], scale bytes [A, nb])."""
    b = _blocks(x.float())
    top = b.abs().amax(-1)
    exponent = torch.frexp(top)[1] - 3  # top = m 2^e with 0.5 <= m < 1
    scale = torch.where(top > 0, exponent + 127, 0).clamp(0, 254)
    q = b.abs() / _power(scale)[..., None]
    code = ((q > 0.25).to(torch.uint8) + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5.0))
    return code | (torch.signbit(b).to(torch.uint8) << 3), scale.to(torch.uint8)


def _plain_pack(x):
    A, H = x.shape
    code, scale = _plain_quant(x)
    code = code.view(A, -1)[:, :H]
    packed = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    return packed.view(torch.float4_e2m1fn_x2), scale.view(A, -1, 2).view(torch.float8_e8m0fnu)


def _plain_values(code):
    lut = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=code.device)
    return lut[code.int()]


def _plain_unpack(packed, scales):
    """Packed rows [..., K / 2] and scales [..., ceil(K / 64), 2] as values [..., K]; K a multiple of 32."""
    bytes_ = packed.view(torch.uint8)
    K = 2 * bytes_.shape[-1]
    v = _plain_values(torch.stack((bytes_ & 15, bytes_ >> 4), dim=-1)).view(bytes_.shape[:-1] + (K // 32, 32))
    s = _power(scales.view(torch.uint8).flatten(-2)[..., :K // 32])
    return (v * s[..., None]).flatten(-2)


def _silu(x):
    return x / (1 + torch.exp(-x))


def _plain_group(s):
    x = _plain_unpack(s["tokens"], s["scales"])
    w = _plain_unpack(s["weight"], s["weight_scales"])
    counts = s["counts"].long()
    E, A = counts.shape[0], x.shape[0]
    expert = torch.repeat_interleave(torch.arange(E, device=x.device), counts, output_size=A)
    at = torch.arange(A, device=x.device) - (torch.cumsum(counts, 0) - counts)[expert]
    rows = torch.zeros(E, s["most"], x.shape[1], device=x.device)
    rows[expert, at] = x
    y = torch.bmm(rows, w.transpose(1, 2).contiguous())[expert, at]
    if s["gated"]:
        gate, up = y.chunk(2, dim=1)
        y = _silu(gate) * up
    if s["row_weight"] is not None:
        y = y * s["row_weight"]
    return y.to(s["dtype"])


def _plain_few(s):
    x = s["x"].float()
    T, k = x.shape[0], s["k"]
    if "logits" in s:
        top, ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)
        p = torch.exp(top - top[:, :1])
        weight = p[:, :k] / (p[:, :k] if s["renorm"] else p).sum(1, keepdim=True)
        ids = ids[:, :k]
    else:
        ids, weight = s["ids"].long(), s["weight"]
    E = s["gate_up"].shape[0]
    experts = torch.arange(E, device=x.device)
    mix = torch.zeros(T, E + 1, device=x.device)  # the last column: experts that are not here
    mix.scatter_add_(1, torch.where(ids < 0, E, ids), weight)
    mix = mix[:, :E]
    if T * k < E:  # fewer choices than experts: only the chosen ones, a choice a time
        experts = ids.flatten().clamp(min=0)
        mix = torch.zeros(T, T * k, device=x.device)
        mix[torch.arange(T, device=x.device).repeat_interleave(k), torch.arange(T * k, device=x.device)] = (
            torch.where(ids < 0, 0.0, weight).flatten())
    pick = (lambda w: w[experts]) if experts.shape[0] < E else (lambda w: w)
    if "down_scales" in s:
        up = _plain_unpack(pick(s["gate_up"].view(torch.uint8)), pick(s["gate_up_scales"].view(torch.uint8)))
        down = _plain_unpack(pick(s["down"].view(torch.uint8)), pick(s["down_scales"].view(torch.uint8)))
    else:
        up, down = pick(s["gate_up"]).float(), pick(s["down"]).float()
    n = up.shape[1] // 2
    h = (up.flatten(0, 1) @ x.t().contiguous()).view(-1, 2, n, T)
    h = _silu(h[:, 0]) * h[:, 1]
    y = torch.bmm(down, h.contiguous())  # [experts, H, T]
    return (y * mix.t()[:, None, :]).sum(0).t().to(s["x"].dtype).contiguous()


def run(state):
    s = state
    if own:
        import moe_token_re_amd as moe

        if s["op"] == "quant":
            packed, scales = moe.mx_quantize(s["x"])
            return {"values": moe.mx_dequantize(packed, scales, dtype=s["x"].dtype), "scales": scales}
        if s["op"] == "group":
            return moe.mx_grouped_mm(s["tokens"], s["scales"], s["weight"], s["weight_scales"], s["counts"],
                                     gated=s["gated"], row_weight=s["row_weight"], dtype=s["dtype"])
        if "logits" in s:
            return moe.moe_few_tokens(s["x"], s["gate_up"], s["down"], router_logits=s["logits"], top_k=s["k"],
                                      renormalize=s["renorm"], gate_up_scales=s.get("gate_up_scales"),
                                      down_scales=s.get("down_scales"))
        return moe.moe_few_tokens(s["x"], s["gate_up"], s["down"], expert_ids=s["ids"], expert_weight=s["weight"],
                                  gate_up_scales=s.get("gate_up_scales"), down_scales=s.get("down_scales"))
    if s["op"] == "quant":
        x = s["x"]
        A, H = x.shape
        code, scale = _plain_quant(x)
        values = _plain_values(code) * _power(scale)[..., None]
        return {"values": values.view(A, -1)[:, :H].to(x.dtype).contiguous(),
                "scales": scale.view(A, -1, 2).view(torch.float8_e8m0fnu)}
    return _plain_group(s) if s["op"] == "group" else _plain_few(s)


# --------------------------------------------------------- the definitions in 64 bits

def _two_to(power):
    """2^power in 64 bits, -1022 <= power <= 1023."""
    return ((power.long() + 1023) << 52).view(torch.float64)


def _exact_unpack(packed, scales):
    """Sign, exponent and mantissa bits of the 4-bit values, in 64 bits."""
    c = packed.view(torch.uint8)
    c = torch.stack((c & 15, c >> 4), -1).flatten(-2).to(torch.int16)
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _two_to(e - 1))
    v = torch.where(c >= 8, -v, v)
    K = v.shape[-1]
    power = scales.view(torch.uint8).flatten(-2)[..., :K // 32].long() - 127
    return v * _two_to(power).repeat_interleave(32, dim=-1)


def _exact_quant(x):
    b = _blocks(x.double())
    top = b.abs().amax(-1)
    power = (top.view(torch.int64) >> 52) - 1023  # floor(log2(top)); far below the clamp where top is 0
    scale = _two_to((power - 2).clamp(-127, 127))[..., None]
    q = b / scale
    step = torch.where(q.abs() < 2, 0.5, torch.where(q.abs() < 4, 1.0, 2.0)).double()
    q = (torch.round(q / step) * step).clamp(-6, 6)
    A, H = x.shape
    return {"values": (q * scale).view(A, -1)[:, :H].contiguous(), "scales": scale.view(A, -1, 2).contiguous()}


def _exact_gate(y):
    gate, up = y.chunk(2, dim=-1)
    return gate * torch.sigmoid(gate) * up


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quant":
        return _exact_quant(s["x"])
    if s["op"] == "group":
        parts, at = [], 0
        for e, count in enumerate(s["counts"].tolist()):
            x = _exact_unpack(s["tokens"][at:at + count], s["scales"][at:at + count])
            y = x @ _exact_unpack(s["weight"][e], s["weight_scales"][e]).t()
            parts.append(_exact_gate(y) if s["gated"] else y)
            at += count
        y = torch.cat(parts)
        return y if s["row_weight"] is None else y * s["row_weight"].double()
    x, k = s["x"].double(), s["k"]
    if "logits" in s:
        p = torch.softmax(s["logits"].double(), dim=1)
        ids = torch.argsort(s["logits"].double(), dim=1, descending=True, stable=True)[:, :k]
        weight = p.gather(1, ids)
        if s["renorm"]:
            weight = weight / weight.sum(1, keepdim=True)
    else:
        ids, weight = s["ids"], s["weight"].double()
    y = torch.zeros_like(x)
    for e in range(s["gate_up"].shape[0]):
        token, choice = torch.nonzero(ids == e, as_tuple=True)
        if token.numel() == 0:
            continue
        if "down_scales" in s:
            up = _exact_unpack(s["gate_up"][e], s["gate_up_scales"][e])
            down = _exact_unpack(s["down"][e], s["down_scales"][e])
        else:
            up, down = s["gate_up"][e].double(), s["down"][e].double()
        out = _exact_gate(x[token] @ up.t()) @ down.t()
        y.index_add_(0, token, out * weight[token, choice][:, None])
    return y
