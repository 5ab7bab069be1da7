"""Cases of the operators around an expert layer, for measuring them: the
root-mean-square norm with the residual's addition and 8-bit rows as output
(and its gradient), the router's choice of experts (and its gradient), tokens
sorted by expert, and the experts' rows summed back by token with the choices'
weights (and its gradient).

`listed()` names the cases, `draw()` gives more of the same ranges,
`prepare()` makes a case's inputs on the GPU from a seed, and `run()` makes
one pass: through the library where `own` is true, else in plain torch
operations in 32 bits (64 where a value next to a rounding border decides).
`exact()` computes the same outputs in 64 bits from the operators'
definitions, and `work()` says what a pass has to move and compute.

Definitions, for rows of H values:
  norm      s = x + residual, rounded to x's type; y = w s / sqrt(mean(s^2) + eps). As int8 and e4m3 rows: scale =
            max |y| / 127 (or 448) of the row, values y / scale rounded to nearest even. As mx rows: blocks of 32
            values share 2^(e - 127), e - 127 = floor(log2(max |y|)) - 8.
  router    the top_k largest logits of a token, ties to the lowest expert; their softmax over all experts, or with
            renorm over the chosen ones. An expert of logit -inf is never chosen.
  permute   choice (t, j) goes to row rank(t, j) of a stable sort of all choices by their expert; choices of experts
            that are not here (id -1) come last, their rows are zeros and their index is -1 - row.
  combine   y[t] = sum over j of weight[t, j] rows[index[t, j]]; negative indices add nothing.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "int8": torch.int8,
           "fp8": torch.float8_e4m3fn}
_EPS = 1e-6


# --------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step's norm of one new token, with 8-bit rows for what follows
        {"name": "norm_one_token", "op": "norm", "T": 1, "H": 7168, "dtype": "bf16", "weight": "bf16",
         "residual": True, "quantize": "int8"},
        # rows of an odd length in half precision, microscaled; no residual
        {"name": "norm_odd_mx", "op": "norm", "T": 777, "H": 1059, "dtype": "f16", "weight": "f32",
         "residual": False, "quantize": "mxfp8"},
        # a long batch of the re-routing's own row count and length
        {"name": "norm_16384", "op": "norm", "T": 16384, "H": 7168, "dtype": "bf16", "weight": "bf16",
         "residual": True, "quantize": "fp8"},
        # a training step's backward pass through the norm and the residual
        {"name": "norm_backward", "op": "norm_backward", "T": 8192, "H": 4096, "dtype": "bf16", "weight": "f32",
         "residual": True},
        # the router of a decode batch
        {"name": "router_decode", "op": "router", "T": 16, "E": 64, "k": 6, "dtype": "f32", "renorm": True,
         "train": False},
        # the router of a training step, forward and backward
        {"name": "router_train", "op": "router", "T": 16384, "E": 256, "k": 8, "dtype": "f32", "renorm": False,
         "train": True},
        # one token's row, copied for each of its experts' ranks
        {"name": "permute_one_token", "op": "permute", "T": 1, "k": 8, "E": 64, "H": 7168, "tokens": "int8",
         "skew": 0.0, "away": 0.0},
        # ragged everything: odd rows, and experts that live on other ranks
        {"name": "permute_ragged", "op": "permute", "T": 1237, "k": 6, "E": 60, "H": 1409, "tokens": "f16",
         "skew": 1.0, "away": 0.25},
        # a long batch of microscaled 8-bit rows on its way to the ranks
        {"name": "permute_16384", "op": "permute", "T": 16384, "k": 8, "E": 256, "H": 7168, "tokens": "fp8",
         "skew": 0.6, "away": 0.0},
        # a decode batch's rows come back
        {"name": "combine_16", "op": "combine", "T": 16, "k": 8, "E": 64, "H": 7168, "dtype": "bf16",
         "weighted": True, "away": 0.0, "train": False},
        # a long batch's rows come back
        {"name": "combine_8192", "op": "combine", "T": 8192, "k": 8, "E": 256, "H": 7168, "dtype": "bf16",
         "weighted": True, "away": 0.0, "train": False},
        # a training step: forward and the gradients of the rows and the weights
        {"name": "combine_train", "op": "combine", "T": 8192, "k": 6, "E": 64, "H": 2048, "dtype": "bf16",
         "weighted": True, "away": 0.0, "train": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "router", "permute", "combine"])
    if op == "router":
        E = _log_int(rng, 4, 1024)
        return {"op": op, "T": _log_int(rng, 1, min(65536, 16384 * 256 // E)), "E": E,
                "k": rng.randint(1, min(16, E)), "dtype": rng.choice(["f32", "bf16", "f16"]),
                "renorm": rng.random() < 0.5, "train": rng.random() < 0.5}
    H = _log_int(rng, 32, 16383)
    if op in ("norm", "norm_backward"):
        case = {"op": op, "T": _log_int(rng, 1, min(65536, (16384 * 3584 if op == "norm" else 8192 * 4096) // H)),
                "H": H, "dtype": rng.choice(["bf16", "f16", "f32"]), "weight": "f32",
                "residual": rng.random() < 0.5}
        if op == "norm":
            case["quantize"] = rng.choice(["none", "int8", "fp8", "mxfp8"])
            if case["quantize"] == "int8":
                case["dtype"] = "bf16"  # whole numbers: every product of two bf16 values is exact in 32 bits
        if case["dtype"] == "bf16" and (case.get("quantize") == "int8" or rng.random() < 0.5):
            case["weight"] = "bf16"
        return case
    k = rng.randint(1, 16)
    E = _log_int(rng, max(2, k), 512)
    case = {"op": op, "k": k, "E": E, "H": H}
    away = rng.choice([0.0, 0.0, 0.25])
    if op == "permute":
        tokens = rng.choice(["int8", "fp8", "bf16", "f16"])
        row = H * _DTYPES[tokens].itemsize
        T = _log_int(rng, 1, max(1, min(65536, 900_000_000 // (row * (k + 1)))))
        return {**case, "T": T, "tokens": tokens, "skew": round(rng.uniform(0.0, 1.2), 2), "away": away}
    dtype, train = rng.choice(["bf16", "f16", "f32"]), rng.random() < 0.5
    row = H * _DTYPES[dtype].itemsize * (3 if train else 1)
    T = _log_int(rng, 1, max(1, min(65536, 900_000_000 // (row * (k + 1)))))
    return {**case, "T": T, "dtype": dtype, "weighted": rng.random() < 0.75, "away": away, "train": train}


def _mx_bytes(H):
    return 2 * ((H + 63) // 64)


def work(case):
    op, T = case["op"], case["T"]
    if op == "router":
        E, k, b = case["E"], case["k"], _DTYPES[case["dtype"]].itemsize
        one_way = T * E * b + 8 * T * k
        return {"bytes": one_way * 2 + 4 * T * k if case["train"] else one_way,
                "flops": T * E * (8 if case["train"] else 4)}
    H = case["H"]
    if op in ("norm", "norm_backward"):
        b, w = _DTYPES[case["dtype"]].itemsize, H * _DTYPES[case["weight"]].itemsize
        if op == "norm_backward":
            return {"bytes": T * H * b * (4 if case["residual"] else 3) + 2 * w, "flops": 11 * T * H}
        out = {"none": H * b, "int8": H + 4, "fp8": H + 4, "mxfp8": H + _mx_bytes(H)}[case["quantize"]]
        return {"bytes": T * (H * b * (3 if case["residual"] else 1) + out) + w, "flops": 6 * T * H}
    k = case["k"]
    if op == "permute":
        row = H * _DTYPES[case["tokens"]].itemsize
        row += {"int8": 4, "fp8": _mx_bytes(H)}.get(case["tokens"], 0)
        # ids and weights read, the tokens once, every row written, with its weight and index
        return {"bytes": 8 * T * k + T * row + T * k * (row + 8) + 4 * case["E"], "flops": T * k}
    row = H * _DTYPES[case["dtype"]].itemsize
    here = 1.0 - case["away"]
    index = T * k * (8 if case["weighted"] else 4)
    one_way = T * k * here * row + T * row + index
    if not case["train"]:
        return {"bytes": one_way, "flops": 2 * T * k * H}
    # the gradient read, the rows read for the weights', the rows' gradient written, and the weights'
    back = T * row + T * k * row + index
    if case["weighted"]:
        back += T * k * here * row + 4 * T * k
    return {"bytes": one_way + back, "flops": 5 * T * k * H}


# -------------------------------------------------------------------- inputs

def _rows(g, rows, n, dtype, device):
    """Activation rows: normal values, rows of different size, some channels larger."""
    x = torch.randn(rows, n, generator=g, device=device)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=device))
    x *= torch.where(torch.rand(n, generator=g, device=device) < 0.01, 8.0, 1.0)
    return x.to(dtype)


def _choices(g, case, device):
    """Distinct experts for each token, some more popular than others; with `away` some are not here."""
    T, k, E = case["T"], case["k"], case["E"]
    rank = torch.randperm(E, generator=g, device=device).float() + 1
    score = -case.get("skew", 0.0) * torch.log(rank) - torch.log(-torch.log(
        torch.rand(T, E, generator=g, device=device).clamp(1e-7, 1 - 1e-6)))
    ids = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :k]
    gone = torch.rand(T, k, generator=g, device=device) < case["away"]
    return torch.where(gone, -1, ids).to(torch.int32).contiguous()


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    op, T = case["op"], case["T"]
    s = {"op": op}
    if op in ("norm", "norm_backward"):
        H, dtype = case["H"], _DTYPES[case["dtype"]]
        s["x"] = _rows(g, T, H, dtype, device)
        s["weight"] = (1 + 0.2 * torch.randn(H, generator=g, device=device)).to(_DTYPES[case["weight"]])
        more = torch.randn(T, H, generator=g, device=device).to(dtype) if case["residual"] else None
        if op == "norm":
            s["residual"], s["quantize"] = more, None if case["quantize"] == "none" else case["quantize"]
        else:
            s["grad_residual"] = more
            s["grad"] = torch.randn(T, H, generator=g, device=device).to(dtype)
        return s
    k, E = case["k"], case["E"]
    if op == "router":
        s["logits"] = (1.5 * torch.randn(T, E, generator=g, device=device)).to(_DTYPES[case["dtype"]])
        s["k"], s["renorm"] = k, case["renorm"]
        s["grad"] = torch.randn(T, k, generator=g, device=device) if case["train"] else None
        return s
    ids = _choices(g, case, device)
    weight = torch.softmax(torch.randn(T, k, generator=g, device=device), dim=1).contiguous()
    if op == "permute":
        s["ids"], s["weight"], s["E"], s["scales"] = ids, weight, E, None
        H = case["H"]
        if case["tokens"] == "int8":
            s["tokens"] = torch.randint(-127, 128, (T, H), generator=g, device=device, dtype=torch.int8)
            s["scales"] = torch.rand(T, generator=g, device=device) * 0.1
        elif case["tokens"] == "fp8":
            s["tokens"] = (60 * torch.randn(T, H, generator=g, device=device)).clamp(-448, 448).to(torch.float8_e4m3fn)
            s["scales"] = torch.randint(110, 130, (T, (H + 63) // 64, 2), generator=g, device=device,
                                        dtype=torch.uint8).view(torch.float8_e8m0fnu)
        else:
            s["tokens"] = _rows(g, T, H, _DTYPES[case["tokens"]], device)
        return s
    dtype = _DTYPES[case["dtype"]]
    s["index"] = _plain_plan(ids, E)[1]
    s["rows"] = _rows(g, T * k, case["H"], dtype, device)
    s["weight"] = weight if case["weighted"] else None
    s["grad"] = torch.randn(T, case["H"], generator=g, device=device).to(dtype) if case["train"] else None
    return s


# --------------------------------------------------------------- plain forms

def _power(code):
    """2^(code - 127) by the bits of a float; the library's powers are not exact."""
    code = code.int()
    return (code.clamp(min=1) << 23).view(torch.float32) * torch.where(code == 0, 0.5, 1.0)


def _plain_norm(s):
    x, q = s["x"], s["quantize"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    out = {} if s["residual"] is None else {"sum": h}
    if q is None:
        f = h.float()
        y = f * torch.rsqrt((f * f).mean(dim=1, keepdim=True) + _EPS) * s["weight"].float()
        return {**out, "y": y.to(x.dtype)}
    # 64 bits: a rounding to 8 bits is decided by how a value compares with a border
    f = h.double()
    p = f * s["weight"].double()
    r = 1 / torch.sqrt((f * f).mean(dim=1, keepdim=True) + _EPS)
    if q != "mxfp8":
        most = 127 if q == "int8" else 448
        top = p.abs().amax(dim=1, keepdim=True)
        v = p * most / torch.where(top > 0, top, 1.0)
        v = torch.round(v).to(torch.int8) if q == "int8" else v.float().clamp(-448, 448).to(torch.float8_e4m3fn)
        return {**out, "y": v, "scales": (r * top / most).float()[:, 0]}
    T, H = x.shape
    nb = 2 * ((H + 63) // 64)
    b = torch.nn.functional.pad(p * r, (0, 32 * nb - H)).view(T, nb, 32)
    top = b.abs().amax(-1)
    code = torch.where(top > 0, torch.frexp(top)[1] - 9 + 127, 0).clamp(0, 254)  # top = m 2^e with 0.5 <= m < 1
    v = (b / _power(code).double()[..., None]).float().clamp(-448, 448).view(T, -1)[:, :H].to(torch.float8_e4m3fn)
    return {**out, "y": v.contiguous(), "scales": code.to(torch.uint8).view(T, -1, 2).view(torch.float8_e8m0fnu)}


def _plain_norm_backward(s):
    x, g, w = s["x"].float(), s["grad"].float(), s["weight"].float()
    r = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + _EPS)
    n = x * r
    gw = g * w
    dx = r * (gw - n * (gw * n).mean(dim=1, keepdim=True))
    if s["grad_residual"] is not None:
        dx = dx + s["grad_residual"].float()
    return {"grad_x": dx.to(s["x"].dtype), "grad_weight": (g * n).sum(0).to(s["weight"].dtype)}


def _plain_router(s):
    x, k = s["logits"].float(), s["k"]
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    p = torch.exp(top - top[:, :1])
    weight = p[:, :k] / (p[:, :k] if s["renorm"] else p).sum(1, keepdim=True)
    ids = ids[:, :k]
    out = {"weight": weight, "ids": ids.to(torch.int32)}
    if s["grad"] is not None:
        share = weight * s["grad"]
        mean = share.sum(1, keepdim=True)
        if s["renorm"]:
            d = torch.zeros_like(x).scatter(1, ids, share - weight * mean)
        else:
            e = torch.exp(x - top[:, :1])
            d = (-mean * e / p.sum(1, keepdim=True)).scatter_add(1, ids, share)
        out["grad_logits"] = d.to(s["logits"].dtype)
    return out


def _plain_plan(ids, E):
    """(choice of each row [T k], index [T, k], rows of each expert [E])"""
    flat = torch.where((ids < 0) | (ids >= E), E, ids).flatten().long()
    order = torch.sort(flat, stable=True)[1]
    at = torch.empty_like(order)
    at[order] = torch.arange(order.numel(), device=ids.device)
    index = torch.where(flat == E, -1 - at, at).to(torch.int32).view(ids.shape)
    num = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    num.scatter_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    return order, index, num[:E]


def _plain_permute(s):
    order, index, num = _plain_plan(s["ids"], s["E"])
    k = s["ids"].shape[1]
    here = index.flatten()[order] >= 0

    def move(v, at):
        b = v.contiguous().view(torch.uint8) if v.dtype.itemsize == 1 else v
        b = b[at]
        return torch.where(here.view(-1, *[1] * (b.dim() - 1)), b, torch.zeros((), dtype=b.dtype,
                                                                              device=b.device)).view(v.dtype)

    out = {"tokens": move(s["tokens"], order // k), "index": index, "num": num,
           "weight": move(s["weight"].view(-1, 1), order)}
    if s["scales"] is not None:
        out["scales"] = move(s["scales"], order // k)
    return out


def _plain_combine(s):
    rows, index, weight = s["rows"], s["index"], s["weight"]
    T, k = index.shape
    here = index >= 0
    at = torch.where(here, index, -1 - index).long()
    y = torch.zeros(T, rows.shape[1], device=rows.device)
    for j in range(k):
        v = rows[at[:, j]].float()
        if weight is not None:
            v = v * weight[:, j:j + 1]
        y += torch.where(here[:, j:j + 1], v, 0.0)
    out = {"y": y.to(rows.dtype)}
    if s["grad"] is not None:
        g = s["grad"].float()
        d = torch.empty_like(rows)
        dw = torch.zeros(T, k, device=rows.device)
        for j in range(k):
            v = g if weight is None else g * weight[:, j:j + 1]
            d[at[:, j]] = torch.where(here[:, j:j + 1], v, 0.0).to(rows.dtype)
            if weight is not None:
                dw[:, j] = torch.where(here[:, j], (g * rows[at[:, j]].float()).sum(1), 0.0)
        out["grad_rows"] = d
        if weight is not None:
            out["grad_weight"] = dw
    return out


def _own(s):
    import moe_token_re_amd as moe

    op = s["op"]
    if op == "norm":
        y, scales, total = moe.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=_EPS,
                                        quantize=s["quantize"])
        out = {"y": y}
        if scales is not None:
            out["scales"] = scales
        if total is not None:
            out["sum"] = total
        return out
    if op == "norm_backward":
        dx, dw = moe.rms_norm_backward(s["grad"], s["x"], s["weight"], grad_residual=s["grad_residual"], eps=_EPS)
        return {"grad_x": dx, "grad_weight": dw}
    if op == "router":
        weight, ids = moe.moe_router_top_k(s["logits"], s["k"], renormalize=s["renorm"])
        out = {"weight": weight, "ids": ids}
        if s["grad"] is not None:
            out["grad_logits"] = moe.moe_router_top_k_backward(s["grad"], s["logits"], weight, ids,
                                                               renormalize=s["renorm"])
        return out
    if op == "permute":
        tokens, scales, index, num, weight = moe.moe_token_permute(
            s["tokens"], s["ids"], s["E"], per_token_scales=s["scales"], expert_weight=s["weight"])
        out = {"tokens": tokens, "index": index, "num": num, "weight": weight}
        if scales is not None:
            out["scales"] = scales
        return out
    out = {"y": moe.moe_token_unpermute(s["rows"], s["index"], expert_weight=s["weight"])}
    if s["grad"] is not None:
        out["grad_rows"], dw = moe.moe_token_unpermute_backward(s["grad"], s["rows"], s["index"],
                                                                expert_weight=s["weight"])
        if dw is not None:
            out["grad_weight"] = dw
    return out


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "router": _plain_router,
            "permute": _plain_permute, "combine": _plain_combine}[state["op"]](state)


# --------------------------------------------------------- the definitions in 64 bits

def _exact_e4m3(v):
    """The nearest e4m3 values, ties to even, beyond 448 to 448, by their step: 2^-9 up to 2^-6, an eighth above."""
    power = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    power = power - (torch.exp2(power) > v.abs().clamp(min=2.0 ** -6)).double()
    step = torch.exp2(power - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_norm(s):
    x = s["x"].double()
    h = x
    if s["residual"] is not None:
        h = (x + s["residual"].double()).to(s["x"].dtype).double()
    out = {} if s["residual"] is None else {"sum": h}
    scale = torch.sqrt(h.square().sum(1) / h.shape[1] + _EPS)
    y = (h / scale[:, None]) * s["weight"].double()
    q = s["quantize"]
    if q is None:
        return {**out, "y": y}
    if q == "mxfp8":
        values, codes = [], []
        for at in range(0, y.shape[1], 32):
            b = y[:, at:at + 32]
            power = ((b.abs().amax(1).view(torch.int64) >> 52) - 1023 - 8).clamp(-127, 127)  # floor(log2) of the largest
            unit = ((power + 1023) << 52).view(torch.float64)
            values.append(_exact_e4m3(b / unit[:, None]))
            codes.append(unit)
        if len(codes) % 2:
            codes.append(torch.full_like(codes[0], 2.0 ** -127))
        return {**out, "y": torch.cat(values, 1), "scales": torch.stack(codes, 1).view(y.shape[0], -1, 2)}
    most = 127 if q == "int8" else 448
    unit = y.abs().amax(1) / most
    # y / unit without the norm, which cancels: quotients halfway between two values are so exactly
    p = h * s["weight"].double()
    y = None if q == "int8" else _exact_e4m3(most * p / p.abs().amax(1).clamp(min=1e-300)[:, None])
    return {**out, "y": y, "scales": unit}


def _exact_norm_backward(s):
    x, g, w = s["x"].double(), s["grad"].double(), s["weight"].double()
    m = x.square().sum(1, keepdim=True) / x.shape[1] + _EPS
    # d/dx of w x m^(-1/2): the second term by the chain through m
    dot = (g * w * x).sum(1, keepdim=True)
    dx = g * w / torch.sqrt(m) - x * dot / (x.shape[1] * m * torch.sqrt(m))
    if s["grad_residual"] is not None:
        dx = dx + s["grad_residual"].double()
    return {"grad_x": dx, "grad_weight": (g * x / torch.sqrt(m)).sum(0)}


def _exact_router(s):
    x, k = s["logits"].double(), s["k"]
    ids = torch.argsort(x, dim=1, descending=True, stable=True)[:, :k]
    chosen = torch.zeros_like(x, dtype=torch.bool).scatter_(1, ids, True)
    p = torch.softmax(x.masked_fill(~chosen, -math.inf) if s["renorm"] else x, dim=1)
    weight = p.gather(1, ids)
    out = {"weight": weight, "ids": None}
    if s["grad"] is not None:
        g = torch.zeros_like(x).scatter_(1, ids, s["grad"].double())  # of every p, 0 where none is returned
        out["grad_logits"] = p * (g - (p * g).sum(1, keepdim=True))
    return out


def _exact_rows(ids, E):
    """Row of every choice, counted expert by expert, those of no expert here last."""
    flat = ids.flatten().long()
    row = torch.full_like(flat, -1)
    at = 0
    for e in list(range(E)) + [None]:
        mine = torch.nonzero(flat == e if e is not None else (flat < 0) | (flat >= E))[:, 0]
        row[mine] = at + torch.arange(mine.numel(), device=ids.device)
        at += mine.numel()
    return row.view(ids.shape)


def _exact_permute(s):
    ids, tokens = s["ids"], s["tokens"]
    T, k = ids.shape
    row = _exact_rows(ids, s["E"])
    here = ((ids >= 0) & (ids < s["E"]))[..., None]

    def place(v, dims):
        if v.dtype == torch.int8:
            return None
        out = torch.empty((T * k,) + tuple(v.shape[1:] if dims else (1,)), dtype=torch.float64, device=v.device)
        for j in range(k):
            r = v.double() if dims else v[:, j:j + 1].double()
            out[row[:, j]] = torch.where(here[:, j].view(-1, *[1] * (r.dim() - 1)), r, 0.0)
        return out

    out = {"tokens": place(tokens, True), "index": None, "num": None, "weight": place(s["weight"], False)}
    if s["scales"] is not None:
        # a scale byte of 0 stands for 2^-127
        v = s["scales"].float() if s["scales"].dtype == torch.float32 else s["scales"].view(torch.uint8)
        v = place(v, True)
        out["scales"] = v if s["scales"].dtype == torch.float32 else torch.exp2(v - 127)
    return out


def _exact_combine(s):
    rows, index = s["rows"].double(), s["index"].long()
    T, k = index.shape
    w = torch.ones(T, k, dtype=torch.float64, device=rows.device) if s["weight"] is None else s["weight"].double()
    w = torch.where(index < 0, 0.0, w)
    at = torch.where(index < 0, -1 - index, index)
    y = torch.empty(T, rows.shape[1], dtype=torch.float64, device=rows.device)
    for t in range(0, T, 256):
        y[t:t + 256] = (rows[at[t:t + 256]] * w[t:t + 256, :, None]).sum(1)
    out = {"y": y}
    if s["grad"] is not None:
        g = s["grad"].double()
        d = torch.empty_like(rows)
        dw = torch.empty_like(w)
        for t in range(0, T, 256):
            one = g[t:t + 256, None, :]
            d[at[t:t + 256].flatten()] = (one * w[t:t + 256, :, None]).flatten(0, 1)
            dw[t:t + 256] = (one * rows[at[t:t + 256]]).sum(2)
        out["grad_rows"] = d
        if s["weight"] is not None:
            out["grad_weight"] = torch.where(index < 0, 0.0, dw)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "router": _exact_router,
            "permute": _exact_permute, "combine": _exact_combine}[case["op"]](s)
