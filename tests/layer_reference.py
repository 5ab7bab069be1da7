"""The operators around an expert layer in 64 bits, from their definitions, on
the CPU: what the GPU tests compare with. Nothing here is shared with the
library."""
import torch

E4M3_MAX, E2M1_MAX = 448.0, 6.0


def e4m3(v):
    """The nearest e4m3 values, ties to even, saturating: steps of 2^-9 up to 2^-6, an eighth of the power above."""
    a = v.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(a)) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def e2m1(v):
    """The nearest e2m1 values, ties to even, saturating: steps of 0.5 up to 2, 1 up to 4, 2 up to 6."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(v.dtype)
    return (torch.round(v / step) * step).clamp(-E2M1_MAX, E2M1_MAX)


def norm_sum(x, residual):
    """What is normalised, as it is stored: rounded once from the exact sum (two 32-bit steps do not differ from one:
    a sum of two 11- or 8-bit numbers that does not fit 24 bits lies far from a halfway point of the type)."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm(s, weight, eps):
    """(y, p): the norm of rows, and their products with the weight, which y is a positive multiple of."""
    s, w = s.double(), weight.double()
    return s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps) * w, s * w


def norm_backward(grad, x, weight, eps, grad_residual=None):
    g, x, w = grad.double(), x.double(), weight.double()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    n = x * r
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    if grad_residual is not None:
        dx = dx + grad_residual.double()
    return dx, (g * n).flatten(0, -2).sum(0)


def router(logits, k, renormalize):
    """(weight, ids) by a loop over tokens."""
    T, E = logits.shape
    weight = torch.zeros(T, k, dtype=torch.float64)
    ids = torch.full((T, k), -1, dtype=torch.int32)
    for t in range(T):
        row = logits[t].double()
        order = sorted((e for e in range(E) if row[e] != float("-inf")),
                       key=lambda e: (0 if torch.isnan(row[e]) else 1, -float(row[e]) if row[e] == row[e] else 0.0, e))
        chosen = order[:k]
        if not chosen:
            continue
        over = chosen if renormalize else order
        p = torch.softmax(row[over], 0)
        for j, e in enumerate(chosen):
            ids[t, j] = e
            weight[t, j] = p[over.index(e)]
    return weight, ids


def router_backward(grad, logits, ids, renormalize):
    T, E = logits.shape
    out = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        chosen = [int(e) for e in ids[t] if 0 <= e < E]
        row = logits[t].double()
        over = chosen if renormalize else [e for e in range(E) if row[e] != float("-inf")]
        if not over:
            continue
        p = torch.softmax(row[over], 0)
        g = torch.zeros(E, dtype=torch.float64)
        for j, e in enumerate(int(e) for e in ids[t]):
            if 0 <= e < E:
                g[e] = grad[t, j].double()
        g = g[over]
        out[t, over] = p * (g - (p * g).sum())
    return out


def plan(ids, E):
    """(row of every choice [T, k], those below 0: -1 - row, rows of each expert) by counting one choice at a time."""
    T, k = ids.shape
    flat = [int(e) if 0 <= e < E else E for e in ids.flatten().tolist()]
    count = [0] * (E + 1)
    for e in flat:
        count[e] += 1
    at, first = [], 0
    for c in count:
        at.append(first)
        first += c
    row = []
    for e in flat:
        row.append(at[e] if e < E else -1 - at[e])
        at[e] += 1
    return torch.tensor(row, dtype=torch.int32).view(T, k), torch.tensor(count[:E], dtype=torch.int32)


def place(v, index):
    """Rows v [T, ...] (or, of one value a choice, [T, k]) at the rows of their choices, zeros for those below 0."""
    T, k = index.shape
    out = torch.zeros((T * k,) + tuple(v.shape[1:]), dtype=v.dtype)
    for j in range(k):
        i = index[:, j].long()
        out[i[i >= 0]] = v[i >= 0]
    return out


def combine(rows, index, weight=None):
    """(y, the sum of the terms' sizes, which rounding errors go by)"""
    T, k = index.shape
    y = torch.zeros(T, rows.shape[1], dtype=torch.float64)
    size = torch.zeros_like(y)
    for j in range(k):
        i = index[:, j].long()
        here = (i >= 0) & (i < rows.shape[0])
        v = rows[i[here]].double()
        if weight is not None:
            v = v * weight[here, j:j + 1].double()
        y[here] += v
        size[here] += v.abs()
    return y, size


def combine_backward(grad, rows, index, weight):
    """(grad_rows, grad_weight, the sum of its terms' sizes)"""
    T, k = index.shape
    d = torch.zeros(rows.shape, dtype=torch.float64)
    dw = torch.zeros(T, k, dtype=torch.float64)
    size = torch.zeros(T, k, dtype=torch.float64)
    for j in range(k):
        i = index[:, j].long()
        here = (i >= 0) & (i < rows.shape[0])
        g = grad[here].double()
        d[i[here]] = g if weight is None else g * weight[here, j:j + 1].double()
        p = g * rows[i[here]].double()
        dw[here, j], size[here, j] = p.sum(1), p.abs().sum(1)
    return d, dw, size
