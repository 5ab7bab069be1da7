"""The experts' operators in 64 bits on the CPU, straight from their
definitions, with bounds on what a kernel's rounding may add.

Bounds. Sums kept in 32 bits: |error| <= (n + 8) 2^-23 sum |x w| for n terms in
any order (each addition off by at most 2^-24 of a partial sum, doubled).
silu(g) = g / (1 + exp(-g)) in 32 bits: a relative (8 + |g|) 2^-22, as the
exponential's argument is off by |g| 2^-23 or so; its slope is at most 1.1.
A result rounded to type t: relative torch.finfo(t).eps / 2, and half its
smallest subnormal."""
import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def blocks(x):
    A, H = x.shape
    pairs = (H + 63) // 64
    b = np.zeros((A, 64 * pairs))
    b[:, :H] = x
    return b.reshape(A, 2 * pairs, 32)


def quantize(x):
    """x [A, H] float64 (values of some float type): (packed uint8, scales uint8)."""
    A, H = x.shape
    b = blocks(x)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    with np.errstate(all="ignore"):
        exponent = np.where(top > 0, np.frexp(np.where(np.isfinite(top), top, 1))[1] - 1, -400)
    s = np.clip(exponent - 2 + 127, 0, 254)
    q = np.abs(np.where(bad[..., None], 0, b)) * np.exp2(127.0 - s)[..., None]
    # nearest value; a tie goes to the even code
    d = np.abs(np.minimum(q, 6)[..., None] - E2M1)
    least = d.min(-1, keepdims=True)
    code = np.where(d == least, np.arange(8) % 2 * 8 + np.arange(8), 99).min(-1) % 8
    code = code | (np.signbit(b).astype(np.int64) << 3)
    code = np.where(bad[..., None], 0, code).reshape(A, -1)[:, :H].astype(np.uint8)
    s = np.where(bad, 255, s).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), s.reshape(A, -1, 2)


def unpack(packed, scales):
    """Packed bytes [..., K/2] and scale bytes [..., ceil(K/64), 2] as float64 [..., K]."""
    packed, scales = np.asarray(packed), np.asarray(scales)
    c = np.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[:-1] + (-1,))
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    K = v.shape[-1]
    s = scales.reshape(scales.shape[:-2] + (-1,)).astype(np.float64)
    f = np.where(s == 255, np.nan, np.exp2(s - 127))
    return v * np.repeat(f, 32, axis=-1)[..., :K]


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def gate(x, w):
    """silu(x Wg) * (x Wu) for w [2 I, K], and its bound."""
    n, K = w.shape[0] // 2, w.shape[1]
    g, u = x @ w[:n].T, x @ w[n:].T
    f = (K + 8) * 2.0 ** -23
    eg, eu = f * (np.abs(x) @ np.abs(w[:n]).T), f * (np.abs(x) @ np.abs(w[n:]).T)
    y = silu(g) * u
    slack = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + np.abs(y) * (8 + np.abs(g)) * 2.0 ** -22
    return y, slack


def rounding(y, slack, dtype):
    """The bound once the result is rounded to dtype."""
    fi = torch.finfo(dtype)
    half = fi.eps / 2
    return slack + (np.abs(y) + slack) * half + fi.tiny * half


def grouped(x, w, counts, gated, row_weight, dtype):
    """x [A, K], w [E, N, K] float64; (y, bound)."""
    ys, es, at = [], [], 0
    for e, c in enumerate(counts):
        xe = x[at:at + c]
        if gated:
            y, err = gate(xe, w[e])
        else:
            y = xe @ w[e].T
            err = (x.shape[1] + 8) * 2.0 ** -23 * (np.abs(xe) @ np.abs(w[e]).T)
        ys.append(y)
        es.append(err)
        at += c
    y, err = np.concatenate(ys), np.concatenate(es)
    if row_weight is not None:
        rw = row_weight.reshape(-1, 1).astype(np.float64)
        y, err = y * rw, err * np.abs(rw) + np.abs(y * rw) * 2.0 ** -23
    return y, rounding(y, err, dtype)


def route(logits, k, renormalize):
    """float64 logits [T, E]: (ids [T, k], -1 where there is none, weights)."""
    T, E = logits.shape
    ids, w = np.full((T, k), -1), np.zeros((T, k))
    for t in range(T):
        row = logits[t]
        key = np.where(np.isnan(row), np.inf, row)
        first = np.where(np.isnan(row), 0, 1)  # NaN before +inf
        order = np.lexsort((np.arange(E), first, -key))[:k]
        order = [e for e in order if not row[e] == -np.inf]
        if not order:
            continue
        with np.errstate(all="ignore"):
            p = np.exp(row - row[order[0]])
            total = p[order].sum() if renormalize else p.sum()
            for j, e in enumerate(order):
                ids[t, j], w[t, j] = e, p[e] / total
    return ids, w


def few_tokens(x, gate_up, down, ids, weights, dtype):
    """x [T, H], gate_up [E, 2I, H], down [E, H, I] float64; ids outside the
    experts choose nothing. (y, bound); h is rounded once to dtype."""
    T, E = x.shape[0], gate_up.shape[0]
    y, err = np.zeros((T, down.shape[1])), np.zeros((T, down.shape[1]))
    I = down.shape[2]
    used = 0
    for t in range(T):
        for e in sorted(set(int(i) for i in ids[t] if 0 <= i < E)):
            p = float(sum(w for i, w in zip(ids[t], weights[t]) if i == e))
            h, eh = gate(x[t:t + 1], gate_up[e])
            h, eh = h * p, np.abs(p) * eh + np.abs(h * p) * 2.0 ** -20  # the weight's own 32 bits
            eh = rounding(h, eh, dtype)
            y[t] += (h @ down[e].T)[0]
            err[t] += ((eh + ((I * len(ids[t])) + 8) * 2.0 ** -23 * (np.abs(h) + eh)) @ np.abs(down[e]).T)[0]
            used += 1
    return y, rounding(y, err, dtype)


def assert_close(got, want, bound, what):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    off = np.abs(got - want) - bound
    off = off[~np.isnan(want)]
    assert off.size == 0 or off.max() <= 0, f"{what}: {off.max()} beyond the bound at {np.argmax(off)}"
