"""fp64 oracle of the expert-layer operators, from their definitions (numpy, no GPU code).

Matrices in 8-bit floating point are pairs (codes as values, scale exponents); routing uses
plain sorting; gradients are the formulas' own (checked against differences in the tests).
"""

import numpy as np


def e4m3(v):
    """v rounded to nearest even in e4m3 (|v| <= 448; NaN and infinities become NaN)."""
    v = np.asarray(v, np.float64)
    bad = ~np.isfinite(v)
    x = np.where(bad, 0.0, v)
    _, q = np.frexp(np.abs(x))                       # |x| in [2^(q-1), 2^q)
    step = np.exp2(np.maximum(q - 1, -6) - 3.0)      # three bits after the leading one
    return np.where(bad, np.nan, np.rint(x / step) * step)


def block_shape(blocks):
    return {"row": (1, 128), "col": (128, 1), "tile": (128, 128)}[blocks]


def quantize(x, blocks):
    """(codes as values, scale bytes) of a matrix."""
    x = np.asarray(x, np.float64)
    br, bc = block_shape(blocks)
    R, C = x.shape
    nr, nc = -(-R // br), -(-C // bc)
    codes, scales = np.zeros((R, C)), np.zeros((nr, nc), np.int64)
    for i in range(nr):
        for j in range(nc):
            b = x[i * br:(i + 1) * br, j * bc:(j + 1) * bc]
            a = np.abs(b[np.isfinite(b)]).max(initial=0.0)
            e = -127
            if a > 0:
                e = max(-127, int(np.ceil(np.log2(a / 448.0))) - 1)
                while a > 448.0 * 2.0 ** e:
                    e += 1
            codes[i * br:(i + 1) * br, j * bc:(j + 1) * bc] = e4m3(b * 2.0 ** -e)
            scales[i, j] = e + 127
    return codes, scales


def dequantize(codes, scales, blocks):
    codes = np.asarray(codes, np.float64)
    br, bc = block_shape(blocks)
    f = np.exp2(np.asarray(scales, np.float64) - 127.0)
    f = np.repeat(np.repeat(f, br, 0), bc, 1)[:codes.shape[0], :codes.shape[1]]
    return codes * f


def product(a, b, form, offsets=None):
    """a: values; b: values (list of one matrix per group for nt and nn)."""
    off = [0, a.shape[0]] if offsets is None else list(offsets)
    if form == "tn":
        return np.stack([a[lo:hi].T @ b[lo:hi] for lo, hi in zip(off[:-1], off[1:])])
    cols = b[0].shape[0] if form == "nt" else b[0].shape[1]
    y = np.zeros((a.shape[0], cols))
    for g, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        y[lo:hi] = a[lo:hi] @ (b[g].T if form == "nt" else b[g])
    return y


def scores(logits, score):
    x = np.asarray(logits, np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    top = x.max(1, keepdims=True)
    e = np.exp(x - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(1, keepdims=True)
    return e / np.where(total == 0, 1.0, total)


def route(logits, top_k, score="softmax", bias=None, groups=1, keep_groups=None,
          group_score="top2", renorm=True, scale=1.0):
    """(weights, ids, decided): decided[t] is False where the choice of token t rests on
    keys that differ by less than 1e-5 of their size without being equal."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    s = scores(x, score)
    key = x if bias is None and groups == 1 else s if bias is None else s + np.asarray(bias, np.float64)
    key = np.where(x == -np.inf, -np.inf, key)
    keep = groups if keep_groups is None else keep_groups
    w, ids, decided = np.zeros((T, top_k)), np.full((T, top_k), -1), np.ones(T, bool)

    def near(a, b):
        return a != b and np.isfinite(a) and np.isfinite(b) and abs(a - b) < 1e-5 * (abs(a) + abs(b)) + 1e-7

    for t in range(T):
        k = key[t].copy()
        if groups > 1:
            run = []
            for g in range(groups):
                best = sorted([v for v in k.reshape(groups, -1)[g] if v > -np.inf], reverse=True)
                n = 1 if group_score == "max" else 2
                run.append(sum(best[:n]) if best else -np.inf)
            order = sorted(range(groups), key=lambda g: (-run[g], g))
            if keep < groups and near(run[order[keep - 1]], run[order[keep]]):
                decided[t] = False
            for g in order[keep:]:
                k.reshape(groups, -1)[g] = -np.inf
        order = sorted(range(E), key=lambda e: (-k[e], e))
        if any(near(k[a], k[b]) for a, b in zip(order[:top_k], order[1:top_k + 1])):
            decided[t] = False
        chosen = [e for e in order[:top_k] if k[e] > -np.inf]
        c = np.array([s[t, e] for e in chosen])
        if renorm:
            c = c / (c.sum() + 1e-20)
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = scale * c
    return w, ids, decided


def route_backward(logits, ids, dweights, score="softmax", renorm=True, scale=1.0):
    s = scores(logits, score)
    T, E = s.shape
    dl = np.zeros((T, E))
    for t in range(T):
        on = [(j, e) for j, e in enumerate(ids[t]) if e >= 0]
        if not on:
            continue
        e = np.array([v for _, v in on])
        g = scale * np.array([dweights[t, j] for j, _ in on], np.float64)
        c = s[t, e]
        if renorm:
            total = c.sum() + 1e-20
            g = (g - (g * c / total).sum()) / total
        ds = np.zeros(E)
        ds[e] = g
        dl[t] = ds * s[t] * (1 - s[t]) if score == "sigmoid" else s[t] * (ds - (ds * s[t]).sum())
    return dl


def plan(ids, experts, n_slots):
    """(counts, offsets, row_of, slot_of)."""
    flat = np.asarray(ids).reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(experts)], np.int64)
    offsets = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    row_of, slot_of = np.full(flat.size, -1), np.full(n_slots, -1)
    at = offsets[:-1].copy()
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            row_of[i], slot_of[at[e]] = at[e], i
            at[e] += 1
    return counts, offsets, row_of.reshape(np.shape(ids)), slot_of


def combine(z, row_of, weights=None):
    z = np.asarray(z, np.float64)
    T, k = row_of.shape
    y = np.zeros((T, z.shape[1]))
    for t in range(T):
        for j in range(k):
            if row_of[t, j] >= 0:
                y[t] += (1.0 if weights is None else float(weights[t, j])) * z[row_of[t, j]]
    return y


def combine_backward(dy, z, row_of, weights=None):
    dy, z = np.asarray(dy, np.float64), np.asarray(z, np.float64)
    T, k = row_of.shape
    dz, dw = np.zeros_like(z), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if row_of[t, j] >= 0:
                dz[row_of[t, j]] = (1.0 if weights is None else float(weights[t, j])) * dy[t]
                dw[t, j] = dy[t] @ z[row_of[t, j]]
    return dz, dw
