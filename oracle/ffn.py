"""fp64 oracle of the feed-forward operators, from their definitions (numpy, no GPU code)."""

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(x, name):
    x = np.asarray(x, np.float64)
    if name == "silu":
        with np.errstate(over="ignore"):
            return x / (1.0 + np.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1.0 + _erf(x / math.sqrt(2.0)))
    return 0.5 * x * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))


def slope(x, name):
    x = np.asarray(x, np.float64)
    if name == "silu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-x))
        return s * (1.0 + x * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + _erf(x / math.sqrt(2.0))) + x * np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = np.tanh(c * (x + 0.044715 * x ** 3))
    return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * x * x)


def runs(rows, offsets=None, counts=None):
    """(first row, row past the last in use) of each run."""
    if offsets is None:
        return [(0, rows)]
    out, lo = [], 0
    off = [min(max(int(o), 0), rows) for o in offsets]
    off = list(np.maximum.accumulate(off))
    for g in range(len(off) - 1):
        n = off[g + 1] - off[g]
        if counts is not None:
            n = min(max(int(counts[g]), 0), n)
        out.append((off[g], off[g] + n))
    return out


def forward(x, up, down, name, offsets=None, counts=None):
    """(y, z) of the block: up [groups, 2 N, K], down [groups, C, N]."""
    x, up, down = (np.asarray(a, np.float64) for a in (x, up, down))
    N = down.shape[2]
    y, z = np.zeros((len(x), down.shape[1])), np.zeros((len(x), 2 * N))
    for g, (lo, hi) in enumerate(runs(len(x), offsets, counts)):
        z[lo:hi] = x[lo:hi] @ up[g].T
        y[lo:hi] = (act(z[lo:hi, :N], name) * z[lo:hi, N:]) @ down[g].T
    return y, z


def backward(dy, x, up, down, z, name, offsets=None, counts=None):
    """(dx, dup, ddown) for given z."""
    dy, x, up, down, z = (np.asarray(a, np.float64) for a in (dy, x, up, down, z))
    N = down.shape[2]
    dx, dup, ddown = np.zeros(x.shape), np.zeros(up.shape), np.zeros(down.shape)
    for g, (lo, hi) in enumerate(runs(len(x), offsets, counts)):
        gate, lin = z[lo:hi, :N], z[lo:hi, N:]
        dh = dy[lo:hi] @ down[g]
        a = act(gate, name)
        dz = np.concatenate([dh * lin * slope(gate, name), dh * a], 1)
        dx[lo:hi] = dz @ up[g]
        dup[g] = dz.T @ x[lo:hi]
        ddown[g] = dy[lo:hi].T @ (a * lin)
    return dx, dup, ddown


def int8_rows(x):
    """(codes, scales) of the rows of x: 127 x / a rounded to nearest even."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        a = np.abs(x).max(1, initial=0.0)
    bad = ~np.isfinite(x).all(1)
    a = np.where(bad, 0.0, a)
    q = 127.0 * np.where(bad[:, None], 0.0, x) / np.where(a > 0, a, 1.0)[:, None]
    return np.rint(q).astype(np.int64), np.where(bad, np.nan, a / 127.0)
