"""Gated feed-forward block on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (a rounding to bf16 is within 2^-8 of the value, to fp32 within
2^-24; a sum of n terms in fp32, in any order and with each partial sum rounded or cut, within
n 2^-23 of the sum of magnitudes; the fast functions behind the activations within 2^-19 of
their size, 1 + |g| for the slopes): each stage's error is carried through the next one's
magnitudes, entry by entry.
"""

import numpy as np
import pytest
import torch

import matrix_aware_optimizers_gb300 as mao
from oracle import ffn as of

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U8, U19, U23 = 2.0 ** -8, 2.0 ** -19, 2.0 ** -23


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g)


def out_slack(y, dtype):
    return (U8 if dtype == BF16 else U23) * np.abs(y)


def bound_z(x, up, rs):
    """Error of the fp32 sums X up^T, entry by entry."""
    e = np.zeros((len(x), up.shape[1]))
    for g, (lo, hi) in enumerate(rs):
        e[lo:hi] = x.shape[1] * U23 * (np.abs(x[lo:hi]) @ np.abs(up[g]).T)
    return e


def check_forward(y, z, x, up, down, name, offsets=None, counts=None):
    X, W, D = np64(x), np64(up), np64(down)
    if W.ndim == 2:
        W, D = W[None], D[None]
    want, wz = of.forward(X, W, D, name, offsets, counts)
    rs = of.runs(len(X), offsets, counts)
    ez, N = bound_z(X, W, rs), D.shape[2]
    if z is not None:
        np.testing.assert_array_less(np.abs(np64(z) - wz), ez + out_slack(np.abs(wz) + ez, z.dtype) + 1e-30)
    G, U, eg, eu = wz[:, :N], wz[:, N:], ez[:, :N], ez[:, N:]
    a = np.abs(of.act(G, name))
    ea = 1.2 * eg + U19 * (a + 2.0 ** -20)  # slopes are below 1.2
    h = a * np.abs(U)
    eh = ea * (np.abs(U) + eu) + a * eu
    eh = eh + U8 * (h + eh)
    err = np.zeros(want.shape)
    for g, (lo, hi) in enumerate(rs):
        aD = np.abs(D[g]).T
        err[lo:hi] = eh[lo:hi] @ aD + N * U23 * ((h + eh)[lo:hi] @ aD)
    err += out_slack(np.abs(want) + err, y.dtype)
    np.testing.assert_array_less(np.abs(np64(y) - want), err + 1e-30)


def check_backward(grads, dy, x, up, down, z, name, offsets=None, counts=None):
    DY, X, W, D, Z = (np64(t) for t in (dy, x, up, down, z))
    if W.ndim == 2:
        W, D = W[None], D[None]
    N, C = D.shape[2], D.shape[1]
    want = of.backward(DY, X, W, D, Z, name, offsets, counts)
    errs = [np.zeros(w.shape) for w in want]
    for g, (lo, hi) in enumerate(of.runs(len(X), offsets, counts)):
        gate, lin = Z[lo:hi, :N], np.abs(Z[lo:hi, N:])
        a, s = np.abs(of.act(gate, name)), np.abs(of.slope(gate, name))
        ea, es = U19 * (a + 2.0 ** -20), U19 * (1.0 + np.abs(gate))
        dh, adh = np.abs(DY[lo:hi] @ D[g]), np.abs(DY[lo:hi]) @ np.abs(D[g])
        edh = C * U23 * adh
        dg, du, h = dh * lin * s, dh * a, a * lin
        edg = lin * (edh * (s + es) + dh * es)
        edu, eh = edh * (a + ea) + dh * ea, ea * lin
        edg, edu, eh = edg + U8 * (dg + edg), edu + U8 * (du + edu), eh + U8 * (h + eh)
        m, e = np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1)
        aW, n = np.abs(W[g]), hi - lo
        errs[0][lo:hi] = e @ aW + 2 * N * U23 * ((m + e) @ aW)
        aX, aY = np.abs(X[lo:hi]), np.abs(DY[lo:hi])
        errs[1][g] = e.T @ aX + (n + 1) * U23 * ((m + e).T @ aX)
        errs[2][g] = aY.T @ eh + (n + 1) * U23 * (aY.T @ (h + eh))
    for t, w, e in zip(grads, want, errs):
        got = np64(t).reshape(w.shape)
        np.testing.assert_array_less(np.abs(got - w), e + out_slack(np.abs(w) + e, t.dtype) + 1e-30)


def make(seed, T, K, N, C, groups=None, device="cuda"):
    s = () if groups is None else (groups,)
    x = randn(seed, T, K).to(BF16).to(device)
    up = (randn(seed + 1, *s, 2 * N, K) * K ** -0.5 * 1.5).to(BF16).to(device)
    down = (randn(seed + 2, *s, C, N) * N ** -0.5).to(BF16).to(device)
    dy = randn(seed + 3, T, C).to(BF16).to(device)
    return x, up, down, dy


SHAPES = [(1, 1, 1, 1), (1, 64, 16, 64), (2, 8, 3, 9), (7, 130, 33, 70), (32, 64, 128, 256), (33, 72, 136, 264),
          (64, 256, 64, 48), (100, 65, 257, 31), (255, 128, 128, 128), (257, 200, 144, 520),
          (300, 515, 260, 301), (513, 96, 384, 96)]


@pytest.mark.parametrize("save", [True, BF16])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("shape", SHAPES)
def test_block(cuda, shape, act, save):
    x, up, down, dy = make(sum(shape), *shape)
    y, z = mao.gated_ffn(x, up, down, act, save=save)
    assert z.dtype == (F32 if save is True else BF16)
    mao.sync_status()
    check_forward(y, z, x, up, down, act)
    assert torch.equal(mao.gated_ffn(x, up, down, act), y)  # without Z
    grads = mao.gated_ffn_backward(dy, x, up, down, z, act)
    mao.sync_status()
    assert [t.dtype for t in grads] == [BF16] * 3
    check_backward(grads, dy, x, up, down, z, act)


@pytest.mark.parametrize("shape", [(5, 40, 24, 56), (300, 515, 260, 301), (130, 1024, 512, 768)])
def test_fp32_outputs(cuda, shape):
    x, up, down, dy = make(9, *shape)
    y, z = mao.gated_ffn(x, up, down, "silu", save=True, out_dtype=F32)
    assert y.dtype == F32
    check_forward(y, z, x, up, down, "silu")
    grads = mao.gated_ffn_backward(dy, x, up, down, z, "silu", grad_dtype=F32)
    assert [t.dtype for t in grads] == [F32] * 3
    check_backward(grads, dy, x, up, down, z, "silu")


@pytest.mark.parametrize("save", [True, BF16])
@pytest.mark.parametrize("T", [1, 3, 8, 9, 16, 17, 48, 127, 128, 129])
def test_few_rows_long_sums(cuda, T, save):
    """Few rows: a kernel of their own, or sums that are split, their parts added by a second kernel."""
    x, up, down, dy = make(T, T, 2048, 1536, 1024)
    y, z = mao.gated_ffn(x, up, down, "silu", save=save)
    check_forward(y, z, x, up, down, "silu")
    check_backward(mao.gated_ffn_backward(dy, x, up, down, z, "silu"), dy, x, up, down, z, "silu")


def test_long_sums_over_rows(cuda):
    """Few outputs of the weights' gradients, many rows."""
    x, up, down, dy = make(77, 20000, 40, 24, 32)
    y, z = mao.gated_ffn(x, up, down, "gelu_tanh", save=True)
    check_forward(y, z, x, up, down, "gelu_tanh")
    check_backward(mao.gated_ffn_backward(dy, x, up, down, z, "gelu_tanh"), dy, x, up, down, z, "gelu_tanh")


RUNS = [([0, 128, 128, 384, 512], [100, 0, 256, 1], 512),
        ([0, 0, 384, 640, 640], [0, 300, 129, 0], 700),
        ([0, 256, 512, 1024, 1024], [256, 255, 512, 0], 1024)]


@pytest.mark.parametrize("save", [True, BF16])
@pytest.mark.parametrize("use_counts", [False, True])
@pytest.mark.parametrize("off,cnt,rows", RUNS)
@pytest.mark.parametrize("dims", [(64, 48, 80), (200, 136, 520), (77, 33, 41)])
def test_runs(cuda, off, cnt, rows, use_counts, dims, save):
    x, up, down, dy = make(rows + dims[0], rows, *dims, groups=4)
    counts = cnt if use_counts else None
    kw = dict(offsets=torch.tensor(off, dtype=torch.int32, device=cuda),
              counts=torch.tensor(cnt, dtype=torch.int32, device=cuda) if use_counts else None)
    y, z = mao.gated_ffn(x, up, down, "silu", save=save, **kw)
    mao.sync_status()
    check_forward(y, z, x, up, down, "silu", off, counts)
    used = torch.zeros(rows, dtype=torch.bool)
    for lo, hi in of.runs(rows, off, counts):
        used[lo:hi] = True
    assert (y[~used.to(cuda)] == 0).all() and (z[~used.to(cuda)] == 0).all()
    grads = mao.gated_ffn_backward(dy, x, up, down, z, "silu", **kw)
    mao.sync_status()
    check_backward(grads, dy, x, up, down, z, "silu", off, counts)
    assert (grads[0][~used.to(cuda)] == 0).all()


def test_forward_runs_anywhere(cuda):
    """The forward pass takes runs that start at any row, fall, or leave the rows."""
    x, up, down, _ = make(3, 300, 64, 48, 80, groups=5)
    for off in ([0, 1, 34, 35, 290, 300], [7, 50, 40, 200, 200, 9999], [-5, 3, 3, 3, 3, 250]):
        t = torch.tensor(off, dtype=torch.int32, device=cuda)
        y, z = mao.gated_ffn(x, up, down, "gelu", offsets=t, save=True)
        mao.sync_status()
        check_forward(y, z, x, up, down, "gelu", off)


def test_counts_out_of_range(cuda):
    x, up, down, _ = make(4, 256, 64, 48, 80, groups=3)
    off, cnt = [0, 128, 128, 256], [-3, 9, 500]
    y = mao.gated_ffn(x, up, down, "silu", offsets=torch.tensor(off, dtype=torch.int32, device=cuda),
                      counts=torch.tensor(cnt, dtype=torch.int32, device=cuda))
    check_forward(y, None, x, up, down, "silu", off, cnt)


def test_padding_rows_hold_anything(cuda):
    """Forward: NaN in rows past the counts. Backward: any finite values there."""
    x, up, down, dy = make(5, 384, 72, 40, 56, groups=3)
    off, cnt = [0, 128, 256, 384], [100, 128, 3]
    kw = dict(offsets=torch.tensor(off, dtype=torch.int32, device=cuda),
              counts=torch.tensor(cnt, dtype=torch.int32, device=cuda))
    xn = x.clone()
    xn[100:128], xn[259:] = float("nan"), float("inf")
    y, z = mao.gated_ffn(xn, up, down, "silu", save=True, **kw)
    y0, z0 = mao.gated_ffn(x, up, down, "silu", save=True, **kw)
    assert torch.equal(y, y0) and torch.equal(z, z0)
    big, dbig = x.clone(), dy.clone()
    big[100:128], dbig[259:] = 3e38, -3e38
    for a, b in zip(mao.gated_ffn_backward(dbig, big, up, down, z, "silu", **kw),
                    mao.gated_ffn_backward(dy, x, up, down, z, "silu", **kw)):
        assert torch.equal(a, b)


def test_strides_and_outputs(cuda):
    """Column slices (aligned and not), outputs with gaps beside them that stay as they were."""
    T, K, N, C = 150, 96, 72, 88
    x, up, down, dy = make(6, T, K, N, C)

    def wide(t, left, right):
        big = torch.full((t.shape[0], left + t.shape[1] + right), 7.0, dtype=t.dtype, device=cuda)
        big[:, left:left + t.shape[1]] = t
        return big[:, left:left + t.shape[1]]

    for left, right, save in ((8, 8, BF16), (1, 2, BF16), (3, 4, BF16), (4, 4, F32), (1, 2, F32)):
        y0, z0 = mao.gated_ffn(x, up, down, "silu", save=save)
        g0 = mao.gated_ffn_backward(dy, x, up, down, z0, "silu")
        xs, us, ds, dys = (wide(t, left, right) for t in (x, up, down, dy))
        out = wide(torch.zeros(T, C, dtype=BF16, device=cuda), left, right)
        Z = wide(torch.zeros(T, 2 * N, dtype=save, device=cuda), left, right)
        y, z = mao.gated_ffn(xs, us, ds, "silu", out=out, Z=Z)
        assert y is out and z is Z and torch.equal(y, y0) and torch.equal(z, z0)
        outs = [wide(torch.zeros_like(t), left, right) for t in (x, up, down)]
        got = mao.gated_ffn_backward(dys, xs, us, ds, Z, "silu", dX=outs[0], dup=outs[1], ddown=outs[2])
        for a, b in zip(got, g0):
            assert torch.equal(a, b)
        for t in [out, Z] + outs:
            base = t._base if t._base is not None else t
            assert (base[:, :left] == 7).all() and (base[:, left + t.shape[1]:] == 7).all()
    only = mao.gated_ffn_backward(dy, x, up, down, z0, "silu", dX=False, ddown=False)
    assert only[0] is None and only[2] is None and torch.equal(only[1], g0[1])


@pytest.mark.parametrize("T", [1, 3, 150])
def test_odd_widths_of_aligned_rows(cuda, T):
    """Slices whose rows start at multiples of 16 bytes and whose widths are no multiples of that: what
    lies beside them takes no part and stays as it is."""
    K, N, C = 97, 71, 83
    x, up, down, dy = make(11, T, K, N, C)

    def wide(t):
        big = torch.full((t.shape[0], (t.shape[1] + 15) // 8 * 8), float("nan"), dtype=t.dtype, device=cuda)
        big[:, :t.shape[1]] = t
        return big[:, :t.shape[1]]

    for save in (F32, BF16):
        y0, z0 = mao.gated_ffn(x, up, down, "gelu", save=save)
        check_forward(y0, z0, x, up, down, "gelu")
        g0 = mao.gated_ffn_backward(dy, x, up, down, z0, "gelu")
        xs, us, ds, dys = (wide(t) for t in (x, up, down, dy))
        out, Z = wide(torch.zeros_like(y0)), wide(torch.zeros_like(z0))
        y, z = mao.gated_ffn(xs, us, ds, "gelu", out=out, Z=Z)
        assert y is out and z is Z and torch.equal(y, y0) and torch.equal(z, z0)
        outs = [wide(torch.zeros_like(t)) for t in (x, up, down)]
        got = mao.gated_ffn_backward(dys, xs, us, ds, Z, "gelu", dX=outs[0], dup=outs[1], ddown=outs[2])
        for a, b in zip(got, g0):
            assert torch.equal(a, b)
        for t in [out, Z] + outs:
            assert t._base[:, t.shape[1]:].isnan().all()
    mao.sync_status()


def test_no_rows(cuda):
    x, up, down, dy = make(8, 0, 40, 24, 32)
    y, z = mao.gated_ffn(x, up, down, "silu", save=True)
    assert y.shape == (0, 32) and z.shape == (0, 48)
    dx, dup, ddown = mao.gated_ffn_backward(dy, x, up, down, z, "silu")
    assert dx.shape == (0, 40) and (dup == 0).all() and (ddown == 0).all()


def test_extreme_values(cuda):
    """Large pre-activations of either sign; an infinite one gives what the formula gives."""
    T, K, N, C = 4, 16, 8, 8
    x = torch.zeros(T, K, dtype=BF16, device=cuda)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 100.0, -100.0, 3e4, -3e4
    up = torch.zeros(2 * N, K, dtype=BF16, device=cuda)
    up[:, 0] = 1.0
    down = torch.eye(8, dtype=BF16, device=cuda)
    for act in ("silu", "gelu", "gelu_tanh"):
        y, z = mao.gated_ffn(x, up, down, act, save=True, out_dtype=F32)
        check_forward(y, z, x, up, down, act)
        dy = torch.ones(T, C, dtype=BF16, device=cuda)
        check_backward(mao.gated_ffn_backward(dy, x, up, down, z, act), dy, x, up, down, z, act)
    x[0, 0] = float("inf")
    y = mao.gated_ffn(x, up, down, "silu")
    assert y[0].isnan().all() or (y[0] == float("inf")).any()
    assert torch.isfinite(y[1:]).all()


def test_gradient_against_differences(cuda):
    """The gradient of sum(dY * Y) in the oracle's own terms, by differences in 64 bits."""
    x, up, down, dy = make(11, 6, 10, 4, 5)
    X, W, D, DY = np64(x), np64(up)[None], np64(down)[None], np64(dy)
    for name in ("silu", "gelu", "gelu_tanh"):
        _, z = of.forward(X, W, D, name)
        want = of.backward(DY, X, W, D, z, name)
        for which, arr in enumerate((X, W, D)):
            flat = arr.reshape(-1)
            for i in range(0, flat.size, 7):
                keep, h = flat[i], 1e-5
                flat[i] = keep + h
                a = (of.forward(X, W, D, name)[0] * DY).sum()
                flat[i] = keep - h
                b = (of.forward(X, W, D, name)[0] * DY).sum()
                flat[i] = keep
                assert abs((a - b) / (2 * h) - want[which].reshape(-1)[i]) < 1e-6
