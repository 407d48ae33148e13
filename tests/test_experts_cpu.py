"""Expert-layer operators without a GPU: the fp64 oracle's own checks (rounding, gradients by
differences) and the argument checks of the C ABI, which launch nothing."""

import ctypes

import numpy as np
import pytest
import torch

from matrix_aware_optimizers_gb300 import _abi
from oracle import experts as ox

FAKE = 0x10000  # never dereferenced


def test_e4m3_rounds_as_the_format_does():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    values = np.unique(codes[np.isfinite(codes)])
    assert values.max() == 448.0
    np.testing.assert_array_equal(ox.e4m3(values), values)
    mid = (values[1:] + values[:-1]) / 2
    x = np.concatenate([mid, np.nextafter(mid, 1e9), np.nextafter(mid, -1e9), np.random.default_rng(0).normal(size=4000) * 50])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()  # fp64 to e4m3, one rounding
    dist = np.abs(x[:, None] - values[None]).min(1)
    np.testing.assert_array_equal(np.abs(ox.e4m3(x) - x), dist)
    far = np.abs(x[:, None] - mid[None]).min(1) > 1e-6
    np.testing.assert_array_equal(ox.e4m3(x)[far], want[far])
    # ties go to the even mantissa: 1.0625 lies between 1.0 (even) and 1.125 (odd)
    assert ox.e4m3(1.0625) == 1.0 and ox.e4m3(1.1875) == 1.25 and np.isnan(ox.e4m3(np.inf))


@pytest.mark.parametrize("blocks", ["row", "col", "tile"])
def test_scales_are_the_smallest_that_hold_the_block(blocks):
    x = np.random.default_rng(1).normal(size=(130, 140)) * np.exp(np.random.default_rng(2).normal(size=(130, 1)) * 6)
    x[0, :3] = [448.0, 449.0, 0.0]
    codes, scales = ox.quantize(x, blocks)
    br, bc = ox.block_shape(blocks)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            a = np.abs(x[i * br:(i + 1) * br, j * bc:(j + 1) * bc]).max()
            e = scales[i, j] - 127
            assert a <= 448.0 * 2.0 ** e and (a == 0 or a > 448.0 * 2.0 ** (e - 1))
    assert np.abs(codes).max() <= 448


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    x, g, opts = rng.normal(size=(5, 12)) * 2, rng.normal(size=(5, 3)), dict(score=score, renorm=renorm, scale=1.7)
    x[2, 4] = -np.inf
    w, ids, _ = ox.route(x, 3, **opts)
    d = ox.route_backward(x, ids, g, **opts)
    assert d[2, 4] == 0
    h = 1e-6
    for t in range(5):
        for e in range(12):
            if not np.isfinite(x[t, e]):
                continue
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            wu, iu, _ = ox.route(up, 3, **opts)
            wd, idn, _ = ox.route(down, 3, **opts)
            assert (iu == ids).all() and (idn == ids).all()
            assert abs((wu[t] - wd[t]) @ g[t] / (2 * h) - d[t, e]) < 1e-7  # h^2 and 1e-16 / h


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(4)
    row_of = np.array([[0, 3], [-1, 2], [4, -1]])
    z, w, dy = rng.normal(size=(6, 5)), rng.normal(size=(3, 2)), rng.normal(size=(3, 5))
    dz, dw = ox.combine_backward(dy, z, row_of, w)
    f = lambda z, w: (ox.combine(z, row_of, w) * dy).sum()  # noqa: E731  (linear in each)
    for i in np.ndindex(z.shape):
        p = z.copy()
        p[i] += 1.0
        assert abs(f(p, w) - f(z, w) - dz[i]) < 1e-12
    for i in np.ndindex(w.shape):
        p = w.copy()
        p[i] += 1.0
        assert abs(f(z, p) - f(z, w) - dw[i]) < 1e-12


def test_plan_keeps_the_order_of_the_tokens():
    counts, offsets, row_of, slot_of = ox.plan(np.array([[1, 0], [1, -1], [0, 1]]), 2, 256)
    assert counts.tolist() == [2, 3] and offsets.tolist() == [0, 128, 256]
    assert row_of.tolist() == [[128, 0], [129, -1], [1, 130]]
    assert slot_of[[0, 1, 128, 129, 130]].tolist() == [1, 4, 0, 2, 5] and (slot_of >= 0).sum() == 5


# ------------------------------------------------------------------------------ refusals


def mat(rows, cols, dtype=_abi.MAO_F32, data=FAKE, ld=None):
    return _abi.MaoMat(data, rows, cols, cols if ld is None else ld, dtype, 0)


def fp8(rows, cols, blocks, count=1, codes=FAKE, scales=FAKE, ld=None, scale_ld=None):
    wide = -(-cols // 16) * 16 if ld is None else ld
    sc = cols if blocks == _abi.MAO_BLOCKS_COL else -(-cols // 128)
    return _abi.MaoFp8(codes, scales, rows, cols, wide, sc if scale_ld is None else scale_ld, count, blocks)


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_quantize_refusals(lib):
    ROW, COL, TILE = 1, 2, 3

    def call(x, row=None, col=None, tile=None, batch=1, stride=0, index=None, n=0, copies=0):
        return lib.fp8_quantize(ref(x), batch, stride, index, n, copies, ref(row), ref(col), ref(tile), None)

    x, bad, mis, uns = mat(4, 40), 1, 3, 2
    assert call(None, fp8(4, 40, ROW)) == bad
    assert call(x) == bad                                             # nothing to write
    assert call(x, row=fp8(4, 40, ROW), tile=fp8(4, 40, TILE)) == bad  # tile goes alone
    assert call(x, row=fp8(4, 40, COL)) == bad
    assert call(x, row=fp8(5, 40, ROW)) == bad
    assert call(x, row=fp8(4, 41, ROW)) == bad
    assert call(x, row=fp8(4, 40, ROW, count=2)) == bad
    assert call(x, row=fp8(4, 40, ROW, ld=40)) == bad                 # rows of 16 bytes
    assert call(x, row=fp8(4, 40, ROW, scale_ld=0)) == bad
    assert call(x, col=fp8(4, 40, COL, scale_ld=39)) == bad
    assert call(x, row=fp8(4, 40, ROW, codes=None)) == bad
    assert call(x, row=fp8(4, 40, ROW, codes=FAKE + 8)) == mis
    assert call(mat(4, 40, data=FAKE + 2), row=fp8(4, 40, ROW)) == mis
    assert call(mat(4, 40, dtype=_abi.MAO_I8), row=fp8(4, 40, ROW)) == bad
    assert call(x, row=fp8(4, 40, ROW), batch=0) == bad
    assert call(x, row=fp8(4, 40, ROW), stride=-1) == bad
    assert call(x, row=fp8(9, 40, ROW), copies=-1) == bad
    assert call(x, row=fp8(9, 40, ROW), n=9, copies=1) == bad          # no index
    assert call(x, row=fp8(9, 40, ROW), index=FAKE + 2, n=9, copies=1) == mis
    assert call(x, row=fp8(9, 40, ROW, count=2), batch=2, stride=160, index=FAKE, n=9, copies=1) == bad
    assert call(x, row=fp8(1 << 31, 40, ROW), index=FAKE, n=1 << 31, copies=1) == uns
    assert call(x, row=fp8((1 << 31) - 1000, 40, ROW), index=FAKE, n=(1 << 31) - 1000, copies=1) == uns
    assert call(mat(0, 40, data=None), row=fp8(0, 40, ROW)) == 0       # no rows: nothing to do


def test_product_refusals(lib):
    ROW, COL, TILE = 1, 2, 3

    def call(a, b, d, form=0, off=None, groups=1, ws=None):
        return lib.fp8_product(ref(a), ref(b), ref(d), form, off, groups, 0, ws, 0, None)

    a, b, d = fp8(8, 32, ROW), fp8(16, 32, TILE), mat(8, 16)
    bad, uns, mis = 1, 2, 3
    assert call(None, b, d) == bad and call(a, None, d) == bad and call(a, b, None) == bad
    assert call(a, b, d, form=3) == bad and call(a, b, d, form=-1) == bad
    assert call(a, b, d, groups=0) == bad
    assert call(a, b, d, groups=2) == bad                              # groups need offsets
    assert call(a, b, d, off=FAKE, groups=1025) == uns
    assert call(a, b, d, off=FAKE + 1) == mis and call(a, b, d, ws=FAKE + 16) == mis
    assert lib.fp8_product_workspace_bytes(None, ref(b), 0) == 0
    assert lib.fp8_product_workspace_bytes(ref(a), ref(b), 3) == 0
    assert call(a, b, d, off=FAKE, groups=2) == bad                    # one matrix, two groups
    assert call(fp8(8, 32, COL), b, d) == bad and call(a, fp8(16, 32, ROW), d) == bad
    assert call(a, fp8(16, 33, TILE), d) == bad and call(a, b, mat(8, 17)) == bad
    assert call(a, b, mat(9, 16)) == bad
    assert call(a, b, mat(8, 16, data=FAKE + 2)) == mis
    assert call(a, b, mat(8, 16, dtype=_abi.MAO_I8)) == bad
    assert call(a, b, d, form=1) == bad                                # nn wants B [32][*]
    t = fp8(8, 16, COL), fp8(8, 32, COL)
    assert call(*t, mat(16, 31), form=2) == bad and call(*t, mat(32, 32), form=2) == bad
    assert call(t[0], fp8(9, 32, COL), mat(16, 32), form=2) == bad


def test_route_plan_combine_refusals(lib):
    bad, uns, mis, wsp = 1, 2, 3, 4
    x = mat(4, 32)

    def route(m, k=2, score=0, groups=1, keep=1, gs=0, scale=1.0, w=FAKE, ids=FAKE, bias=None):
        return lib.expert_route(ref(m), bias, k, score, groups, keep, gs, 1, scale, w, ids, None)

    assert route(None) == bad and route(x, k=0) == bad and route(x, k=33) == bad
    assert route(mat(4, 64), k=33) == uns and route(mat(4, 1025)) == uns
    assert route(x, groups=3) == bad and route(x, groups=4, keep=5) == bad and route(x, groups=4, keep=0) == bad
    assert route(x, k=9, groups=4, keep=1) == bad and route(mat(4, 64), groups=64, keep=8) == uns
    assert route(x, score=2) == bad and route(x, gs=2) == bad and route(x, scale=float("nan")) == bad
    assert route(x, w=None) == bad and route(x, ids=FAKE + 2) == mis and route(x, bias=FAKE + 1) == mis
    assert route(mat(0, 32, data=None), w=None, ids=None) == 0

    back = lambda m, d, k=2, ids=FAKE, g=FAKE: lib.expert_route_backward(  # noqa: E731
        ref(m), ids, g, k, 0, 1, 1.0, ref(d), None)
    assert back(x, mat(4, 31)) == bad and back(x, x, k=0) == bad and back(x, x, ids=None) == bad
    assert back(x, x, g=FAKE + 2) == mis and back(x, x, k=40) == uns

    assert lib.expert_rows(8, 128) == 1024 and lib.expert_rows(0, 4) == 0 and lib.expert_rows(-1, 4) == 0
    assert lib.expert_rows(1000, 2) == 1152
    assert lib.expert_plan_workspace_bytes(-1, 4) == 0 and lib.expert_plan_workspace_bytes(8, 1025) == 0

    def plan(n=8, e=4, slots=1024, ids=FAKE, ws=FAKE, wsb=1 << 20, off=FAKE):
        return lib.expert_plan(ids, n, e, FAKE, off, FAKE, FAKE, slots, ws, wsb, None)

    assert plan(n=-1) == bad and plan(e=0) == bad and plan(e=1025) == uns and plan(n=(1 << 24) + 1, slots=1 << 31) == uns
    assert plan(slots=256) == bad and plan(ids=None) == bad and plan(off=None) == bad
    assert plan(ws=FAKE + 16) == mis and plan(off=FAKE + 2) == mis
    assert plan(n=5000, slots=8192, ws=None) == bad and plan(n=5000, slots=8192, wsb=0) == wsp

    comb = lambda z, y, t=4, k=2, r=FAKE, w=FAKE: lib.expert_combine(ref(z), r, w, t, k, ref(y), None)  # noqa: E731
    assert comb(x, mat(4, 31)) == bad and comb(x, x, t=5) == bad and comb(x, x, k=0) == bad
    assert comb(x, x, k=33) == uns and comb(x, x, r=None) == bad and comb(x, x, w=FAKE + 1) == mis
    cb = lambda dy, z, dz, slot=FAKE, row=FAKE, dw=FAKE: lib.expert_combine_backward(  # noqa: E731
        ref(dy), ref(z), row, slot, None, 2, ref(dz), dw, None)
    assert cb(x, mat(256, 31), mat(256, 31)) == bad and cb(x, mat(256, 32), mat(255, 32)) == bad
    assert cb(x, mat(256, 32), mat(256, 32), slot=None) == bad and cb(x, mat(256, 32), mat(256, 32), row=None) == bad
    assert cb(x, mat(256, 32), mat(256, 32), dw=FAKE + 2) == mis
