"""Expert-layer operators on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24 is fp32's rounding, 2^-9 bf16's):
  codes, scales, ids, plans   equal
  products   the terms are exact in fp32; a sum of K terms, in any order and with each partial
             sum rounded or cut, is within K 2^-23 of the sum of magnitudes, and its store in
             bf16 within 2^-9 of the value
  weights    E terms of a softmax and a few roundings: (E + 32) 2^-23 relative
"""

import numpy as np
import pytest
import torch

import matrix_aware_optimizers_gb300 as mao
from oracle import experts as ox

pytestmark = pytest.mark.gpu

U23 = 2.0 ** -23


def dt(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g)


def out_slack(y, dtype):
    return 2.0 ** -8 * np.abs(y) if dtype == torch.bfloat16 else 2.0 ** -23 * np.abs(y)


# ------------------------------------------------------------------------------ quantise


def spread(seed, R, C):
    return randn(seed, R, C) * torch.exp(2 * randn(seed + 1, R, 1)) * torch.exp(randn(seed + 2, 1, C))


def check_quantized(codes, scales, x, blocks):
    want, bytes_ = ox.quantize(x, blocks)
    np.testing.assert_array_equal(scales.cpu().numpy().astype(np.int64), bytes_)
    np.testing.assert_array_equal(np64(codes), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("blocks", ["row", "col", "tile", "both"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (128, 1), (3, 130), (129, 7), (127, 129),
                                   (256, 256), (300, 520)])
def test_quantize(cuda, dtype, blocks, shape):
    x = spread(sum(shape), *shape).to(dt(dtype)).to(cuda)
    out = mao.fp8_quantize(x, blocks)
    mao.sync_status()
    kinds = ("row", "col") if blocks == "both" else (blocks,)
    for i, k in enumerate(kinds):
        assert out[2 * i].dtype == torch.float8_e4m3fn and out[2 * i].stride(0) % 16 == 0
        check_quantized(out[2 * i], out[2 * i + 1], np64(x), k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("blocks", ["row", "col", "tile"])
def test_quantize_special_values(cuda, dtype, blocks):
    """Zeros, the largest and the smallest numbers, ties, signed zeros, NaN and infinities."""
    x = torch.zeros(256, 384)
    x[0, :128] = torch.linspace(-448, 448, 128)             # ties between codes
    x[1, 0], x[1, 1] = 448.0 * 2.0 ** 7, 449.0 * 2.0 ** 7   # at and above the largest code
    x[2, :4] = torch.tensor([1.7e38, -3.3e38, 1.0, -0.0])
    x[3, 128:132] = torch.tensor([1e-40, -1e-38, 2.0 ** -126, 0.0])
    x[130, 5], x[130, 6], x[130, 7] = float("nan"), float("inf"), -float("inf")
    x[130, 8:20] = torch.arange(12.0)
    x[140, 260] = float("nan")                              # a block with nothing finite but 0
    x = x.to(dt(dtype)).to(cuda)
    codes, scales = mao.fp8_quantize(x, blocks)
    check_quantized(codes, scales, np64(x), blocks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_strides_and_stacks(cuda, dtype):
    """Column slices (aligned and not), stacked matrices, lists, outputs with gaps beside
    them that stay as they were."""
    big = spread(3, 200, 700).to(dt(dtype)).to(cuda)
    for c0, C in ((0, 300), (8, 256), (1, 257)):
        x = big[:, c0:c0 + C]
        codes, scales = mao.fp8_quantize(x, "tile")
        check_quantized(codes, scales, np64(x), "tile")
    s = torch.stack([spread(i, 130, 150) for i in range(5)]).to(dt(dtype)).to(cuda)
    for X in (s, list(s.unbind(0)), s[:, 1:, 3:], s[::2]):
        codes, scales = mao.fp8_quantize(X, "row")
        for i, x in enumerate(X):
            check_quantized(codes[i], scales[i], np64(x), "row")
    many = [spread(i, 20, 33).to(dt(dtype)).to(cuda) for i in range(70)]  # more than one launch
    codes, scales = mao.fp8_quantize(many, "col")
    for i in (0, 63, 64, 69):
        check_quantized(codes[i], scales[i], np64(many[i]), "col")
    wide = torch.full((200, 320), 7, dtype=torch.uint8, device=cuda)
    sc = torch.full((200, 5), 9, dtype=torch.uint8, device=cuda)
    x = big[:, :300]
    mao.fp8_quantize(x, "row", out=(wide[:, :300], sc[:, :3]))
    check_quantized(wide[:, :300].view(torch.float8_e4m3fn), sc[:, :3], np64(x), "row")
    assert (wide[:, 300:] == 7).all() and (sc[:, 3:] == 9).all()


@pytest.mark.parametrize("copies", [1, 3])
def test_quantize_gather(cuda, copies):
    x = spread(5, 40, 200).to(cuda)
    g = torch.Generator().manual_seed(1)
    rows = torch.randint(-3, 40 * copies + 2, (300,), generator=g).to(torch.int32)
    rows[128:256] = -1                                       # a block of padding
    src = torch.div(rows, copies, rounding_mode="floor").long()
    have = (rows >= 0) & (src < 40)
    y = torch.where(have[:, None], x.cpu()[torch.where(have, src, 0)], 0.0)
    out = mao.fp8_quantize(x, "both", rows=rows.to(cuda), copies=copies)
    check_quantized(out[0], out[1], np64(y), "row")
    check_quantized(out[2], out[3], np64(y), "col")
    none = mao.fp8_quantize(x, "row", rows=rows[:0].to(cuda))
    assert none[0].shape == (0, 200) and none[1].shape == (0, 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("blocks", ["row", "col", "both"])
@pytest.mark.parametrize("copies", [1, 7, 2 ** 20 + 1])
def test_quantize_gather_whole_tiles(cuda, dtype, blocks, copies):
    """Blocks of rows that all exist, some that do not, and a ragged last one."""
    x = spread(6, 33, 256).to(dtype).to(cuda)
    g = torch.Generator().manual_seed(2)
    rows = torch.randint(0, 33 * copies, (330,), generator=g)
    rows[:4] = torch.tensor([0, copies - 1, copies, 33 * copies - 1])  # ends of runs of copies
    rows[130], rows[200], rows[201] = -1, 33 * copies, 2 ** 31 - 1
    src = torch.div(rows, copies, rounding_mode="floor")
    have = (rows >= 0) & (src < 33)
    y = torch.where(have[:, None], x.cpu()[torch.where(have, src, 0)], torch.zeros((), dtype=dtype))
    out = mao.fp8_quantize(x, blocks, rows=rows.to(torch.int32).to(cuda), copies=copies)
    if blocks != "col":
        check_quantized(out[0], out[1], np64(y), "row")
    if blocks != "row":
        check_quantized(out[-2], out[-1], np64(y), "col")


# ------------------------------------------------------------------------------ products


def operands(form, R, N, K, groups, seed, device):
    """Quantised operands and their values."""
    a = spread(seed, R, K if form == "nt" else N) if R else torch.zeros(0, K if form == "nt" else N)
    ak = "col" if form == "tn" else "row"
    A, As = mao.fp8_quantize(a.to(device), ak)
    av = ox.dequantize(np64(A), As.cpu().numpy(), ak)
    if form == "tn":
        B, Bs = mao.fp8_quantize((spread(seed + 7, R, K) if R else torch.zeros(0, K)).to(device), "col")
        return A, As, B, Bs, av, ox.dequantize(np64(B), Bs.cpu().numpy(), "col")
    b = torch.stack([spread(seed + 11 * i + 7, N, K) for i in range(groups)])
    B, Bs = mao.fp8_quantize(b.to(device), "tile")
    bv = [ox.dequantize(np64(B[i]), Bs[i].cpu().numpy(), "tile") for i in range(groups)]
    return A, As, B, Bs, av, bv


def check_product(out, av, bv, form, offsets, extra=None):
    want = ox.product(av, bv, form, offsets)
    mag = ox.product(np.abs(av), np.abs(bv) if form == "tn" else [np.abs(b) for b in bv], form, offsets)
    depth = max(1, av.shape[1] if form != "tn" else av.shape[0])
    if extra is not None:
        want, mag = want + extra, mag + np.abs(extra)
    got = np64(out).reshape(want.shape)
    tol = (depth + 2) * U23 * mag + out_slack(want, out.dtype)
    assert (np.abs(got - want) <= tol).all(), float(np.max(np.abs(got - want) - tol))


DENSE = [(1, 1, 1), (1, 128, 128), (5, 16, 300), (130, 257, 129), (128, 256, 512), (300, 200, 1000),
         (257, 520, 136), (64, 768, 256), (515, 264, 648)]


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape", DENSE)
def test_product_dense(cuda, form, out, shape):
    R, N, K = shape
    A, As, B, Bs, av, bv = operands(form, R, N, K, 1, R + N + K, cuda)
    y = mao.fp8_product(A, As, B, Bs, form, out_dtype=dt(out))
    mao.sync_status()
    check_product(y, av, bv, form, None)


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_product_long_sum_is_split(cuda, form, out, accumulate):
    """Few outputs and a long sum: parts of it, of unlike sizes, added up in their order."""
    deep = 7001
    R, N, K = {"nt": (37, 130, deep), "nn": (37, deep, 130), "tn": (deep, 37, 130)}[form]
    A, As, B, Bs, av, bv = operands(form, R, N, K, 1, 31, cuda)
    shape = ox.product(av, bv, form, None).shape
    base = randn(3, *shape).to(dt(out)).to(cuda)
    y = base.clone()
    assert mao.lib().fp8_product_workspace_bytes(
        mao.ctypes.byref(mao._fp8(A, As, "col" if form == "tn" else "row", "A")),
        mao.ctypes.byref(mao._fp8(B, Bs, "col" if form == "tn" else "tile", "B")),
        {"nt": 0, "nn": 1, "tn": 2}[form]) > 0
    mao.fp8_product(A, As, B, Bs, form, out=y, accumulate=accumulate)
    mao.sync_status()
    check_product(y, av, bv, form, None, np64(base).reshape(shape) if accumulate else None)
    z = base.clone()  # too small a workspace: in one part
    mao.fp8_product(A, As, B, Bs, form, out=z, accumulate=accumulate,
                    ws=torch.empty(256, dtype=torch.uint8, device=cuda))
    check_product(z, av, bv, form, None, np64(base).reshape(shape) if accumulate else None)


SIZES = [[0, 128, 0, 256, 384, 0], [128], [0, 0], [640, 128, 0, 0, 128], [128] * 9]


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("rest", [0, 200])
def test_product_groups(cuda, form, out, sizes, rest):
    """Groups of whole blocks, some of them empty, with rows past the last group."""
    R, N, K = sum(sizes) + rest, 144, 272
    off = np.concatenate([[0], np.cumsum(sizes)])
    A, As, B, Bs, av, bv = operands(form, R, N, K, len(sizes), len(sizes), cuda)
    o = torch.tensor(off, dtype=torch.int32, device=cuda)
    y = mao.fp8_product(A, As, B, Bs, form, offsets=o, out_dtype=dt(out))
    mao.sync_status()
    check_product(y, av, bv, form, off)
    # added to what is there: rows and matrices without a group keep their values
    base = randn(3, *y.shape).to(dt(out)).to(cuda)
    acc = base.clone()
    mao.fp8_product(A, As, B, Bs, form, offsets=o, out=acc, accumulate=True)
    check_product(acc, av, bv, form, off, np64(base).reshape(ox.product(av, bv, form, off).shape))
    if form != "tn" and rest:
        assert torch.equal(acc[off[-1]:], base[off[-1]:])


@pytest.mark.parametrize("form", ["nt", "nn"])
def test_product_groups_of_any_size(cuda, form):
    sizes = [1, 0, 31, 129, 7, 255, 257]
    R, N, K = sum(sizes), 136, 150
    off = np.concatenate([[0], np.cumsum(sizes)])
    A, As, B, Bs, av, bv = operands(form, R, N, K, len(sizes), 77, cuda)
    y = mao.fp8_product(A, As, B, Bs, form, offsets=torch.tensor(off, dtype=torch.int32, device=cuda),
                        out_dtype=torch.float32)
    check_product(y, av, bv, form, off)


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_product_offsets_are_cut_to_the_rows(cuda, form):
    """Offsets outside the rows name no row: nothing is read or written there."""
    R, N, K = 256, 64, 128
    A, As, B, Bs, av, bv = operands(form, R, N, K, 3, 5, cuda)
    o = torch.tensor([-128, 128, 1 << 30, 1 << 30], dtype=torch.int32, device=cuda)
    y = mao.fp8_product(A, As, B, Bs, form, offsets=o, out_dtype=torch.float32)
    mao.sync_status()
    check_product(y, av, bv, form, [0, 128, 256, 256])


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_product_into_slices(cuda, form, out):
    """Outputs with odd strides and starts; what lies beside them stays."""
    R, N, K = 200, 130, 261
    A, As, B, Bs, av, bv = operands(form, R, N, K, 1, 9, cuda)
    rows, cols = {"nt": (R, N), "nn": (R, K), "tn": (N, K)}[form]
    for pad, left in ((3, 1), (8, 4)):
        buf = torch.full((rows, cols + pad), 5.0, dtype=dt(out), device=cuda)
        y = buf[:, left:left + cols]
        mao.fp8_product(A, As, B, Bs, form, out=y)
        check_product(y, av, bv, form, None)
        assert (buf[:, :left] == 5).all() and (buf[:, left + cols:] == 5).all()


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_product_scales_of_every_size(cuda, form):
    """Scales from one end of the range to the other, and zero blocks."""
    R, N, K = 256, 256, 384
    A, As, B, Bs, _, _ = operands(form, R, N, K, 1, 21, cuda)
    g = torch.Generator().manual_seed(2)
    As.copy_(torch.randint(90, 165, tuple(As.shape), generator=g))
    Bs.copy_(torch.randint(90, 165, tuple(Bs.shape), generator=g))
    As.view(-1)[::5] = 0
    A[::7] = 0.0
    ak, bk = ("col", "col") if form == "tn" else ("row", "tile")
    av = ox.dequantize(np64(A), As.cpu().numpy(), ak)
    bv = ox.dequantize(np64(B if form == "tn" else B[0]), (Bs if form == "tn" else Bs[0]).cpu().numpy(), bk)
    y = mao.fp8_product(A, As, B, Bs, form, out_dtype=torch.float32)
    check_product(y, av, bv if form == "tn" else [bv], form, None)


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_product_nan_reaches_its_row_only(cuda, form):
    R, N, K = 256, 160, 256
    a = spread(1, R, K if form == "nt" else N)
    a[130, 20] = float("inf")
    A, As = mao.fp8_quantize(a.to(cuda), "col" if form == "tn" else "row")
    b = spread(2, R, K) if form == "tn" else spread(2, N, K)[None]
    B, Bs = mao.fp8_quantize(b.to(cuda), "col" if form == "tn" else "tile")
    y = mao.fp8_product(A, As, B, Bs, form, out_dtype=torch.float32)
    y = y[0] if form == "tn" else y
    nan = torch.isnan(y).all(1).nonzero().flatten().tolist()
    assert nan == [20 if form == "tn" else 130]
    assert int(torch.isnan(y).sum()) == y.shape[1]


def test_product_zero_rows(cuda):
    for form in ("nt", "nn"):
        A, As, B, Bs, _, _ = operands(form, 0, 32, 48, 2, 1, cuda)
        o = torch.zeros(3, dtype=torch.int32, device=cuda)
        assert mao.fp8_product(A, As, B, Bs, form, offsets=o).shape[0] == 0
    A, As, B, Bs, _, _ = operands("tn", 0, 32, 48, 1, 1, cuda)
    y = mao.fp8_product(A, As, B, Bs, "tn", offsets=torch.zeros(4, dtype=torch.int32, device=cuda))
    assert y.shape == (3, 32, 48) and (y == 0).all()


def test_product_repeats_exactly_on_another_stream(cuda):
    A, As, B, Bs, _, _ = operands("nt", 700, 520, 1100, 1, 4, cuda)
    y = mao.fp8_product(A, As, B, Bs, "nt", out_dtype=torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        z = mao.fp8_product(A, As, B, Bs, "nt", out_dtype=torch.float32, stream=s)
        s.synchronize()
        assert torch.equal(y, z)


def test_product_in_a_graph(cuda):
    """A captured product reads its operands and offsets at each replay."""
    A, As, B, Bs, av, bv = operands("nt", 512, 200, 300, 2, 6, cuda)
    o = torch.tensor([0, 128, 512], dtype=torch.int32, device=cuda)
    y = torch.zeros(512, 200, device=cuda)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        mao.fp8_product(A, As, B, Bs, "nt", offsets=o, out=y)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mao.fp8_product(A, As, B, Bs, "nt", offsets=o, out=y)
    for off in ([0, 384, 512], [0, 0, 130]):
        o.copy_(torch.tensor(off, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        check_product(y, av, bv, "nt", off)


def test_product_wait_limit(cuda):
    """With a limit of 0 every wait that is not over at once gives up: the error is reported,
    and the next product is whole again."""
    A, As, B, Bs, av, bv = operands("nt", 600, 300, 4000, 1, 8, cuda)
    torch.cuda.synchronize()
    limit = mao.get_wait_limit()
    mao.set_wait_limit(0)
    try:
        mao.fp8_product(A, As, B, Bs, "nt", out_dtype=torch.float32)
        with pytest.raises(mao.MaoError) as e:
            mao.sync_status()
        assert "TIMEOUT" in str(e.value)
    finally:
        mao.set_wait_limit(limit)
    y = mao.fp8_product(A, As, B, Bs, "nt", out_dtype=torch.float32)
    mao.sync_status()
    check_product(y, av, bv, "nt", None)


# ------------------------------------------------------------------------------ routing


def grid_logits(seed, T, E, dtype, masked=False):
    """Logits on a coarse grid, so that equal ones (ties) are common and near ones far."""
    x = (randn(seed, T, E) * 12).round() / 8
    if masked:
        g = torch.Generator().manual_seed(seed)
        x[torch.rand(T, E, generator=g) < 0.3] = -float("inf")
        x[torch.rand(T, generator=g) < 0.2] = -float("inf")
        x[0] = -float("inf")
    return x.to(dtype)


ROUTES = [dict(E=8, k=2), dict(E=1, k=1), dict(E=128, k=8), dict(E=60, k=4, renorm=False),
          dict(E=256, k=8, groups=8, keep_groups=4, score="sigmoid", bias=True, scale=2.5),
          dict(E=160, k=6, groups=8, keep_groups=3, group_score="max"),
          dict(E=64, k=3, groups=32, keep_groups=5, bias=True), dict(E=1000, k=32, score="sigmoid"),
          dict(E=384, k=8, score="sigmoid", bias=True, renorm=False), dict(E=33, k=32, bias=True)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("case", range(len(ROUTES)))
def test_route(cuda, dtype, masked, case):
    c = dict(ROUTES[case])
    E, k = c.pop("E"), c.pop("k")
    T = 37
    x = grid_logits(case, T, E, dt(dtype), masked)
    bias = (randn(case + 50, E) * 4).round() / 64 if c.pop("bias", False) else None
    w, ids = mao.expert_route(x.to(cuda), k, bias=None if bias is None else bias.to(cuda), **c)
    want_w, want_ids, decided = ox.route(np64(x), k, bias=None if bias is None else bias.numpy(), **c)
    assert decided.mean() > 0.5
    np.testing.assert_array_equal(ids.cpu().numpy()[decided], want_ids[decided])
    tol = (E + 32) * U23 * np.abs(want_w[decided]) + 1e-38
    assert (np.abs(np64(w)[decided] - want_w[decided]) <= tol).all()

    # gradient of the logits
    g = randn(case + 9, T, k)
    opts = {n: c[n] for n in ("score", "renorm", "scale") if n in c}
    d = mao.expert_route_backward(x.to(cuda), ids, g.to(cuda), **opts)
    assert d.dtype == x.dtype
    want = ox.route_backward(np64(x), ids.cpu().numpy(), g.numpy(), **opts)
    # the chosen scores' differences: each ds within (E + 32) 2^-23 of the gradients' sizes
    size = np.abs(g.numpy()).sum(1, keepdims=True) * c.get("scale", 1.0)
    s = ox.scores(np64(x), c.get("score", "softmax"))
    total = np.array([sum(s[t, e] for e in i if e >= 0) for t, i in enumerate(ids.cpu().numpy())])
    size = size / np.maximum(total, 1e-20)[:, None] if c.get("renorm", True) else size
    tol = (E + 64) * U23 * s * size + out_slack(want, x.dtype) + 1e-37
    assert (np.abs(np64(d) - want) <= tol).all()


def test_route_one_and_no_token(cuda):
    for T in (0, 1):
        x = randn(1, T, 16).to(cuda)
        w, ids = mao.expert_route(x, 2)
        assert w.shape == ids.shape == (T, 2)
        assert mao.expert_route_backward(x, ids, w).shape == (T, 16)
    x = torch.tensor([[0.5, -0.0, 0.0, 0.5]], device=cuda)  # ties, and zeros of both signs
    assert mao.expert_route(x, 4)[1].tolist() == [[0, 3, 1, 2]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_lone_expert_has_no_gradient(cuda, score):
    """With renorm a single expert's weight is 1 whatever its score."""
    x = randn(5, 300, 60).to(cuda)
    w, ids = mao.expert_route(x, 1, score=score, scale=2.5)
    assert (w == 2.5).all()
    assert (mao.expert_route_backward(x, ids, randn(6, 300, 1).to(cuda), score=score, scale=2.5) == 0).all()


def test_route_nan_and_infinity(cuda):
    x = torch.tensor([[1.0, float("nan"), 2.0, 0.0], [1.0, float("inf"), 2.0, 0.0]], device=cuda)
    w, ids = mao.expert_route(x, 2)
    assert ids.tolist() == [[2, 0], [1, 2]] and torch.isnan(w).all()
    w, ids = mao.expert_route(x, 2, score="sigmoid", renorm=False)
    assert ids.tolist() == [[2, 0], [1, 2]] and w[1, 0] == 1.0 and torch.isfinite(w).all()


def test_route_strided_logits(cuda):
    big = grid_logits(4, 20, 100, torch.float32).to(cuda)
    x = big[:, 3:67]
    w, ids = mao.expert_route(x, 4)
    w2, ids2 = mao.expert_route(x.contiguous(), 4)
    assert torch.equal(w, w2) and torch.equal(ids, ids2)
    dl = torch.full((20, 100), 3.0, device=cuda)
    mao.expert_route_backward(x, ids, w, dlogits=dl[:, 3:67])
    assert torch.equal(dl[:, 3:67], mao.expert_route_backward(x, ids, w))
    assert (dl[:, :3] == 3).all() and (dl[:, 67:] == 3).all()


# ------------------------------------------------------------------------------ plan, combine


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 128), (40, 3, 7), (500, 2, 1),
                                   (1000, 8, 256), (3000, 4, 1000), (9001, 8, 60)])
def test_plan(cuda, T, k, E):
    g = torch.Generator().manual_seed(T + E)
    ids = torch.randint(-1, E + 1, (T, k), generator=g).to(torch.int32)  # some dropped
    p = mao.expert_plan(ids.to(cuda), E)
    mao.sync_status()
    n = mao.expert_rows(T * k, E)
    counts, offsets, row_of, slot_of = ox.plan(ids.numpy(), E, n)
    assert offsets[-1] <= n
    np.testing.assert_array_equal(p.counts.cpu().numpy(), counts)
    np.testing.assert_array_equal(p.offsets.cpu().numpy(), offsets)
    np.testing.assert_array_equal(p.row_of.cpu().numpy(), row_of)
    np.testing.assert_array_equal(p.slot_of.cpu().numpy(), slot_of)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,H,E", [(1, 1, 1, 1), (1, 8, 2048, 128), (33, 3, 24, 5), (70, 32, 770, 40),
                                     (129, 2, 4100, 8)])
@pytest.mark.parametrize("weighted", [False, True])
def test_combine(cuda, dtype, T, k, H, E, weighted):
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, E, (T, k), generator=g).to(torch.int32).to(cuda)
    p = mao.expert_plan(ids, E)
    rows = mao.expert_rows(T * k, E)
    z = randn(1, rows, H).to(dt(dtype)).to(cuda)
    w = randn(2, T, k).to(cuda) if weighted else None
    row_of = p.row_of.cpu().numpy()
    wn = None if w is None else w.cpu().numpy()
    y = mao.expert_combine(z, p.row_of, w)
    want = ox.combine(np64(z), row_of, wn)
    mag = ox.combine(np.abs(np64(z)), row_of, None if wn is None else np.abs(wn))
    assert (np.abs(np64(y) - want) <= (k + 1) * U23 * mag + out_slack(want, y.dtype)).all()
    dy = randn(3, T, H).to(dt(dtype)).to(cuda)
    dz, dw = mao.expert_combine_backward(dy, z, p.row_of, p.slot_of, w)
    want_z, want_w = ox.combine_backward(np64(dy), np64(z), row_of, wn)
    assert (np.abs(np64(dz) - want_z) <= out_slack(want_z, dz.dtype)).all()
    _, mag = ox.combine_backward(np.abs(np64(dy)), np.abs(np64(z)), row_of, wn)
    assert (np.abs(np64(dw) - want_w) <= (H + 1) * U23 * mag).all()


def test_combine_dropped_tokens_and_slices(cuda):
    z = randn(1, 256, 40).to(cuda)
    row_of = torch.full((5, 2), -1, dtype=torch.int32, device=cuda)
    row_of[1, 0], row_of[3, 1], row_of[4, 0] = 3, 200, 10 ** 6  # the last is outside Z
    buf = torch.full((5, 50), 8.0, device=cuda)
    y = mao.expert_combine(z[:, 3:33], row_of, out=buf[:, 5:35])
    want = torch.zeros(5, 30, device=cuda)
    want[1], want[3] = z[3, 3:33], z[200, 3:33]
    assert torch.equal(y, want) and (buf[:, :5] == 8).all() and (buf[:, 35:] == 8).all()


# ------------------------------------------------------------------------------ refusals


def test_overlapping_rows_are_refused(cuda):
    """A row repeated by a stride of 0 is not a matrix in memory."""
    row = torch.zeros(1, 32, device=cuda).expand(8, 32)
    slots = torch.zeros(8, dtype=torch.int32, device=cuda)
    places = torch.zeros(8, 1, dtype=torch.int32, device=cuda)
    with pytest.raises(ValueError):
        mao.fp8_quantize(row, "row")
    with pytest.raises(ValueError):
        mao.fp8_quantize(row[None].expand(2, 8, 32), "row")
    with pytest.raises(ValueError):
        mao.fp8_quantize(torch.zeros(2, 1, 32, device=cuda).expand(2, 8, 32), "row")
    with pytest.raises(ValueError):
        mao.expert_route(row, 2)
    with pytest.raises(ValueError):
        mao.expert_combine_backward(row, torch.zeros(8, 32, device=cuda), places, slots)
    with pytest.raises(ValueError):
        mao.apply_update(torch.zeros(8, 32, device=cuda), 0.1, U=row)


def test_refusals(cuda):
    x = torch.zeros(4, 32, device=cuda)
    codes, scales = mao.fp8_quantize(x, "row")
    wc, ws = mao.fp8_quantize(x[None], "tile")
    with pytest.raises(ValueError):
        mao.fp8_quantize(x, "blocks")
    with pytest.raises(ValueError):
        mao.fp8_quantize(x.cpu(), "row")
    with pytest.raises(ValueError):
        mao.fp8_quantize(x.half(), "row")
    with pytest.raises(ValueError):
        mao.fp8_product(codes, scales[:, :0], wc, ws, "nt")
    with pytest.raises(ValueError):
        mao.fp8_product(codes, scales, wc, ws, "tt")
    with pytest.raises(mao.MaoError):
        mao.fp8_product(codes, scales, *mao.fp8_quantize(torch.zeros(1, 4, 48, device=cuda), "tile"), "nt")
    with pytest.raises(mao.MaoError):  # two groups need two matrices
        mao.fp8_product(codes, scales, wc, ws, "nt",
                        offsets=torch.zeros(3, dtype=torch.int32, device=cuda))
    with pytest.raises(mao.MaoError):  # rows of codes are 16-byte aligned
        mao.fp8_product(torch.zeros(4, 33, dtype=torch.uint8, device=cuda)[:, 1:], scales, wc, ws, "nt")
    with pytest.raises(mao.MaoError):
        mao.expert_route(x, 33)
    with pytest.raises(mao.MaoError):
        mao.expert_route(x, 5, groups=8, keep_groups=1)
    with pytest.raises(mao.MaoError):
        mao.expert_route(torch.zeros(2, 1025, device=cuda), 2)
    with pytest.raises(ValueError):
        mao.expert_plan(torch.zeros(4, 2, device=cuda), 4)
    with pytest.raises(mao.MaoError):
        mao.expert_combine(x, torch.zeros(2, 33, dtype=torch.int32, device=cuda))
