"""Expert-layer operators at the ends of their ranges, against the fp64 oracle.

u = 2^-23 bounds fp32's roundings: a softmax over E experts, its sums and the few products and
divisions after it are within (E + 64) u of their terms' magnitudes.
"""

import numpy as np
import pytest
import torch

import matrix_aware_optimizers_gb300 as mao
from oracle import experts as ox

pytestmark = pytest.mark.gpu

U23 = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------------------ routing


@pytest.mark.parametrize("top_k", [1, 2, 3])
def test_route_gradient_of_experts_of_tiny_probability(cuda, top_k):
    """A bias chooses experts whose scores are as small as the 1e-20 of the weights'
    denominator: then the weights do depend on the sum of the scores."""
    low = -np.log(10.0) * np.array([18, 19, 19.5, 20, 20.5, 21, 22])
    x = np.zeros((7, 12), np.float32)
    x[:, 0], x[:, 1] = 1.0, -2.0
    for t in range(7):
        x[t, 2:9] = np.roll(low, t)
    x[:, 9:] = -30.0
    bias = np.zeros(12, np.float32)
    bias[2:5] = [8.0, 6.0, 4.0]
    g = np.random.default_rng(top_k).normal(size=(7, top_k)).astype(np.float32)
    X, G = torch.from_numpy(x).to(cuda), torch.from_numpy(g).to(cuda)
    w, ids = mao.expert_route(X, top_k, bias=torch.from_numpy(bias).to(cuda), scale=1.5)
    assert ids.tolist() == [list(range(2, 2 + top_k))] * 7
    ww, _, _ = ox.route(x, top_k, bias=bias, scale=1.5)
    assert (np.abs(np64(w) - ww) <= (12 + 64) * U23 * ww).all()
    d = np64(mao.expert_route_backward(X, ids, G, scale=1.5))
    want = ox.route_backward(x, ids.cpu().numpy(), g, scale=1.5)
    s = ox.scores(x, "softmax")
    chosen = np.zeros_like(s)
    chosen[:, 2:2 + top_k] = 1.0
    total = (s * chosen).sum(1, keepdims=True) + 1e-20
    size = 1.5 * np.abs(g).sum(1, keepdims=True)
    # s_j (ds_j - dot) of the chosen, s_i dot of the others, with dot = mean 1e-20 / total
    tol = (12 + 64) * U23 * s * size / total * np.where(chosen > 0, 1.0, 1e-20)
    assert (np.abs(d - want) <= tol + 1e-37).all(), np.abs(d - want).max()
    assert np.abs(want[:, 0]).min() > 1e-4  # the expert that was not chosen has a gradient


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_sigmoid_far_below_zero(cuda, dtype):
    """Scores down to fp32's smallest numbers, in the order of the logits. An exponential (2 units
    in the last place), a sum and a quotient (2 more): 5 u, and below 2^-126 units of 2^-149."""
    x = torch.arange(-100.0, -68.0, 0.5)[torch.randperm(64, generator=torch.Generator().manual_seed(1))]
    x = x.view(2, 32).to(dtype)  # halves below 128 are exact in bf16
    want = ox.scores(np64(x), "sigmoid")
    for opts in (dict(groups=2, keep_groups=2), dict(bias=torch.zeros(32, device=cuda)), {}):
        w, ids = mao.expert_route(x.to(cuda), 32, score="sigmoid", renorm=False, **opts)
        order = np.argsort(-np64(x), 1)
        np.testing.assert_array_equal(ids.cpu().numpy(), order)
        s = np.take_along_axis(want, order, 1)
        assert (np.abs(np64(w) - s) <= 5 * U23 * s + 2 * 2.0 ** -149).all()


# ------------------------------------------------------------------------------ products


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off", [[200, 456, 600], [700, 700, 700], [1, 1, 2]])
def test_product_rows_before_the_first_group_are_zero(cuda, form, dtype, off):
    """They belong to no group, like the rows past the last; with accumulate both stay."""
    g = torch.Generator().manual_seed(off[0])
    a, b = torch.randn(700, 200, generator=g).to(cuda), torch.randn(2, 200, 200, generator=g).to(cuda)
    A, B = mao.fp8_quantize(a, "row"), mao.fp8_quantize(b, "tile")
    o = torch.tensor(off, dtype=torch.int32, device=cuda)
    alone = mao.fp8_product(*A, *B, form, offsets=torch.tensor([0] + off[1:], dtype=torch.int32, device=cuda),
                            out_dtype=dtype)
    y = torch.full((700, 200), 7.0, dtype=dtype, device=cuda)
    z = y.clone()
    mao.fp8_product(*A, *B, form, offsets=o, out=y)
    mao.fp8_product(*A, *B, form, offsets=o, out=z, accumulate=True)
    mao.sync_status()
    lo, hi = off[0], off[-1]
    assert torch.equal(y[lo:hi], alone[lo:hi])
    assert (y[:lo] == 0).all() and (y[hi:] == 0).all()
    assert (z[:lo] == 7).all() and (z[hi:] == 7).all()


@pytest.mark.parametrize("form", ["nt", "nn"])
def test_product_of_the_most_rows(cuda, form):
    """2^31 - 1024 rows, in more tiles than fit beside them in 32 bits: rows here and there against
    the oracle's values, all others zero."""
    R = 2 ** 31 - 1024
    free, _ = torch.cuda.mem_get_info()
    if free < 70e9:
        pytest.skip("needs 70 GB of device memory")
    A = torch.zeros(R, 16, dtype=torch.uint8, device=cuda)
    As = torch.full((R, 1), 127, dtype=torch.uint8, device=cuda)
    some = torch.tensor([0, 1, 255, 256, 2 ** 30 - 1, 2 ** 30, 2139127680, R - 257, R - 256, R - 1], device=cuda)
    A[some] = torch.arange(1, 17, dtype=torch.uint8, device=cuda) + 0x38 + some[:, None].to(torch.uint8) % 8
    B, Bs = mao.fp8_quantize(torch.arange(1.0, 3.0, device=cuda)[:, None].expand(2, 16).contiguous() if form == "nt"
                             else torch.arange(1.0, 3.0, device=cuda).expand(16, 2).contiguous(), "tile")
    y = mao.fp8_product(A, As, B, Bs, form, out_dtype=torch.bfloat16)
    mao.sync_status()
    v = np64(A[some].view(torch.float8_e4m3fn)).sum(1)[:, None] * np.array([1.0, 2.0])
    np.testing.assert_allclose(np64(y[some]), v, rtol=2.0 ** -8, atol=0)
    y[some] = 0
    for at in range(0, R, 2 ** 28):
        assert not y[at:at + 2 ** 28].any()


# ------------------------------------------------------------------------------ combination


@pytest.mark.parametrize("zt,yt", [("f32", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("H", [24, 770, 2056])
def test_combine_of_mixed_types(cuda, zt, yt, H):
    """Z, Y and the gradients each of its own type: one rounding, to the result's."""
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    T, k, E = 70, 5, 9
    g = torch.Generator().manual_seed(H)
    p = mao.expert_plan(torch.randint(-1, E, (T, k), generator=g).to(torch.int32).to(cuda), E)
    rows = p.slot_of.numel()
    z = torch.randn(rows, H, generator=g).to(dt[zt]).to(cuda)
    w = torch.randn(T, k, generator=g).to(cuda)
    dy = torch.randn(T, H, generator=g).to(dt[yt]).to(cuda)
    y = mao.expert_combine(z, p.row_of, w, out=torch.empty(T, H, dtype=dt[yt], device=cuda))
    row_of, wn = p.row_of.cpu().numpy(), w.cpu().numpy()
    step = {"f32": U23, "bf16": 2.0 ** -8}
    want, mag = ox.combine(np64(z), row_of, wn), ox.combine(np.abs(np64(z)), row_of, np.abs(wn))
    assert (np.abs(np64(y) - want) <= (k + 1) * U23 * mag + step[yt] * np.abs(want)).all()
    want_z, want_w = ox.combine_backward(np64(dy), np64(z), row_of, wn)
    _, mag = ox.combine_backward(np.abs(np64(dy)), np.abs(np64(z)), row_of, wn)
    for dzt in dt:
        dz, dw = mao.expert_combine_backward(dy, z, p.row_of, p.slot_of, w,
                                             dZ=torch.empty(rows, H, dtype=dt[dzt], device=cuda))
        mao.sync_status()
        assert (np.abs(np64(dz) - want_z) <= step[dzt] * np.abs(want_z)).all()
        assert (np.abs(np64(dw) - want_w) <= (H + 1) * U23 * mag).all()


# ------------------------------------------------------------------------------ graphs


def test_every_call_in_one_graph(cuda):
    """A layer's calls captured once: each replay works on what its inputs hold then, as the same
    calls outside the graph do."""
    T, H, N, E, k = 130, 256, 192, 8, 2
    g = torch.Generator(device="cuda")
    W8 = mao.fp8_quantize(torch.randn(E, N, H, generator=g.manual_seed(1), device=cuda), "tile")
    x = torch.empty(T, H, device=cuda)
    logits = torch.empty(T, E, device=cuda)
    dy = torch.empty(T, N, device=cuda)

    def fill(seed):
        for t in (x, logits, dy):
            t.copy_(torch.randn(t.shape, generator=g.manual_seed(seed), device=cuda))

    def layer():
        w, ids = mao.expert_route(logits, k)
        p = mao.expert_plan(ids, E)
        xr, xrs, xc, xcs = mao.fp8_quantize(x, "both", rows=p.slot_of, copies=k)
        z = mao.fp8_product(xr, xrs, *W8, "nt", offsets=p.offsets, out_dtype=torch.float32)
        y = mao.expert_combine(z, p.row_of, w)
        dz, dw = mao.expert_combine_backward(dy, z, p.row_of, p.slot_of, w)
        zr, zrs, zc, zcs = mao.fp8_quantize(dz, "both")
        dx = mao.expert_combine(mao.fp8_product(zr, zrs, *W8, "nn", offsets=p.offsets), p.row_of)
        dW = mao.fp8_product(zc, zcs, xc, xcs, "tn", offsets=p.offsets)
        return [w, ids, p.counts, p.offsets, p.row_of, p.slot_of, y, dx, dW,
                mao.expert_route_backward(logits, ids, dw)]

    fill(2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = layer()
    for seed in (3, 4, 5):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        want = layer()
        mao.sync_status()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ------------------------------------------------------------------------------ long tensors
#
# More than 2^31 entries: the last rows come out as in a call on them alone.

LONG = 1_050_240  # rows; a multiple of 256, and with 2048 columns or more past 2^31


def long_matrix(cols, dtype, seed, rows=LONG):
    free, _ = torch.cuda.mem_get_info()
    if free < 60e9:
        pytest.skip("needs 60 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(rows, cols, dtype=dtype, device="cuda")
    x.normal_(generator=g)
    assert x.numel() > 2 ** 31
    return x


@pytest.mark.parametrize("blocks", ["row", "col", "tile", "both"])
def test_quantize_of_many_entries(cuda, blocks):
    x = long_matrix(2048, torch.bfloat16, 1)
    out = mao.fp8_quantize(x, blocks)
    tail = mao.fp8_quantize(x[-256:], blocks)
    mao.sync_status()
    for a, b in zip(out, tail):
        assert torch.equal(a[-b.shape[0]:].view(torch.uint8), b.view(torch.uint8))
    if blocks in ("row", "both"):
        rows = torch.tensor([LONG - 1, 0, LONG - 5, -1, LONG], dtype=torch.int32, device=cuda)
        got = mao.fp8_quantize(x, "row", rows=rows)[0].view(torch.uint8)
        want = mao.fp8_quantize(x[[LONG - 1, 0, LONG - 5]], "row")[0].view(torch.uint8)
        assert torch.equal(got[:3], want) and not got[3:].any()


def test_route_of_many_entries(cuda):
    x = long_matrix(2 ** 8, torch.float32, 2, rows=8 * LONG)
    w, ids = mao.expert_route(x, 4)
    d = mao.expert_route_backward(x, ids, w, renorm=False)
    w2, ids2 = mao.expert_route(x[-100:], 4)
    mao.sync_status()
    assert torch.equal(w[-100:], w2) and torch.equal(ids[-100:], ids2)
    assert torch.equal(d[-100:], mao.expert_route_backward(x[-100:], ids2, w2, renorm=False))


def test_combine_of_many_entries(cuda):
    z = long_matrix(2056, torch.bfloat16, 3)
    row_of = torch.tensor([[LONG - 1, 7], [LONG - 300, -1], [0, LONG - 2]], dtype=torch.int32, device=cuda)
    w = torch.tensor([[0.5, 2.0], [1.5, 3.0], [0.25, 1.0]], device=cuda)
    y = mao.expert_combine(z, row_of, w)
    want = w[:, :1] * z[row_of[:, 0].long()].float() + w[:, 1:] * z[row_of[:, 1].clamp_min(0).long()].float()
    want[1] = 1.5 * z[LONG - 300].float()
    assert (y.float() - want).abs().le(2.0 ** -8 * want.abs() + 4 * U23 * 8).all()
    slot_of = torch.full((LONG,), -1, dtype=torch.int32, device=cuda)
    for t, j in ((0, 0), (0, 1), (1, 0), (2, 0), (2, 1)):
        slot_of[row_of[t, j].long()] = 2 * t + j
    dy = torch.randn(3, 2056, device=cuda).bfloat16()
    dz, dw = mao.expert_combine_backward(dy, z, row_of, slot_of, w)
    mao.sync_status()
    for t, j in ((0, 0), (0, 1), (1, 0), (2, 0), (2, 1)):
        r = int(row_of[t, j])
        assert torch.equal(dz[r], (w[t, j] * dy[t].float()).bfloat16())
        dz[r] = 0
        dot, mag = (dy[t].double() * z[r].double()).sum(), (dy[t].double() * z[r].double()).abs().sum()
        assert abs(float(dw[t, j]) - float(dot)) <= 2057 * U23 * float(mag)
    assert dw[1, 1] == 0
    for at in range(0, LONG, 65536):
        assert not dz[at:at + 65536].any()


@pytest.mark.parametrize("form", ["nt", "nn"])
def test_product_of_many_entries(cuda, form):
    free, _ = torch.cuda.mem_get_info()
    if free < 60e9:
        pytest.skip("needs 60 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(4)
    A = mao.fp8_quantize(torch.randn(LONG, 128, generator=g, device=cuda), "row")
    b = torch.randn(2050, 128, generator=g, device=cuda)
    B = mao.fp8_quantize(b if form == "nt" else b.T.contiguous(), "tile")
    y = mao.fp8_product(*A, *B, form)
    assert y.numel() > 2 ** 31
    tail = mao.fp8_product(A[0][-256:], A[1][-256:], *B, form)
    mao.sync_status()
    assert torch.equal(y[-256:], tail)


def test_weight_gradients_of_many_entries(cuda):
    free, _ = torch.cuda.mem_get_info()
    if free < 60e9:
        pytest.skip("needs 60 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(5)
    A = mao.fp8_quantize(torch.randn(256, 2048, generator=g, device=cuda), "col")
    B = mao.fp8_quantize(torch.randn(256, 2100, generator=g, device=cuda), "col")
    off = torch.zeros(513, dtype=torch.int32, device=cuda)
    off[300:], off[512:] = 128, 256  # group 299 has the first block, group 511 the second
    y = mao.fp8_product(*A, *B, "tn", offsets=off, out_dtype=torch.float32)
    assert y.numel() > 2 ** 31
    mao.sync_status()
    for e, lo in ((299, 0), (511, 128)):
        alone = mao.fp8_product(A[0][lo:lo + 128], A[1][lo // 128:lo // 128 + 1], B[0][lo:lo + 128],
                                B[1][lo // 128:lo // 128 + 1], "tn", out_dtype=torch.float32)
        assert torch.equal(y[e], alone[0])
        y[e] = 0
    for e in range(512):
        assert not y[e].any()
