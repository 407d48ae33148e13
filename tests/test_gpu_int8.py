"""8-bit integer rows and products on the GPU against the oracle.

Codes of plain rows are equal to the oracle's. Products of codes are exact and their fp32 sums
are whole numbers below 2^24 here, so the scaled outputs are equal, bit by bit. Gated rows: the
value's fp32 arithmetic is within 2^-20 of it (three roundings and CUDA's functions, each within
2 units), so a code is within 1/2 + 254 2^-20 of 127 x / a.
"""

import numpy as np
import pytest
import torch

import matrix_aware_optimizers_gb300 as mao
from oracle import ffn as of

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g)


def spread(seed, R, C):
    return randn(seed, R, C) * torch.exp(2 * randn(seed + 1, R, 1)) * torch.exp(randn(seed + 2, 1, C))


def check_rows(codes, scales, x):
    want, s = of.int8_rows(np64(x))
    np.testing.assert_array_equal(codes.cpu().numpy().astype(np.int64), want)
    np.testing.assert_array_equal(scales.cpu().numpy(), (np64(x).__abs__().max(1, initial=0).astype(np.float32) / np.float32(127)) if np.isfinite(s).all() else s.astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1), (1, 8), (3, 7), (5, 130), (400, 33), (64, 1024), (33, 1025), (20, 2048),
                                   (700, 4096), (9, 4104), (400, 8200), (2, 20000), (3, 16385), (1, 40001)])
def test_quantize(cuda, dtype, shape):
    x = spread(sum(shape), *shape).to(dtype).to(cuda)
    codes, scales = mao.int8_quantize(x)
    assert codes.dtype == torch.int8 and (codes.stride(0) % 16 == 0 or shape[0] == 1)
    check_rows(codes, scales, x)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_special_values(cuda, dtype):
    """Zeros, ties, the largest and the smallest numbers, and rows that are not finite."""
    x = torch.zeros(12, 300)
    x[1] = torch.arange(300) - 150.0
    x[2, :255] = torch.arange(255) / 2.0 - 63.5       # 127 x / 63.5: whole and halves
    x[2, 0] = 63.5
    x[3, :4] = torch.tensor([3.3e38, -1.7e38, 1.3e36, 1e-40])
    x[4, :5] = torch.tensor([1e-40, -2e-40, 3e-40, 1e-45, 0.0])
    x[5, :3] = torch.tensor([2.0 ** -126, 2.0 ** -127, -2.0 ** -126])
    x[6, 7] = -0.0
    x[10, 0] = 254.0                                  # ties of a row of whole numbers
    x[10, 1:254] = torch.arange(1, 254) * 1.0
    x = x.to(dtype).to(cuda)
    codes, scales = mao.int8_quantize(x)
    want, _ = of.int8_rows(np64(x))
    np.testing.assert_array_equal(codes.cpu().numpy().astype(np.int64), want)
    np.testing.assert_array_equal(scales.cpu().numpy(), x.abs().amax(1).float().cpu().numpy() / np.float32(127))
    x[7, 3], x[8, 299], x[9, 0] = float("nan"), float("inf"), -float("inf")
    codes, scales = mao.int8_quantize(x)
    assert scales[7:10].isnan().all() and (codes[7:10] == 0).all()
    np.testing.assert_array_equal(codes[:7].cpu().numpy().astype(np.int64), want[:7])


def test_quantize_ties_and_borders(cuda):
    """Values a few units to either side of every border between two codes."""
    a = torch.tensor([1.0, 1.7, 63.5, 1.2345e-7, 127.0, 2.0 ** 100 * 1.1])
    rows = []
    for v in a:
        b = ((torch.arange(-127, 127, dtype=torch.float64) + 0.5) / 127.0 * v.double()).float()
        row = [v[None]]
        for k in range(-3, 4):
            c = b
            for _ in range(abs(k)):
                c = torch.nextafter(c, torch.full_like(c, 1e38 if k > 0 else -1e38))
            row.append(c)
        rows.append(torch.cat(row))
    x = torch.stack(rows).to(cuda)
    codes, scales = mao.int8_quantize(x)
    check_rows(codes, scales, x)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_strides_and_stacks(cuda, dtype):
    big = spread(3, 200, 700).to(dtype).to(cuda)
    for c0, C in ((0, 300), (8, 256), (1, 257)):
        check_rows(*mao.int8_quantize(big[:, c0:c0 + C]), big[:, c0:c0 + C])
    s = torch.stack([spread(i, 30, 150) for i in range(5)]).to(dtype).to(cuda)
    for X in (s, list(s.unbind(0)), s[:, 1:, 3:], s[::2], [s[0], s[1, :, :].clone()]):
        codes, scales = mao.int8_quantize(X)
        for i, x in enumerate(X):
            check_rows(codes[i], scales[i], x)
    many = [spread(i, 20, 33).to(dtype).to(cuda) for i in range(70)]
    many[3] = torch.cat([many[3], many[3]], 1)[:, :33]  # another row stride
    codes, scales = mao.int8_quantize(many)
    for i in (0, 3, 63, 64, 69):
        check_rows(codes[i], scales[i], many[i])
    even = spread(4, 50, 704).to(dtype).to(cuda)  # aligned rows, widths that are no multiple of a load
    for C in (1, 3, 8, 33, 300, 699, 702, 704):
        check_rows(*mao.int8_quantize(even[:, :C]), even[:, :C])
    wide = torch.full((200, 320), 7, dtype=torch.int8, device=cuda)
    sc = torch.empty(200, device=cuda)
    mao.int8_quantize(big[:, :300], out=(wide[:, :300], sc))
    check_rows(wide[:, :300], sc, big[:, :300])
    assert (wide[:, 300:] == 7).all()
    none = mao.int8_quantize(big[:0])
    assert none[0].shape == (0, 700) and none[1].shape == (0,)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (40, 768), (5, 1030), (300, 2053), (2, 14336), (2, 9001)])
def test_quantize_gated(cuda, dtype, gate, shape):
    R, C = shape
    x = (randn(R + C, R, 2 * C) * 2).to(dtype).to(cuda)
    codes, scales = mao.int8_quantize(x, gate=gate)
    v = np64(x)
    h = of.act(v[:, :C], gate) * v[:, C:]
    a = np.abs(h).max(1)
    np.testing.assert_array_less(np.abs(scales.cpu().numpy() * 127.0 - a), 2.0 ** -19 * a + 1e-38)
    # 1 + erf and 1 + tanh round to 2^-24 of 1, not of the small sum: |g| |u| 2^-24 absolute
    slack = 0.5 + 127.0 * (2.0 ** -19 + 2.0 ** -22 * np.abs(v[:, :C] * v[:, C:]) / a[:, None])
    np.testing.assert_array_less(np.abs(codes.cpu().numpy() - 127.0 * h / a[:, None]), slack)
    # the arithmetic as documented, step by step, in torch's own fp32 operations
    g, u = x[:, :C].float(), x[:, C:].float()
    if gate == "silu":
        w = g / (1.0 + torch.exp(-g)) * u
    elif gate == "gelu":
        w = 0.5 * g * (1.0 + torch.erf(g * 0.5 ** 0.5)) * u
    else:
        w = 0.5 * g * (1.0 + torch.tanh((2.0 / np.pi) ** 0.5 * (g + 0.044715 * g * g * g))) * u
    check_rows(codes, scales, w)


@pytest.mark.parametrize("gate", ["silu", "gelu", "gelu_tanh"])
def test_quantize_gated_in_doubt(cuda, gate):
    """Rows in which many values come near to the largest or to borders, and rows near the ends of fp32's
    range: the codes are those of the documented arithmetic."""
    C = 1536
    g = randn(1, 12, C) * 3
    u = randn(2, 12, C)
    g[0], u[0] = 1.25, 0.75                              # one value throughout
    g[1], u[1] = torch.linspace(1.0, 1.0001, C), 1.0     # all near the largest
    g[2] = -6.0 - randn(3, C).abs()                          # small gates of large factors
    g[3] = -30.0 - 25.0 * randn(4, C).abs()                  # next to nothing
    g[4], u[4] = g[4] * 1e-22, u[4] * 1e-22              # products below fp32's range
    g[5], u[5] = g[5].abs() * 1e18, u[5] * 1e18          # and near its other end
    g[6] *= 40.0
    u[7] = 0.0
    g[8] = 0.0
    g[9] = 2.0                                           # whole and half multiples of one value
    u[9] = torch.randint(-254, 255, (C,), generator=torch.Generator().manual_seed(3)) / 2.0
    g[10, ::2] = -200.0
    x = torch.cat([g, u], 1)
    for dtype in (F32, BF16):
        xx = x.to(dtype).to(cuda)
        a, b = xx[:, :C].float(), xx[:, C:].float()
        if gate == "silu":
            w = a / (1.0 + torch.exp(-a)) * b
        elif gate == "gelu":
            w = 0.5 * a * (1.0 + torch.erf(a * 0.5 ** 0.5)) * b
        else:
            w = 0.5 * a * (1.0 + torch.tanh((2.0 / np.pi) ** 0.5 * (a + 0.044715 * a * a * a))) * b
        check_rows(*mao.int8_quantize(xx, gate=gate), w)


def test_quantize_gated_extremes(cuda):
    x = torch.tensor([[200.0, -200.0, 0.0, 1.0, 3.0, 5.0, -2.0, 0.25],
                      [1e20, 1.0, 1.0, 1.0, 1e20, 1.0, 1.0, 1.0],
                      [float("inf"), 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0]], device=cuda)
    for gate in ("silu", "gelu", "gelu_tanh"):
        codes, scales = mao.int8_quantize(x, gate=gate)
        want, s = of.int8_rows(of.act(np64(x[:1, :4]), gate) * np64(x[:1, 4:]))
        np.testing.assert_array_equal(codes[:1].cpu().numpy(), want)
        assert scales[1:].isnan().all() and (codes[1:] == 0).all()  # beyond fp32's range


# ------------------------------------------------------------------------------- products


def codes(seed, *shape, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    ld = -(-shape[-1] // 16) * 16
    c = torch.randint(-127, 128, (*shape[:-1], ld), generator=g, dtype=torch.int8).to(device)
    return c[..., :shape[-1]], torch.exp(torch.randn(shape[:-1], generator=g)).to(device)


def want_product(a, sa, b, sb, dtype, offsets=None, counts=None):
    """Scaled and rounded as documented: the sum is a whole number below 2^24."""
    A, B = a.cpu().numpy().astype(np.float64), b.cpu().numpy().astype(np.float64)
    SA, SB = sa.cpu().numpy(), sb.cpu().numpy()
    if B.ndim == 2:
        B, SB = B[None], SB[None]
    y = np.zeros((len(A), B.shape[1]), np.float32)
    for g, (lo, hi) in enumerate(of.runs(len(A), offsets, counts)):
        s = A[lo:hi] @ B[g].T
        assert np.abs(s).max(initial=0) < 2 ** 24
        y[lo:hi] = s.astype(np.float32) * SA[lo:hi, None] * SB[g][None]
    return torch.from_numpy(y).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 16, 64), (3, 5, 7), (16, 256, 128), (31, 33, 100), (64, 64, 1040),
                                   (129, 255, 129), (256, 256, 256), (257, 513, 300), (600, 770, 520)])
def test_product(cuda, dtype, shape):
    T, N, K = shape
    a, sa = codes(T, T, K)
    b, sb = codes(N + 1000, N, K)
    y = mao.int8_product(a, sa, b, sb, out_dtype=dtype)
    mao.sync_status()
    assert torch.equal(y.cpu(), want_product(a, sa, b, sb, dtype))


@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 15, 16, 17, 40, 100, 128, 200])
def test_product_few_rows(cuda, T):
    """Few rows and long sums, which are split."""
    a, sa = codes(T, T, 4000)
    b, sb = codes(5, 1100, 4000)
    for dtype in (F32, BF16):
        y = mao.int8_product(a, sa, b, sb, out_dtype=dtype)
        assert torch.equal(y.cpu(), want_product(a, sa, b, sb, dtype))


def test_product_few_rows_in_runs(cuda):
    """Runs of no, one, two and more rows, side by side; a depth that ends inside a load."""
    cnt = [0, 1, 2, 3, 1, 8, 9, 2, 0, 17, 1, 2]
    off = [96 * i for i in range(13)]
    for N, K in ((300, 700), (40, 16), (528, 2064)):
        a, sa = codes(13, 96 * 12, K)
        b, sb = codes(14, 12, N, K)
        y = mao.int8_product(a, sa, b, sb, offsets=torch.tensor(off, dtype=I32, device=cuda),
                             counts=torch.tensor(cnt, dtype=I32, device=cuda), out_dtype=F32)
        mao.sync_status()
        assert torch.equal(y.cpu(), want_product(a, sa, b, sb, F32, off, cnt))


def test_product_exact_at_the_limit(cuda):
    """Sums of the largest codes are exact up to 2^24: 1040 products of 127 * 127 (codes of
    int8_quantize), 1024 of 128 * 128 (any codes)."""
    one = lambda n: torch.ones(n, device=cuda)  # noqa: E731
    for K, x, z in ((1040, 127, 127), (1040, -127, 127), (1024, -128, -128), (1024, 127, -128)):
        a = torch.full((40, K), x, dtype=torch.int8, device=cuda)
        b = torch.full((300, K), z, dtype=torch.int8, device=cuda)
        b[:, 1] += 1 if z < 0 else -1
        y = mao.int8_product(a, one(40), b, one(300), out_dtype=F32)
        assert (y == float(x * (z * K + (1 if z < 0 else -1)))).all()
    # 1039 of 127 * -128 and one of 127 * 127: 16,873,855 is odd and above 2^24, where fp32 holds even
    # numbers only; the two sums at the end that pass 2^24 may each be cut by less than 2
    a = torch.full((40, 1040), 127, dtype=torch.int8, device=cuda)
    b = torch.full((300, 1040), -128, dtype=torch.int8, device=cuda)
    b[:, 1] = 127
    y = mao.int8_product(a, one(40), b, one(300), out_dtype=F32)
    assert ((y.double() - 127.0 * (-128.0 * 1039 + 127)).abs() <= 4).all()


@pytest.mark.parametrize("use_counts", [False, True])
@pytest.mark.parametrize("off,cnt,rows", [([0, 128, 128, 384, 512], [100, 0, 256, 1], 512),
                                          ([3, 40, 41, 300, 690], [30, 1, 200, 390], 700)])
@pytest.mark.parametrize("dims", [(48, 80), (300, 520), (33, 77)])
def test_product_runs(cuda, off, cnt, rows, use_counts, dims):
    N, K = dims
    a, sa = codes(1, rows, K)
    b, sb = codes(2, 4, N, K)
    counts = cnt if use_counts else None
    y = mao.int8_product(a, sa, b, sb, offsets=torch.tensor(off, dtype=I32, device=cuda),
                         counts=torch.tensor(cnt, dtype=I32, device=cuda) if use_counts else None)
    mao.sync_status()
    assert torch.equal(y.cpu(), want_product(a, sa, b, sb, BF16, off, counts))


def test_product_many_tiles(cuda):
    """More tiles than pairs of SMs: accumulators follow one another, of all heights."""
    for T in (2100, 5000):
        a, sa = codes(T, T, 200)
        b, sb = codes(9, 4100, 200)
        assert torch.equal(mao.int8_product(a, sa, b, sb).cpu(), want_product(a, sa, b, sb, BF16))
    off = list(range(0, 128 * 65, 128))
    g = torch.Generator().manual_seed(1)
    cnt = torch.randint(0, 129, (64,), generator=g).tolist()
    a, sa = codes(10, 128 * 64, 144)
    b, sb = codes(11, 64, 400, 144)
    y = mao.int8_product(a, sa, b, sb, offsets=torch.tensor(off, dtype=I32, device=cuda),
                         counts=torch.tensor(cnt, dtype=I32, device=cuda))
    assert torch.equal(y.cpu(), want_product(a, sa, b, sb, BF16, off, cnt))


def test_product_runs_of_all_heights(cuda):
    """Tiles of up to 128 rows and higher ones follow one another in each pair of SMs; the depth ends in
    the first half of a stage, or in the second."""
    g = torch.Generator().manual_seed(2)
    cnt = torch.randint(0, 400, (90,), generator=g).tolist()
    off = [0]
    for n in cnt:
        off.append(off[-1] + (n + 15) // 16 * 16)
    for K in (700, 736):
        a, sa = codes(K, off[-1], K)
        b, sb = codes(12, 90, 520, K)
        y = mao.int8_product(a, sa, b, sb, offsets=torch.tensor(off, dtype=I32, device=cuda),
                             counts=torch.tensor(cnt, dtype=I32, device=cuda))
        mao.sync_status()
        assert torch.equal(y.cpu(), want_product(a, sa, b, sb, BF16, off, cnt))


def test_product_outputs_and_nan(cuda):
    a, sa = codes(1, 50, 96)
    b, sb = codes(2, 60, 96)
    want = want_product(a, sa, b, sb, BF16).to(cuda)
    for left in (1, 2):
        big = torch.full((50, 64 + left), 7.0, dtype=BF16, device=cuda)
        out = mao.int8_product(a, sa, b, sb, out=big[:, left:left + 60])
        assert torch.equal(out, want) and (big[:, :left] == 7).all() and (big[:, left + 60:] == 7).all()
    sa[3], sb[7] = float("nan"), float("nan")
    y = mao.int8_product(a, sa, b, sb)
    bad = torch.zeros(50, 60, dtype=torch.bool, device=cuda)
    bad[3], bad[:, 7] = True, True
    assert torch.equal(y.isnan(), bad) and torch.equal(y[~bad], want[~bad])
    assert mao.int8_product(a[:0], sa[:0], b, sb).shape == (0, 60)


def test_served_block(cuda):
    """Weights and rows quantised, the gate between the products, against the block's formula on the
    values that the codes stand for."""
    T, K, N = 70, 256, 160
    x = randn(1, T, K).to(BF16).to(cuda)
    up, down = (randn(2, 2 * N, K) * K ** -0.5).to(cuda), (randn(3, K, N) * N ** -0.5).to(cuda)
    u8, us = mao.int8_quantize(up)
    d8, ds = mao.int8_quantize(down)
    x8, xs = mao.int8_quantize(x)
    z = mao.int8_product(x8, xs, u8, us, out_dtype=F32)
    h8, hs = mao.int8_quantize(z, gate="silu")
    y = mao.int8_product(h8, hs, d8, ds, out_dtype=F32)
    mao.sync_status()
    val = lambda c, s: np64(c) * np64(s)[:, None]  # noqa: E731
    # sums of codes first: whole numbers, exact in 64 bits too (sums of scaled values are not: where
    # the codes' sum is 0 they leave some 2^-53)
    prod = lambda a, sa, b, sb: (np64(a) @ np64(b).T) * np64(sa)[:, None] * np64(sb)  # noqa: E731
    zz = prod(x8, xs, u8, us)
    np.testing.assert_allclose(np64(z), zz, rtol=2.0 ** -21, atol=0)  # three roundings
    h = of.act(np64(z)[:, :N], "silu") * np64(z)[:, N:]
    # a code is off by half a step and what the gate's arithmetic adds
    step = np.abs(h).max(1, keepdims=True) / 127.0
    assert (np.abs(val(h8, hs) - h) <= 0.5001 * step + 1e-30).all()
    np.testing.assert_allclose(np64(y), prod(h8, hs, d8, ds), rtol=2.0 ** -21, atol=0)
