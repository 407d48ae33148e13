"""8-bit products in which every pair of CTAs takes several tiles, bit by bit.

Codes are small whole numbers and scales 1/2, 1 or 2, so every product is a multiple of 1/4 and at
most 16, and every partial sum of up to 2^12 of them is below 2^16 in steps of 2^-2: 18 bits, so
fp32 holds each one exactly in any order, and the fp32 result has to be equal. A bf16 result is
that value rounded to nearest even once, so it has to be equal too. Sums over more terms (the
split ones) keep below 2^18: 20 bits.
"""

import pytest
import torch

import matrix_aware_optimizers_gb300 as mao

pytestmark = pytest.mark.gpu

OUT = {"f32": torch.float32, "bf16": torch.bfloat16}


def operand(g, rows, cols, blocks, count=None):
    """Codes and scale bytes as fp8_quantize lays them out, and their values in fp64."""
    n = 1 if count is None else count
    v = torch.randint(-2, 3, (n, rows, cols), generator=g, device="cuda")
    codes = torch.zeros(n, rows, -(-cols // 16) * 16, dtype=torch.float8_e4m3fn, device="cuda")
    codes[:, :, :cols] = v.to(torch.float32).to(torch.float8_e4m3fn)
    codes = codes[:, :, :cols]
    br, bc = {"row": (1, 128), "col": (128, 1), "tile": (128, 128)}[blocks]
    e = torch.randint(-1, 2, (n, -(-rows // br), -(-cols // bc)), generator=g, device="cuda")
    f = torch.exp2(e.double()).repeat_interleave(br, 1).repeat_interleave(bc, 2)
    v = v.double() * f[:, :rows, :cols]
    s = (e + 127).to(torch.uint8)
    return (codes[0], s[0], v[0]) if count is None else (codes, s, v)


def case(form, rows, n, k, sizes, seed):
    """Operands of a product, its offsets and its value in fp64."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    tn = form == "tn"
    A, As, a = operand(g, rows, k if form == "nt" else n, "col" if tn else "row")
    off = [0, rows] if sizes is None else [0] + torch.tensor(sizes).cumsum(0).tolist()
    if tn:
        B, Bs, b = operand(g, rows, k, "col")
        want = torch.stack([a[lo:hi].T @ b[lo:hi] for lo, hi in zip(off[:-1], off[1:])])
    else:
        B, Bs, b = operand(g, n, k, "tile", len(off) - 1)
        want = torch.zeros(rows, n if form == "nt" else k, dtype=torch.float64, device="cuda")
        for i, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
            want[lo:hi] = a[lo:hi] @ (b[i].T if form == "nt" else b[i])
    o = None if sizes is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    return (A, As, B, Bs, form), o, want


def check(args, offsets, want, out):
    dtype = OUT[out]
    exact = want.float().to(dtype)
    assert want.float().double().equal(want)
    # several launches in a row, each on its own output, then all looked at
    got = [mao.fp8_product(*args, offsets=offsets, out_dtype=dtype) for _ in range(3)]
    mao.sync_status()
    for y in got:
        assert torch.equal(y.view(exact.shape), exact), int((y.view(exact.shape) != exact).sum())
    # added to what is there
    base = torch.randint(-9, 10, want.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    y = base.to(dtype)
    mao.fp8_product(*args, offsets=offsets, out=y, accumulate=True)
    mao.sync_status()
    assert torch.equal(y, (want + base).float().to(dtype))


def pairs():
    return torch.cuda.get_device_properties(0).multi_processor_count // 2


def tiles(n, of=256):
    return -(-n // of)


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("depth", [100, 200, 640, 2570])
def test_dense_products_of_many_tiles(cuda, form, out, depth):
    """21 tiles of rows (bands of 8, 8 and 5) by 11 or more of columns; one, two, five and
    twenty-one blocks of depth."""
    R, C = 5200, 2700 if depth < 2570 else 2640
    assert tiles(R) * tiles(C) > 3 * pairs()
    n, k = (C, depth) if form == "nt" else (depth, C)
    check(*case(form, R, n, k, None, depth), out)


# a group of up to 256 rows is one tile; 300 rows are tiles of 160 and 140, 440 and 650 of 224, 513
# of 192, and 512 and 2100 (nine tiles: two bands) of 256
MIXED = [128, 300, 256, 0, 512, 224, 0, 440, 650, 2100, 30, 1, 513, 0]


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("depth", [100, 136, 700, 2570])
def test_groups_of_many_tiles(cuda, form, out, depth):
    """Groups of mixed heights above and below 224 rows, some empty, with rows past the last."""
    sizes, C = MIXED * 2, 1300
    assert sum(tiles(s) for s in sizes) * tiles(C) > 3 * pairs()
    n, k = (C, depth) if form == "nt" else (depth, C)
    check(*case(form, sum(sizes) + 77, n, k, sizes, depth + 1), out)


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("size", [224, 256])
@pytest.mark.parametrize("depth", [128, 600])
def test_groups_of_one_height(cuda, form, size, depth):
    """All tiles just without, or all with, the columns that two accumulators share."""
    sizes = [size] * 60
    n, k = (1030, depth) if form == "nt" else (depth, 1030)
    assert 60 * tiles(1030) > 3 * pairs()
    check(*case(form, sum(sizes), n, k, sizes, size + depth), "f32")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[128, 0, 0, 256, 2560, 0, 384, 128, 1280, 0] * 6, [0, 128] * 40,
                                   [0] * 50 + [640] + [0] * 20 + [128, 512]])
def test_weight_gradients_of_many_tiles(cuda, out, sizes):
    """Groups of one to twenty blocks of depth between empty ones, whose matrices are zero."""
    n, k = (520, 600) if len(sizes) < 70 else (520, 360)
    assert len(sizes) * tiles(n) * tiles(k) > 3 * pairs()
    check(*case("tn", sum(sizes), n, k, sizes, len(sizes)), out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [100, 128, 1000])
def test_dense_weight_gradients_of_many_tiles(cuda, out, rows):
    n, k = 4100, 3900
    assert tiles(n) * tiles(k) > 3 * pairs()
    check(*case("tn", rows, n, k, None, rows), out)


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_split_sums(cuda, form, out):
    """Few outputs and a long sum, in parts that a second kernel adds up; ragged everywhere."""
    deep = 9003
    R, n, k = {"nt": (300, 270, deep), "nn": (300, deep, 270), "tn": (deep, 300, 270)}[form]
    args, o, want = case(form, R, n, k, None, 5)
    A, As, B, Bs, _ = args
    kinds = ("col", "col") if form == "tn" else ("row", "tile")
    assert mao.lib().fp8_product_workspace_bytes(
        mao.ctypes.byref(mao._fp8(A, As, kinds[0], "A")), mao.ctypes.byref(mao._fp8(B, Bs, kinds[1], "B")),
        {"nt": 0, "nn": 1, "tn": 2}[form]) > 0
    check(args, o, want, out)


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (5, 16, 300), (130, 257, 129), (257, 520, 136), (515, 264, 648)])
def test_small_products_exactly(cuda, form, shape):
    check(*case(form, *shape, None, sum(shape)), "f32")
