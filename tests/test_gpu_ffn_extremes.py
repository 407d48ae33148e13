"""Feed-forward calls at the ends of their range."""

import numpy as np
import pytest
import torch

import matrix_aware_optimizers_gb300 as mao
from oracle import ffn as of

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("K", [2 ** 20, 2 ** 20 - 16])
@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 16, 17])
def test_longest_sums_of_codes(cuda, T, K):
    """Sums of 2^14 over and over are exact in fp32 however they are added up; those of another product are
    where eight parts have 2^17 of it each. Of any codes: each of at most eight parts is rounded to
    fp32, and each of seven additions, within 2^-24 of the sum (all products are positive)."""
    N = 24
    one = lambda n: torch.ones(n, device=cuda)  # noqa: E731
    for a, b in ((-128, -128), (127, 127), (-127, 127), (127, -128), (-128, 127)):
        A = torch.full((T, K), a, dtype=torch.int8, device=cuda)
        B = torch.full((N, K), b, dtype=torch.int8, device=cuda)
        if a * b != 16384 and (T > 16 or K < 2 ** 20):
            continue  # (tiles add up in fp32 from the first product on)
        y = mao.int8_product(A, one(T), B, one(N), out_dtype=F32)
        assert (y == float(np.float32(a * b * K))).all(), (a, b)
    if T > 16:
        return
    g = torch.Generator(device=cuda).manual_seed(T)
    A = torch.randint(-128, -100, (T, K), generator=g, dtype=torch.int8, device=cuda)
    B = torch.randint(-128, -100, (N, K), generator=g, dtype=torch.int8, device=cuda)
    want = A.double() @ B.double().T  # whole numbers below 2^53
    y = mao.int8_product(A, one(T), B, one(N), out_dtype=F32)
    assert ((y.double() - want).abs() <= 8 * 2.0 ** -24 * (1 + 2.0 ** -20) * want).all()
    mao.sync_status()


@pytest.mark.parametrize("saved", [F32, BF16])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("C", [8, 4096])
def test_slopes_of_large_gates(cuda, act, C, saved):
    """Where G's square passes fp32's range, the slope is 1 or 0, and so is dG (C = 4096: a sum that is
    split, its epilogue a kernel of its own)."""
    G = [1e19, -1e19, 1e20, -1e20, 3e38, -3e38, 4.0, -4.0]
    z = torch.tensor([G + [1.0] * 8], dtype=saved, device=cuda)
    down = torch.zeros(C, 8, dtype=BF16, device=cuda)
    down[:8] = torch.eye(8)
    dy = torch.zeros(1, C, dtype=BF16, device=cuda)
    dy[:, :8] = 1.0  # dH = 1
    up = torch.zeros(16, 8, dtype=BF16, device=cuda)
    up[:8] = torch.eye(8)  # dX = dG
    x = torch.ones(1, 8, dtype=BF16, device=cuda)
    dX, dup, ddown = mao.gated_ffn_backward(dy, x, up, down, z, act, grad_dtype=F32)
    mao.sync_status()
    want = of.slope(np.array(G), act)
    assert want[:6].tolist() == [1.0, 0.0, 1.0, 0.0, 1.0, 0.0]
    # the slope's own arithmetic: 2^-19 of 1 + |g|; its rounding to bf16: 2^-8
    own = 2.0 ** -19 * 5
    slack = own + 2.0 ** -8 * (np.abs(want) + own)
    slack[:6] = 0.0
    assert (np.abs(dX[0].double().cpu().numpy() - want) <= slack).all()
    assert torch.equal(dup[:8, 0], dX[0])  # dG^T X
    assert torch.isfinite(dup).all() and torch.isfinite(ddown).all()


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_infinite_gates(cuda, act, T):
    """G = U = inf: H is infinite, and the sums multiply it by zero weights too: NaN. G = -inf: -inf times 0
    in the activation."""
    x = torch.zeros(T, 16, dtype=BF16, device=cuda)
    x[0, 0], x[1, 0], x[2:, 0] = float("inf"), float("-inf"), 2.0
    up = torch.zeros(16, 16, dtype=BF16, device=cuda)
    up[:, 0] = 1.0
    down = torch.eye(8, dtype=BF16, device=cuda)
    y = mao.gated_ffn(x, up, down, act, out_dtype=F32)
    mao.sync_status()
    assert y[:2].isnan().all() and torch.isfinite(y[2:]).all()
