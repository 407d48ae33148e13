"""Feed-forward calls at the ends of their range."""

import numpy as np
import pytest
import torch

import matrix_aware_optimizers_gb300 as mao

pytestmark = pytest.mark.gpu

F32 = torch.float32


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
