"""Feed-forward calls with as many runs of rows as they take (1024), or nearly: the last runs' tokens are
in the outputs, and every other row is zero. Bounds as in test_gpu_ffn; products bit by bit."""

import numpy as np
import pytest
import torch

import matrix_aware_optimizers_gb300 as mao
from oracle import ffn as of
from test_gpu_ffn import check_backward, check_forward, make
from test_gpu_int8 import codes, want_product

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
GROUPS = [1021, 1023, 1024]
K, N, C = 40, 24, 32


def nan(*shape, dtype=BF16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def spoiled(nbytes):
    return torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")


def some_counts(groups, copies):
    """Tokens of a few runs, the last one among them; of sixteen or more it has nine, more than a pass takes."""
    cnt = [0] * groups
    cnt[-1] = 9 if copies >= 16 else 1
    for i in range(copies - cnt[-1]):
        cnt[i * (groups - 2) // copies] += 1
    assert sum(cnt) == copies
    return cnt


def padded(cnt):
    return np.concatenate([[0], np.cumsum([(c + 127) // 128 * 128 for c in cnt])])


def check_unused(rows, off, cnt, *tensors):
    used = torch.zeros(rows, dtype=torch.bool)
    for lo, hi in of.runs(rows, off, cnt):
        used[lo:hi] = True
    for t in tensors:
        assert (t[~used.to(t.device)] == 0).all()


def check_calls(cuda, groups, off, cnt, rows):
    kw = dict(offsets=torch.tensor(off, dtype=I32, device=cuda),
              counts=None if cnt is None else torch.tensor(cnt, dtype=I32, device=cuda))
    x, up, down, _ = make(groups, rows, K, N, C, groups=groups)
    y, z = mao.gated_ffn(x, up, down, "silu", out=nan(rows, C), Z=nan(rows, 2 * N, dtype=F32),
                         ws=spoiled(mao.gated_ffn_workspace_bytes(x, up, down, groups)), **kw)
    a, sa = codes(1, rows, K)
    b, sb = codes(2, groups, N, K)
    p = mao.int8_product(a, sa, b, sb, out=nan(rows, N, dtype=F32),
                         ws=spoiled(mao.int8_product_workspace_bytes(a, sa, b, sb, grouped=True)), **kw)
    mao.sync_status()
    check_forward(y, z, x, up, down, "silu", off, cnt)
    assert torch.equal(p.cpu(), want_product(a, sa, b, sb, F32, off, cnt))
    check_unused(rows, off, cnt, y, z, p)


@pytest.mark.parametrize("copies", [1, 8, 16, 24])
@pytest.mark.parametrize("groups", GROUPS)
def test_few_rows(cuda, groups, copies):
    cnt = some_counts(groups, copies)
    off = padded(cnt)
    assert off[-1] <= 2048
    check_calls(cuda, groups, off.tolist(), cnt, int(off[-1]))


@pytest.mark.parametrize("groups", GROUPS)
def test_tiles(cuda, groups):
    """Runs that follow one another without gaps, one row in two of them, more in the last."""
    off = (np.arange(groups + 1) // 2).tolist()
    off[-1] += 300
    check_calls(cuda, groups, off, None, off[-1] + 5)


@pytest.mark.parametrize("groups", GROUPS)
def test_tiles_of_counted_rows(cuda, groups):
    """More rows than the few rows' kernel takes: tiles, over runs with padding."""
    cnt = some_counts(groups, 8)
    cnt[-1], cnt[0], cnt[7] = 300, 129, 1000
    off = padded(cnt)
    assert off[-1] > 2048
    check_calls(cuda, groups, off.tolist(), cnt, int(off[-1]) + 128)


@pytest.mark.parametrize("use_counts", [False, True])
@pytest.mark.parametrize("groups", GROUPS)
def test_gradients(cuda, groups, use_counts):
    cnt = some_counts(groups, 16)
    off = padded(cnt).tolist()
    rows, counts = off[-1], cnt if use_counts else None
    kw = dict(offsets=torch.tensor(off, dtype=I32, device=cuda),
              counts=torch.tensor(cnt, dtype=I32, device=cuda) if use_counts else None)
    x, up, down, dy = make(groups, rows, K, N, C, groups=groups)
    y, z = mao.gated_ffn(x, up, down, "gelu", save=True, **kw)
    check_forward(y, z, x, up, down, "gelu", off, counts)
    outs = dict(dX=nan(rows, K), dup=nan(groups, 2 * N, K), ddown=nan(groups, C, N))
    grads = mao.gated_ffn_backward(dy, x, up, down, z, "gelu", **outs, **kw)
    mao.sync_status()
    check_backward(grads, dy, x, up, down, z, "gelu", off, counts)
    check_unused(rows, off, counts, grads[0])


FALLING = [([0, 300, 100, 400], [200, 50, 100]), ([-9, 128, 500, 90, 90, 700], [3, 128, 300, 90, 1000]),
           ([60, 50, 40, 3000, 2800, 3100], [7, 7, 2000, 40, 90]), ([0, 40, 20, 200, 150, 300], [9, 1, 150, 60, 100])]


@pytest.mark.parametrize("off,cnt", FALLING)
def test_counted_runs_of_falling_offsets(cuda, off, cnt):
    """Offsets that fall are raised to the largest before them, by every part of a call: what the
    workspace held before is in no output. The last case is one of few rows."""
    check_calls(cuda, len(cnt), off, cnt, max(off) - (20 if len(cnt) == 5 else 0))
