"""Feed-forward calls in the ways a program makes them: on other streams, captured and replayed, two at
once, with workspaces of its own, with waits that run out, on tensors of more than 2^31 entries; and
a layer of experts trained and then served with them."""

import numpy as np
import pytest
import torch

import matrix_aware_optimizers_gb300 as mao
from matrix_aware_optimizers_gb300 import _abi
from oracle import ffn as of
from test_gpu_ffn import check_backward, check_forward, make, randn

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def step(x, up, down, dy, **kw):
    y, z = mao.gated_ffn(x, up, down, "silu", save=True, **kw)
    return (y,) + mao.gated_ffn_backward(dy, x, up, down, z, "silu", **kw)


def served(x, u8, us, d8, ds, **kw):
    x8, xs = mao.int8_quantize(x, **{k: v for k, v in kw.items() if k == "stream"})
    z = mao.int8_product(x8, xs, u8, us, **kw)
    h8, hs = mao.int8_quantize(z, gate="silu", **{k: v for k, v in kw.items() if k == "stream"})
    return mao.int8_product(h8, hs, d8, ds, **kw)


@pytest.mark.parametrize("T", [5, 300])
def test_another_stream(cuda, T):
    x, up, down, dy = make(1, T, 256, 200, 136)
    u8, us = mao.int8_quantize(up)
    d8, ds = mao.int8_quantize(down)
    want = step(x, up, down, dy) + (served(x, u8, us, d8, ds),)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(x, up, down, dy, stream=s) + (served(x, u8, us, d8, ds, stream=s),)
    mao.sync_status(s)
    with torch.cuda.stream(s):
        more = step(x, up, down, dy) + (served(x, u8, us, d8, ds),)
    s.synchronize()
    for a, b, c in zip(want, got, more):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("T", [3, 16, 500])
def test_captured_and_replayed(cuda, T):
    """Two graphs with private pools, replayed in turn with new inputs, give what eager calls give."""
    x, up, down, dy = make(2, T, 128, 96, 128)
    u8, us = mao.int8_quantize(up)
    d8, ds = mao.int8_quantize(down)
    run = lambda: step(x, up, down, dy) + (served(x, u8, us, d8, ds),)  # noqa: E731
    graphs, outs = [], []
    for _ in range(2):
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    for seed in range(3):
        x.copy_(randn(seed, *x.shape))
        dy.copy_(randn(seed + 9, *dy.shape))
        want = run()
        for g, o in zip(graphs, outs):
            for t in o:
                t.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(want, o):
                assert torch.equal(a, b)


def test_two_at_once(cuda):
    """Calls on two streams do not disturb one another."""
    sets = [make(s, T, 512, 384, 256) for s, T in ((3, 700), (4, 900))]
    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [step(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for a, b in zip(w, g):
                assert torch.equal(a, b)


def test_workspaces(cuda):
    """A workspace of the reported size does, one byte less is refused; it is clobbered, not read."""
    x, up, down, dy = make(5, 40, 2048, 512, 256)
    y0, z0 = mao.gated_ffn(x, up, down, "silu", save=True)
    g0 = mao.gated_ffn_backward(dy, x, up, down, z0, "silu")
    n = mao.gated_ffn_workspace_bytes(x, up, down)
    nb = mao.gated_ffn_backward_workspace_bytes(dy, x, up, down)
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=cuda)
        wb = torch.full((nb,), fill, dtype=torch.uint8, device=cuda)
        assert torch.equal(mao.gated_ffn(x, up, down, "silu", ws=ws), y0)
        for a, b in zip(mao.gated_ffn_backward(dy, x, up, down, z0, "silu", ws=wb), g0):
            assert torch.equal(a, b)
    short = torch.empty(n - 1, dtype=torch.uint8, device=cuda)
    with pytest.raises(mao.MaoError) as e:
        mao.gated_ffn(x, up, down, "silu", ws=short)
    assert e.value.status == _abi.MAO_ERR_WORKSPACE
    with pytest.raises(mao.MaoError) as e:
        mao.gated_ffn_backward(dy, x, up, down, z0, "silu", ws=torch.empty(nb - 1, dtype=torch.uint8, device=cuda))
    assert e.value.status == _abi.MAO_ERR_WORKSPACE
    with pytest.raises(mao.MaoError) as e:
        mao.gated_ffn(x, up, down, "silu", ws=torch.empty(n + 256, dtype=torch.uint8, device=cuda)[1:])
    assert e.value.status == _abi.MAO_ERR_MISALIGNED
    a8, as_ = mao.int8_quantize(x)
    b8, bs = mao.int8_quantize(up)
    p0 = mao.int8_product(a8, as_, b8, bs)
    m = mao.int8_product_workspace_bytes(a8, as_, b8, bs)
    for fill in (0, 255):
        assert torch.equal(mao.int8_product(a8, as_, b8, bs, ws=torch.full((m,), fill, dtype=torch.uint8, device=cuda)), p0)
    with pytest.raises(mao.MaoError) as e:
        mao.int8_product(a8, as_, b8, bs, ws=torch.empty(m - 1, dtype=torch.uint8, device=cuda))
    assert e.value.status == _abi.MAO_ERR_WORKSPACE


def test_waits_that_run_out(cuda):
    """A wait that gives up is reported by sync_status, and the next call is sound again."""
    x, up, down, dy = make(6, 600, 512, 384, 256)
    # few rows: weights larger than L2, so that loads are waited for (a wait that finds its load
    # complete is none, and four blocks' loads from L2 all are in time; so are now and then all
    # loads of the 8-bit product, whose warps take longer for a stage than memory does)
    g = torch.Generator(device=cuda).manual_seed(1)
    few = [torch.randn(*s, generator=g, device=cuda).to(BF16) for s in ((3, 8192), (16384, 8192), (64, 8192))]
    f8, fs = mao.int8_quantize(few[0])
    g8 = torch.randint(-127, 128, (40000, 8192), generator=g, device=cuda, dtype=torch.int8)
    gs = torch.ones(40000, device=cuda)
    a8, as_ = mao.int8_quantize(x)
    b8, bs = mao.int8_quantize(up)
    y0, z0 = mao.gated_ffn(x, up, down, save=True)
    calls = {"block": lambda: mao.gated_ffn(x, up, down), "few rows": lambda: mao.gated_ffn(*few),
             "gradients": lambda: mao.gated_ffn_backward(dy, x, up, down, z0)[0],
             "8-bit product": lambda: mao.int8_product(a8, as_, b8, bs),
             "8-bit product of few rows": lambda: mao.int8_product(f8, fs, g8, gs)}
    limit = mao.get_wait_limit()
    for name, call in calls.items():
        want = call()
        mao.sync_status()
        mao.set_wait_limit(0)
        try:
            for _ in range(100):
                got = call()
                try:
                    mao.sync_status()
                except mao.MaoError as e:
                    assert e.status == _abi.MAO_ERR_TIMEOUT, name
                    break
                assert torch.equal(got, want), name  # no wait ran out
            else:
                pytest.fail(name + ": no wait ran out")
        finally:
            mao.set_wait_limit(limit)
        assert torch.equal(call(), want), name
        mao.sync_status()


def test_many_tiles(cuda):
    """More tiles than pairs of SMs, of all heights: accumulators follow one another."""
    x, up, down, dy = make(7, 5000, 264, 1032, 520)
    y, z = mao.gated_ffn(x, up, down, "silu", save=True)
    mao.sync_status()
    check_forward(y, z, x, up, down, "silu")
    check_backward(mao.gated_ffn_backward(dy, x, up, down, z, "silu"), dy, x, up, down, z, "silu")
    g = torch.Generator().manual_seed(1)
    cnt = torch.randint(0, 400, (40,), generator=g)
    off = torch.zeros(41, dtype=torch.int64)
    off[1:] = ((cnt + 127) // 128 * 128).cumsum(0)
    rows = int(off[-1]) + 128
    x, up, down, dy = make(8, rows, 136, 200, 264, groups=40)
    kw = dict(offsets=off.to(I32).to(cuda), counts=cnt.to(I32).to(cuda))
    y, z = mao.gated_ffn(x, up, down, "gelu_tanh", save=True, **kw)
    check_forward(y, z, x, up, down, "gelu_tanh", off.tolist(), cnt.tolist())
    grads = mao.gated_ffn_backward(dy, x, up, down, z, "gelu_tanh", **kw)
    mao.sync_status()
    check_backward(grads, dy, x, up, down, z, "gelu_tanh", off.tolist(), cnt.tolist())


def test_gradients_of_many_tiles(cuda):
    """So many that each gradient has a launch of its own; the same with some not wanted."""
    g = torch.Generator().manual_seed(2)
    cnt = torch.randint(0, 60, (64,), generator=g)
    off = torch.arange(65) * 128
    x, up, down, dy = make(9, 64 * 128, 520, 520, 264, groups=64)
    kw = dict(offsets=off.to(I32).to(cuda), counts=cnt.to(I32).to(cuda))
    y, z = mao.gated_ffn(x, up, down, "silu", save=True, **kw)
    grads = mao.gated_ffn_backward(dy, x, up, down, z, "silu", **kw)
    mao.sync_status()
    check_backward(grads, dy, x, up, down, z, "silu", off.tolist(), cnt.tolist())
    for only in range(3):
        flags = {k: None if i == only else False for i, k in enumerate(("dX", "dup", "ddown"))}
        some = mao.gated_ffn_backward(dy, x, up, down, z, "silu", **flags, **kw)
        assert [t is None for t in some] == [i != only for i in range(3)]
        assert torch.equal(some[only], grads[only])


@pytest.mark.parametrize("most", [1, 8, 20])
def test_few_rows_in_many_runs(cuda, most):
    """A token's copies in a few of many runs of 128 rows: some runs hold more rows than a pass takes."""
    E, act = 70, "gelu"
    cnt = [0] * E
    for i, g in enumerate((0, 3, 40, 41, 69)):
        cnt[g] = most - i % 2 if most > 1 else 1
    off = np.concatenate([[0], np.cumsum([(c + 127) // 128 * 128 for c in cnt])])
    rows = int(off[-1]) + 40
    for dims in ((264, 72, 136), (77, 33, 41), (1100, 1030, 520)):
        x, up, down, _ = make(most, rows, *dims, groups=E)
        kw = dict(offsets=torch.tensor(off, dtype=I32, device=cuda), counts=torch.tensor(cnt, dtype=I32, device=cuda))
        y, z = mao.gated_ffn(x, up, down, act, save=True, **kw)
        mao.sync_status()
        check_forward(y, z, x, up, down, act, off.tolist(), cnt)
        used = torch.zeros(rows, dtype=torch.bool, device=cuda)
        for lo, hi in of.runs(rows, off, cnt):
            used[lo:hi] = True
        assert (y[~used] == 0).all() and (z[~used] == 0).all()
        a8, as_ = mao.int8_quantize(x)
        b8, bs = mao.int8_quantize(up)
        p = mao.int8_product(a8, as_, b8, bs, out_dtype=F32, **kw)
        whole = torch.zeros_like(p)
        for g, (lo, hi) in enumerate(of.runs(rows, off, cnt)):
            s = a8[lo:hi].double() @ b8[g].double().T  # whole numbers below 2^24
            whole[lo:hi] = s.float() * as_[lo:hi, None] * bs[g]
        assert torch.equal(p, whole)


def test_more_than_2_31_entries(cuda):
    """Tensors whose offsets pass 32 bits: the last rows and columns are right."""
    T, K, N, C = 70016, 32768, 16, 24
    g = torch.Generator(device=cuda).manual_seed(1)
    x = torch.empty(T, K, dtype=BF16, device=cuda).normal_(generator=g)
    up = (torch.randn(2 * N, K, generator=g, device=cuda) * K ** -0.5).to(BF16)
    down = torch.randn(C, N, generator=g, device=cuda).to(BF16)
    dy = torch.randn(T, C, generator=g, device=cuda).to(BF16)
    y, z = mao.gated_ffn(x, up, down, "silu", save=True)
    dx, dup, ddown = mao.gated_ffn_backward(dy, x, up, down, z, "silu")
    mao.sync_status()
    for rows in (slice(0, 40), slice(65520, 65560), slice(T - 40, T)):
        check_forward(y[rows], z[rows], x[rows], up, down, "silu")
        part = mao.gated_ffn_backward(dy[rows], x[rows], up, down, z[rows], "silu")
        assert (dx[rows].float() - part[0].float()).abs().max() <= 2.0 ** -7 * part[0].float().abs().max()
    # the weights' gradients: sums over all rows, by parts of them
    sup, sdown = torch.zeros(dup.shape, device=cuda), torch.zeros(ddown.shape, device=cuda)
    for r in range(0, T, 8752):
        sl = slice(r, r + 8752)
        part = mao.gated_ffn_backward(dy[sl], x[sl], up, down, z[sl], "silu", dX=False, grad_dtype=F32)
        sup += part[1]
        sdown += part[2]
    # the same terms, summed in fp32 in another order, rounded to bf16: 2^-8 of the entry, and the sums'
    # rounding, which is far below 2^-8 of the largest entry
    for a, b in ((dup, sup), (ddown, sdown)):
        assert ((a.float() - b).abs() <= 2.0 ** -8 * b.abs() + 2.0 ** -12 * b.abs().max()).all()
    del x, dx
    a8 = torch.randint(-127, 128, (T, K), generator=g, device=cuda, dtype=torch.int8)
    b8 = torch.randint(-127, 128, (40, K), generator=g, device=cuda, dtype=torch.int8)
    one = lambda n: torch.ones(n, device=cuda)  # noqa: E731
    p = mao.int8_product(a8, one(T), b8, one(40), out_dtype=F32)
    for rows in (slice(0, 40), slice(65520, 65560), slice(T - 40, T)):
        assert torch.equal(p[rows].double(), a8[rows].double() @ b8.double().T)
    wide = torch.randn(5, 2 ** 20, generator=g, device=cuda)
    codes, scales = mao.int8_quantize(wide)
    want, _ = of.int8_rows(wide.cpu().numpy())
    np.testing.assert_array_equal(codes.cpu().numpy(), want)


def test_layer_of_experts_trained_and_served(cuda):
    """Tokens to experts, the block over the plan's runs, back, a Muon step on its weights; then the
    new weights in 8 bits, served. Values and gradients against the formulas in 64 bits."""
    T, K, N, E, k = 300, 128, 96, 6, 2
    x = randn(1, T, K).to(BF16).to(cuda)
    logits = randn(2, T, E).to(cuda)
    up, down = (randn(3, E, 2 * N, K) * K ** -0.5).to(BF16).to(cuda), (randn(4, E, K, N) * N ** -0.5).to(BF16).to(cuda)
    weights, ids = mao.expert_route(logits, k)
    plan = mao.expert_plan(ids, E)
    src = torch.where(plan.slot_of >= 0, plan.slot_of // k, -1)[:, None].contiguous()
    xs = mao.expert_combine(x, src)  # the dispatch: a copy of a token in each row, zeros between
    kw = dict(offsets=plan.offsets, counts=plan.counts)
    h, z = mao.gated_ffn(xs, up, down, "silu", save=True, **kw)
    y = mao.expert_combine(h, plan.row_of, weights)
    off, cnt = plan.offsets.tolist(), plan.counts.tolist()
    check_forward(h, z, xs, up, down, "silu", off, cnt)
    dy = randn(5, T, K).to(BF16).to(cuda)
    dh, dw = mao.expert_combine_backward(dy, h, plan.row_of, plan.slot_of, weights)
    dxs, dup, ddown = mao.gated_ffn_backward(dh, xs, up, down, z, "silu", **kw)
    mao.sync_status()
    check_backward((dxs, dup, ddown), dh, xs, up, down, z, "silu", off, cnt)
    dx = mao.expert_combine(dxs, plan.row_of)
    # the tokens' gradient: their copies' added up, each rounded to bf16 before (k of them)
    want = dxs.float()[plan.row_of.long()].sum(1)
    assert ((dx.float() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-30).all()
    mats = list(up.unbind(0)) + list(down.unbind(0))
    before = [m.clone() for m in mats]
    mao.muon_step(mats, [torch.zeros_like(m) for m in mats], list(dup.unbind(0)) + list(ddown.unbind(0)), mu=0.9, lr=0.01)
    assert all(not torch.equal(a, b) for a, b in zip(before, mats))
    # served: 8-bit rows and weights
    u8, us = mao.int8_quantize(up)
    d8, ds = mao.int8_quantize(down)
    x8, xss = mao.int8_quantize(xs)
    zz = mao.int8_product(x8, xss, u8, us, out_dtype=F32, **kw)
    h8, hs = mao.int8_quantize(zz, gate="silu")
    out = mao.int8_product(h8, hs, d8, ds, out_dtype=F32, **kw)
    ys = mao.expert_combine(out, plan.row_of, weights)
    mao.sync_status()
    val = lambda c, s: c.double() * s.double()[..., None]  # noqa: E731
    ref = torch.zeros(len(xs), K, dtype=torch.float64, device=cuda)
    for e, (lo, hi) in enumerate(of.runs(len(xs), off, cnt)):
        ref[lo:hi] = val(h8, hs)[lo:hi] @ val(d8, ds)[e].T
        zr = val(x8, xss)[lo:hi] @ val(u8, us)[e].T
        assert ((zz[lo:hi] - zr).abs() <= 2.0 ** -21 * zr.abs() + 1e-12).all()
    # sums of products of codes are exact; three roundings of the scaled value
    assert ((out - ref).abs() <= 2.0 ** -21 * ref.abs() + 1e-12).all()
    assert ys.shape == y.shape and torch.isfinite(ys).all()
