"""The expert layer of examples/expert_layer.py: its gradients against autograd on the
quantised values, and a short training with Muon."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def values(codes, scales, br, bc):
    f = torch.exp2(scales.double() - 127).repeat_interleave(br, -2).repeat_interleave(bc, -1)
    return codes.double() * f[..., :codes.shape[-2], :codes.shape[-1]]


def rel(a, b):
    return float((a.double() - b.detach().double()).norm() / b.detach().double().norm())


def test_layer_against_autograd(cuda):
    """The layer in 64 bits with the quantised weights. What differs are the 8-bit roundings of
    activations and gradients: each at most 2^-4 of an entry (three mantissa bits), about 2.6%
    of a tensor's norm; three or four of them lie on a path, so 12% bounds every result."""
    from expert_layer import ExpertLayer

    layer = ExpertLayer(256, 128, 8, 2, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(300, 256, generator=g, device=cuda).to(torch.bfloat16)
    dy = torch.randn(300, 256, generator=g, device=cuda).to(torch.bfloat16)
    y, saved = layer.forward(x)
    drouter, dup, ddown = layer.backward(dy, saved)

    router = layer.router.double().requires_grad_(True)
    up = values(*layer.up8, 128, 128).requires_grad_(True)
    down = values(*layer.down8, 128, 128).requires_grad_(True)
    ids = saved[3].long()
    p = torch.softmax(x.double() @ router.T, 1).gather(1, ids)
    p = p / p.sum(1, keepdim=True)
    want = torch.zeros(300, 256, dtype=torch.float64, device=cuda)
    for e in range(8):
        for j in range(2):
            t = (ids[:, j] == e).nonzero().flatten()
            h = x[t].double() @ up[e].T
            a = torch.nn.functional.silu(h[:, :128]) * h[:, 128:]
            want = want.index_add(0, t, p[t, j, None] * (a @ down[e].T))
    assert rel(y, want) < 0.12
    want.backward(dy.double())
    assert rel(drouter, router.grad) < 0.12
    assert rel(dup, up.grad) < 0.12
    assert rel(ddown, down.grad) < 0.12


def test_layer_learns(cuda):
    """The loss falls by far more than batches differ: a batch's loss is a mean over 512 tokens
    of 256 squares, so it varies by about 1%, the mean of five by half of that, and a tenth is
    beyond chance. How fast it falls is the optimizer's affair, and not checked here."""
    from expert_layer import train

    curve = train(steps=60)
    assert all(v == v for v in curve)
    assert sum(curve[-5:]) < 0.9 * sum(curve[:5])
