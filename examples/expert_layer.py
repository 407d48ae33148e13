"""Trains one layer of experts in 8-bit floating point with Muon.

Each token goes to the best top_k of the experts, each a gated two-matrix network; the layer
learns to imitate a fixed layer of the same form. One step:

  forward    expert_route, expert_plan, fp8_quantize (the dispatch: the tokens' copies gathered
             in the order of the experts), fp8_product "nt", the gate, fp8_product "nt",
             expert_combine
  backward   expert_combine_backward, fp8_quantize, fp8_product "nn" (inputs' gradients) and
             "tn" (weights' gradients), expert_route_backward
  update     muon_step on the experts' matrices, then fp8_quantize of the new weights

Run on a GPU:  python examples/expert_layer.py [steps]
"""

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_aware_optimizers_gb300 as mao  # noqa: E402


class ExpertLayer:
    """`experts` networks x -> (silu(x W1a^T) * (x W1b^T)) W2^T, mixed by a router."""

    def __init__(self, hidden, inner, experts, top_k, seed, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        new = lambda *shape: torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5  # noqa: E731
        self.experts, self.top_k, self.inner = experts, top_k, inner
        self.router = new(experts, hidden)
        self.up = new(experts, 2 * inner, hidden).to(torch.bfloat16)
        self.down = new(experts, hidden, inner).to(torch.bfloat16)
        self.requantize()

    def requantize(self):
        self.up8 = mao.fp8_quantize(self.up, "tile")
        self.down8 = mao.fp8_quantize(self.down, "tile")

    def forward(self, x):
        """Outputs of the tokens x [T, hidden] (bfloat16), and what backward needs."""
        k = self.top_k
        logits = x.float() @ self.router.T
        weights, ids = mao.expert_route(logits, k, score="softmax", renorm=True)
        plan = mao.expert_plan(ids, self.experts)
        # row blocks for the forward product, column blocks for the weights' gradient
        xr, xrs, xc, xcs = mao.fp8_quantize(x, "both", rows=plan.slot_of, copies=k)
        h = mao.fp8_product(xr, xrs, *self.up8, "nt", offsets=plan.offsets)
        a = F.silu(h[:, :self.inner].float()) * h[:, self.inner:].float()
        ar, ars, ac, acs = mao.fp8_quantize(a, "both")
        z = mao.fp8_product(ar, ars, *self.down8, "nt", offsets=plan.offsets)
        y = mao.expert_combine(z, plan.row_of, weights)
        return y, (x, logits, weights, ids, plan, h, z, (xc, xcs), (ac, acs))

    def backward(self, dy, saved):
        """Gradients of router, up and down for the outputs' gradient dy."""
        x, logits, weights, ids, plan, h, z, x8, a8 = saved
        dz, dw = mao.expert_combine_backward(dy, z, plan.row_of, plan.slot_of, weights)
        zr, zrs, zc, zcs = mao.fp8_quantize(dz, "both")
        da = mao.fp8_product(zr, zrs, *self.down8, "nn", offsets=plan.offsets).float()
        ddown = mao.fp8_product(zc, zcs, *a8, "tn", offsets=plan.offsets, out_dtype=torch.float32)
        gate, lin = h[:, :self.inner].float(), h[:, self.inner:].float()
        s = torch.sigmoid(gate)
        dh = torch.cat([da * lin * s * (1.0 + gate * (1.0 - s)), da * gate * s], 1)
        hc, hcs = mao.fp8_quantize(dh, "col")
        dup = mao.fp8_product(hc, hcs, *x8, "tn", offsets=plan.offsets, out_dtype=torch.float32)
        dlogits = mao.expert_route_backward(logits, ids, dw, score="softmax", renorm=True)
        return dlogits.T @ x.float(), dup, ddown


def train(steps=60, tokens=512, hidden=256, inner=128, experts=8, top_k=2, lr=0.02, seed=0):
    """Losses of the steps (mean squared difference from the teacher, relative to its size)."""
    teacher = ExpertLayer(hidden, inner, experts, top_k, seed=seed + 1)
    layer = ExpertLayer(hidden, inner, experts, top_k, seed=seed + 2)
    layer.router.copy_(teacher.router)  # the layer starts with the teacher's choice of experts
    mats = list(layer.up.unbind(0)) + list(layer.down.unbind(0))
    momenta = [torch.zeros_like(m) for m in mats]
    ws = mao.workspace(mats, "bf16", mats[0].device)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
        want = teacher.forward(x)[0].float()
        y, saved = layer.forward(x)
        diff = y.float() - want
        losses.append(diff.square().mean() / want.square().mean())
        drouter, dup, ddown = layer.backward(diff.to(torch.bfloat16), saved)
        grads = list(dup.unbind(0)) + list(ddown.unbind(0))
        rate = lr * (1.0 - step / steps)
        mao.muon_step(mats, momenta, grads, mu=0.9, lr=rate, ws=ws)
        layer.router -= 0.1 * rate * drouter / (drouter.norm() + 1e-12)
        layer.requantize()
    mao.sync_status()
    return [float(v) for v in losses]


if __name__ == "__main__":
    curve = train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    for i in range(0, len(curve), 10):
        print("step %3d  loss %.4f" % (i, curve[i]))
    print("last      loss %.4f" % curve[-1])
