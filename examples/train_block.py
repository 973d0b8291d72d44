"""One pre-norm block with GELU experts, trained for a few steps on synthetic
data with this library's operators:

    v = x + r,  z = norm(v)                       LayerNorm (residual fused)
    routing of z: logits, top-K, gates, sorting   moe_gate, moe_permute
    h = z_sorted W1_g^T,  a = gelu(h),
    o = a W2_g^T                                   GroupedLinear
    y = v + sum_k gate_k o                         moe_combine

and back: GroupedLinear.input_grad / weight_grad, the norm's backward with the
residual's gradient added, and the orthogonalized update of the expert weights
(Muon; every expert's matrix at once). The router stays as it is: its gates
enter the gradients as constants. The target is a fixed random block of the
same shape, so that the loss can fall.

Run: python examples/train_block.py [steps]     (one MI355X)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_mixture_experts_gate_amd as M  # noqa: E402
from sparse_mixture_experts_gate_amd import Workload  # noqa: E402


class GeluMoEBlock:
    """Weights in bf16 with fp32 masters; the experts' are updated by Muon."""

    def __init__(self, d=512, hidden=768, experts=8, top_k=2, seed=0, device="cuda:0"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)
        self.wl = Workload("gelu_block", T=0, d=d, E=experts, K=top_k, I=64, Is=0)
        self.norm = M.LayerNorm(torch.ones(d, device=device), torch.zeros(d, device=device))
        self.w_router = rand(experts, d) / d ** 0.5
        self.bias = torch.zeros(experts, device=device)
        self.w1 = rand(experts, hidden, d) / d ** 0.5
        self.w2 = rand(experts, d, hidden) / hidden ** 0.5
        self.m1, self.m2 = torch.zeros_like(self.w1), torch.zeros_like(self.w2)
        self.muon = M.Muon(momentum=0.9)
        self.device = device

    def route(self, z):
        """Selection, gates and the counting sort of z's rows by expert."""
        T, E, K, dev = z.shape[0], self.wl.E, self.wl.K, self.device
        desc = M.make_desc(self.wl, T)
        i32 = dict(dtype=torch.int32, device=dev)
        logits = torch.empty(T, E, device=dev)
        idx, gate = torch.empty(T, K, **i32), torch.empty(T, K, device=dev)
        counts, near = torch.empty(E, **i32), torch.empty(1, **i32)
        ws = torch.empty(M.moe_workspace_size(desc), dtype=torch.uint8, device=dev)
        M.moe_gate(desc, z, self.w_router, self.bias, logits, idx, gate, counts, near, ws)
        offsets, perm = torch.empty(E + 1, **i32), torch.empty(T * K, **i32)
        inv, z_sorted = torch.empty(T, K, **i32), torch.empty(T * K, z.shape[1], dtype=z.dtype,
                                                              device=dev)
        M.moe_permute(desc, idx, counts, z, offsets, perm, inv, z_sorted)
        return desc, gate, offsets, perm, inv, z_sorted

    def forward(self, x, r):
        """y and what the backward needs."""
        n = self.norm.forward(x, r)
        desc, gate, offsets, perm, inv, zs = self.route(n["y"])
        up = M.GroupedLinear(self.w1.bfloat16())
        down = M.GroupedLinear(self.w2.bfloat16())
        h = up.forward(zs, offsets)
        a = torch.nn.functional.gelu(h)
        o = down.forward(a, offsets)
        routed = torch.empty_like(x)
        M.moe_combine(desc, o, inv, gate, None, routed)
        y = n["sum"] + routed
        return y, (n, gate, offsets, perm, inv, zs, up, down, h, a)

    def backward(self, dy, saved):
        """Gradients: dx (also the residual's), the norm's and the experts'."""
        n, gate, offsets, perm, inv, zs, up, down, h, a = saved
        pairs = gate.new_empty(gate.numel())
        pairs[inv.reshape(-1).long()] = gate.reshape(-1)  # gates in sorted order
        do = (dy[perm.long()].float() * pairs[:, None]).bfloat16()
        dw2 = down.weight_grad(do, a, offsets)
        da = down.input_grad(do, offsets)
        dh = torch.ops.aten.gelu_backward(da, h)
        dw1 = up.weight_grad(dh, zs, offsets)
        dzs = up.input_grad(dh, offsets)
        dz = dzs[inv.long()].float().sum(1).bfloat16()
        g = self.norm.backward(dz, n["sum"], n["mean"], n["rstd"], dy)
        return {**g, "dw1": dw1, "dw2": dw2}

    def update(self, grads, lr):
        """Orthogonalized step of the experts, plain step of the norm."""
        for w, m, name in ((self.w1, self.m1, "dw1"), (self.w2, self.m2, "dw2")):
            step, _ = self.muon.direction(grads[name], m, out_momentum=m)
            w.add_(step.float(), alpha=-lr * 0.2 * max(w.shape[1:]) ** 0.5)
        self.norm.weight.add_(grads["dweight"], alpha=-lr)
        self.norm.bias.add_(grads["dbias"], alpha=-lr)


def train(steps=8, tokens=1000, lr=0.02, verbose=True):
    block, target = GeluMoEBlock(seed=0), GeluMoEBlock(seed=1)
    target.w_router = block.w_router
    g = torch.Generator(device="cuda:0")
    g.manual_seed(2)
    x, r = (torch.randn(tokens, 512, generator=g, device="cuda:0").bfloat16() for _ in range(2))
    want = target.forward(x, r)[0].float()
    losses = []
    for step in range(steps):
        y, saved = block.forward(x, r)
        err = y.float() - want
        losses.append(float(err.square().mean()))
        grads = block.backward((2.0 * err / err.numel()).bfloat16(), saved)
        block.update(grads, lr)
        if verbose:
            print(f"step {step}: loss {losses[-1]:.5f}", flush=True)
    return losses


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
