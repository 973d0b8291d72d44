"""The example block: its gradients against torch's autograd over the same
block in fp32, and a loss that falls under the orthogonalized updates."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_gradients_against_autograd():
    """bf16 activations pass through about eight roundings of at most 2^-8
    (random in sign) on their way; 2-norms within 2%."""
    from train_block import GeluMoEBlock
    block = GeluMoEBlock(d=128, hidden=192, experts=4)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(3)
    x, r, dy = (torch.randn(77, 128, generator=g, device="cuda:0").bfloat16() for _ in range(3))
    y, saved = block.forward(x, r)
    grads = block.backward(dy, saved)
    n, gate, offsets, perm, inv, *_ = saved
    v = (x.float() + r.float()).requires_grad_()
    p = [t.clone().requires_grad_() for t in (block.norm.weight, block.norm.bias,
                                              block.w1.bfloat16().float(),
                                              block.w2.bfloat16().float())]
    z = torch.nn.functional.layer_norm(v, (128,), p[0], p[1], 1e-5)
    zs, off = z[perm.long()], offsets.tolist()
    o = torch.cat([torch.nn.functional.gelu(zs[off[e]:off[e + 1]] @ p[2][e].t()) @ p[3][e].t()
                   for e in range(4)])
    ref = v + (o[inv.long()] * gate[:, :, None]).sum(1)
    ref.backward(dy.float())
    rel = lambda a, b: float((a.float() - b).norm() / b.norm())
    assert rel(y, ref.detach()) < 0.02
    for name, t in (("dx", v), ("dweight", p[0]), ("dbias", p[1]), ("dw1", p[2]), ("dw2", p[3])):
        assert rel(grads[name], t.grad) < 0.02, name


def test_loss_falls():
    from train_block import train
    losses = train(steps=8, verbose=False)
    assert losses[-1] < 0.5 * losses[0], losses
