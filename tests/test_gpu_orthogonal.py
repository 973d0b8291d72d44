"""Orthogonalized updates on the GPU against the fp64 definition.

Bound: rounding to bf16 (8 significant bits) leaves an error uniform within half
a unit in the last place, 2^-9 in the 2-norm at the mean of the significands. The products' operands carry 2^-12 each (fp16, half a unit): per
step the Gram matrix, its square and the polynomial's product add about
sqrt(3) 2^-12 of the off-diagonal parts to a result whose saturated singular
values pass errors on with a factor below 1 but for their rotations; five steps
add up, as independent roundings, to sqrt(5) sqrt(3) 2^-12 = 9.5e-4, and twice
that is allowed: 2^-9 + 1.9e-3 = 3.9e-3.
"""
import numpy as np
import pytest
import torch

import oracle.block_ops as B
from parity_util import host

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -9 + 1.9e-3


def _rand(seed, *shape):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda:0")


def _check(out, grad, mom=None, beta=0.95, nesterov=True, steps=5, new=None, tol=TOL):
    out, grad = host(out).astype(np.float64), host(grad)
    for i in range(len(grad)):
        ref, m = B.orthogonalize(grad[i], None if mom is None else host(mom)[i], np.float32(beta),
                                 nesterov, steps)
        err = np.linalg.norm(out[i] - ref) / max(np.linalg.norm(ref), 1e-30)
        assert err <= tol, (i, grad.shape, err)
        if new is not None:
            got = host(new)[i]
            mag = np.abs(host(mom)[i]) + np.abs(grad[i])
            assert (np.abs(got - m) <= 2.0 ** -23 * mag).all()


# one workgroup a matrix up to 128 x 256, else 128 x 128 tiles, else 256 x 256
SIZES = [(1, 128, 256), (300, 20, 30), (1, 256, 128), (1, 129, 256), (1, 128, 257), (80, 270, 400),
         (1, 1, 1), (2, 1, 40), (2, 40, 1), (3, 16, 16), (2, 7, 100), (1, 100, 7), (4, 63, 65),
         (3, 128, 256), (2, 129, 130), (1, 257, 300), (1, 300, 257), (2, 64, 1000), (1, 520, 776),
         (1, 777, 521), (33, 24, 40)]


@pytest.mark.parametrize("mats,rows,cols", SIZES)
@pytest.mark.parametrize("mom", [False, True])
def test_random_matrices(mats, rows, cols, mom):
    import sparse_mixture_experts_gate_amd as M
    g = _rand(1, mats, rows, cols) * 1e-3
    m = _rand(2, mats, rows, cols) * 2e-3 if mom else None
    out, new = M.Muon().direction(g, m)
    assert out.dtype == torch.bfloat16 and out.shape == g.shape
    _check(out, g, m, new=new)


@pytest.mark.parametrize("scale", [1e-20, 1e-4, 1e15])
def test_scale_of_the_gradient(scale):
    """The norm is taken in fp64: squares of 1e-20 and of 1e15 neither vanish
    nor overflow. 1e-20 disappears against the 1e-7 of the definition."""
    import sparse_mixture_experts_gate_amd as M
    g = _rand(1, 2, 48, 80) * scale
    out, _ = M.Muon().direction(g)
    if scale < 1e-10:
        assert float(out.abs().max()) < 1e-8
    else:
        _check(out, g)


@pytest.mark.parametrize("rank", [1, 5, 32])
@pytest.mark.parametrize("rows,cols", [(200, 330), (64, 1000), (100, 240)])
@pytest.mark.parametrize("steps", [5, 8])
def test_rank_deficient_updates(rank, rows, cols, steps):
    """The null space must stay empty: rounding noise there would grow 3.44
    times per step."""
    import sparse_mixture_experts_gate_amd as M
    g = _rand(1, 2, rows, rank) @ _rand(2, 2, rank, cols)
    out, _ = M.Muon(steps=steps).direction(g)
    _check(out, g, steps=steps)
    out, _ = M.Muon(steps=steps).direction(g.transpose(1, 2).contiguous())
    _check(out, g.transpose(1, 2), steps=steps)


def test_wide_spectrum_bf16_gradients_and_plain_momentum():
    import sparse_mixture_experts_gate_amd as M
    g = (_rand(1, 2, 150, 260) * torch.exp(2 * _rand(2, 2, 150, 1))).bfloat16()
    m = _rand(3, 2, 150, 260)
    for nesterov in (False, True):
        out, new = M.Muon(0.9, nesterov, 5).direction(g, m)
        _check(out, g, m, 0.9, nesterov, new=new)
    # in place
    m2 = m.clone()
    out2, same = M.Muon(0.9, True, 5).direction(g, m2, out_momentum=m2)
    assert same is m2 and torch.equal(m2, new) and torch.equal(out2, out)


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_step_counts(steps):
    import sparse_mixture_experts_gate_amd as M
    g = _rand(1, 2, 90, 140)
    out, _ = M.Muon(steps=steps).direction(g)
    _check(out, g, steps=steps)


@pytest.mark.parametrize("rows,cols", [(70, 90), (150, 290), (300, 130)])
def test_zero_nan_and_neighbours(rows, cols):
    """A zero matrix stays zero; NaN fills its own matrix only; results do not
    depend on what else is in the batch or in the workspace."""
    import sparse_mixture_experts_gate_amd as M
    g = _rand(1, 4, rows, cols)
    alone = [M.Muon().direction(g[i:i + 1].contiguous())[0][0] for i in range(4)]
    g[1] = 0
    g[2, 3, 4] = float("nan")
    op = M.Muon()
    for fill in (0, 255):
        out, _ = op.direction(g)
        assert torch.equal(out[0], alone[0]) and torch.equal(out[3], alone[3])
        assert not out[1].any() and bool(torch.isnan(out[2]).all())
        for buf in op._ws._bufs.values():
            buf.fill_(255 - fill)


def test_leading_dimensions_stream_and_repeat():
    import sparse_mixture_experts_gate_amd as M
    g = _rand(1, 2, 3, 130, 64)
    op = M.Muon()
    out, _ = op.direction(g)
    _check(out.reshape(6, 130, 64), g.reshape(6, 130, 64))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again, _ = op.direction(g, stream=s)
    s.synchronize()
    assert torch.equal(out, again)
    assert op.direction(g[:0])[0].shape == (0, 3, 130, 64)


def test_result_is_nearly_orthogonal():
    import sparse_mixture_experts_gate_amd as M
    out, _ = M.Muon().direction(_rand(1, 1, 256, 700))
    s = np.linalg.svd(host(out[0]).astype(np.float64), compute_uv=False)
    assert 0.6 < s.min() and s.max() < 1.25
