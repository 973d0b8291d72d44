"""Orthogonalized updates at the sizes of wide experts, where the products run
on 256 x 256 tiles and the last round's Gram tiles are shared by several
workgroups, against the definition in fp64 (torch products of single matrices).

Bound: that of the smaller sizes, which does not depend on the size. Rounding
to bf16 leaves 2^-9 in the 2-norm; the operands' fp16 roundings add sqrt(3)
2^-12 per step, five of them as independent roundings 9.5e-4, and twice that is
allowed.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -9 + 1.9e-3
U = 2.0 ** -24


def _rand(seed, *shape):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda:0")


def _exact(u, steps=5):
    u = u.double()
    x = u.t().contiguous() if u.shape[0] > u.shape[1] else u
    x = x / ((x ** 2).sum().sqrt() + 1e-7)
    a, b, c = 3.4445, -4.7750, 2.0315
    for _ in range(steps):
        A = x @ x.t().contiguous()
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.t() if u.shape[0] > u.shape[1] else x


def _check(out, updates):
    for i, u in enumerate(updates):
        ref = _exact(u)
        err = float((out[i].double() - ref).norm() / ref.norm())
        assert err <= TOL, (i, list(u.shape), err)


# 256 x 256 tiles in every product, of whole and of odd sizes; with the last
# round of Gram tiles shared; with all of them shared; 128 x 128 Gram tiles
# shared, alone and behind whole rounds
SIZES = [(40, 520, 776), (40, 519, 777), (8, 2040, 3000), (3, 2039, 3999), (1, 300, 4100),
         (87, 400, 1500)]


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("mats,n,m", SIZES)
def test_random_matrices(mats, n, m, tall):
    import sparse_mixture_experts_gate_amd as M
    g = _rand(1, mats, m, n) if tall else _rand(1, mats, n, m)
    out, _ = M.Muon().direction(g)
    _check(out, g)


@pytest.mark.parametrize("mats,rows,cols", [(8, 2040, 3000), (8, 3000, 2040), (40, 777, 519)])
def test_momentum_bf16_gradients_in_place_and_repeat(mats, rows, cols):
    """The new momentum is one rounded product and sum off (2 u of its terms),
    also where it replaces the old one; a repeat gives the same bits, whichever
    workgroup adds a shared tile."""
    import sparse_mixture_experts_gate_amd as M
    g, m = _rand(1, mats, rows, cols).bfloat16(), _rand(2, mats, rows, cols)
    beta = float(torch.tensor(0.9))
    muon = M.Muon(0.9)
    out, new = muon.direction(g, m)
    exact = m.double() * beta + g.double()
    assert bool(((new.double() - exact).abs() <= 2 * U * (m.double().abs() + g.double().abs())).all())
    _check(out, g.double() + beta * exact)
    m2 = m.clone()
    again, same = muon.direction(g, m2, out_momentum=m2)
    assert same is m2 and torch.equal(m2, new) and torch.equal(again, out)


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("rank", [1, 40])
def test_rank_deficient_updates(rank, tall):
    import sparse_mixture_experts_gate_amd as M
    g = torch.stack([_rand(i, 2040, rank) @ _rand(50 + i, rank, 3000) for i in range(8)])
    g = g.transpose(1, 2).contiguous() if tall else g
    out, _ = M.Muon().direction(g)
    _check(out, g)


@pytest.mark.parametrize("rows,cols", [(2040, 3000), (3000, 2040)])
def test_zero_nan_and_neighbours(rows, cols):
    """A zero matrix stays zero, NaN fills its own matrix only, and the others
    do not change, whatever the workspace held."""
    import sparse_mixture_experts_gate_amd as M
    g = _rand(1, 8, rows, cols)
    clean, _ = M.Muon().direction(g)
    g[3] = 0
    g[7, 5, 6] = float("nan")
    desc = M.MoeOrthDesc(n_mats=8, rows=rows, cols=cols, grad_dtype=M.MOE_DT_F32, steps=5)
    ws = torch.full((M.moe_orthogonalize_workspace_size(desc),), 255, dtype=torch.uint8,
                    device="cuda:0")
    out = torch.empty(8, rows, cols, dtype=torch.bfloat16, device="cuda:0")
    M.moe_orthogonalize(desc, g, None, None, out, ws)
    keep = [0, 1, 2, 4, 5, 6]
    assert torch.equal(out[keep], clean[keep])
    assert not out[3].any() and bool(torch.isnan(out[7]).all())
