"""Each tile of the 4-bit products: rows and columns that end inside it, several groups,
one of them empty, strided outputs in both types, against the definition in 64 bits, and
the same bits as the tile of few rows gives. The bound is that of test_gpu_mx4."""
import numpy as np
import pytest
import torch

import oracle.token_ops as B
from parity_util import host
from test_gpu_mx4 import DEV, DT, RND, _rand

pytestmark = pytest.mark.gpu

CASES = [  # rows, groups, n, k and the tile that they take
    (4095, 1, 4095, 1000, "256"), (6000, 1, 2500, 777, "256"), (16000, 3, 1030, 1290, "256"),
    (28240, 5, 843, 1497, "256"),
    (4099, 3, 2048, 300, "128"), (5000, 3, 2100, 2000, "128"), (4097, 1, 4095, 1000, "128"),
    (2000, 3, 1000, 520, "64"), (1500, 5, 4096, 256, "64"), (1030, 1, 2050, 264, "64"),
    (8, 8, 2816, 300, "32"), (100, 7, 2000, 1000, "32"), (40, 1, 5000, 70, "32"),
    (40, 3, 129, 257, "thin"), (9, 512, 40, 70, "thin"), (33, 1, 65, 1031, "thin")]


def _split(rows, G):
    """Ascending offsets, rows before the first group and behind the last, an empty group."""
    first, last = (5, rows - 3) if rows > 20 else (0, rows)
    cut = np.sort(np.random.default_rng(rows).integers(first, last + 1, size=G - 1))
    if G > 2:
        cut[1] = cut[0]
    return np.r_[first, cut, last].astype(np.int32)


def _sample(off, rows):
    """Rows at the groups' ends and at multiples of 32 to 256 behind their starts."""
    g = np.random.default_rng(rows + 1)
    pick = set(g.integers(off[0], off[-1], size=24).tolist())
    for a, b in zip(off, off[1:]):
        for at in (a, a + 1, a + 31, a + 32, a + 63, a + 64, a + 127, a + 128, a + 255, a + 256,
                   a + (b - a) // 256 * 256 - 1, a + (b - a) // 256 * 256, b - 2, b - 1):
            if a <= at < b:
                pick.add(int(at))
    return np.array(sorted(pick))


@pytest.mark.parametrize("rows,G,n,k,tile", CASES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_tile(rows, G, n, k, tile, out):
    import sparse_mixture_experts_gate_amd as M
    lin = M.MX4Linear.from_weight(_rand(rows + 1, G, n, k, dt="bf16", spread=2.0))
    x = _rand(rows + 2, rows, k, dt="bf16", spread=2.0)
    codes, scales = M.mx4_quantize(x)
    off = _split(rows, G)
    t_off = torch.from_numpy(off).to(DEV)
    wide = torch.full((rows, n + 5), 7.0, dtype=DT[out], device=DEV)
    desc = M.MoeMx4GemmDesc(rows=rows, n_groups=G, n=n, k=k, ld_y=n + 5,
                            out_dtype=M.MOE_DT_BF16 if out == "bf16" else M.MOE_DT_F32)
    M.moe_mx4_gemm(desc, codes, scales, lin.codes, lin.scales, t_off, wide[:, 2:2 + n])
    y = wide[:, 2:2 + n].clone()
    for edge in (wide[:, :2], wide[:, 2 + n:], y[:off[0]], y[off[-1]:]):
        assert bool((edge == 7).all())
    assert torch.equal(lin.forward(x, t_off, out_dtype=DT[out])[off[0]:off[-1]], y[off[0]:off[-1]])

    pick = _sample(off, rows)
    sel = torch.from_numpy(pick).to(DEV)
    small = np.searchsorted(pick, off).astype(np.int32)
    # the definition
    q = host(M.mx4_dequantize(codes[sel], scales[:, sel].contiguous(), k, torch.float32))
    ref, mag = B.mx4_product(q.astype(np.float64), host(lin.values()).astype(np.float64), small)
    got = host(y[sel]).astype(np.float64)
    bad = ~(np.abs(got - ref) <= (k / 64 + 8) * 2.0 ** -23 * mag + RND[out] * np.abs(ref))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])
    # few rows of the same, a group at a time
    for g in range(G):
        a, b = small[g], min(small[g + 1], small[g] + 8)
        if a < b:
            one = M.MX4Linear(lin.codes[g:g + 1].clone(), lin.scales[g:g + 1].clone(), k)
            few = one.forward(x[sel[a:b]], torch.tensor([0, b - a], dtype=torch.int32, device=DEV),
                              out_dtype=DT[out])
            assert torch.equal(few, y[sel[a:b]])


@pytest.mark.parametrize("rows,n,k,bad,split", [
    (50, 40, 64, [-9, 10, 5, 2 ** 31 - 1, 3], [0, 10, 10, 50, 50]),
    (50, 40, 64, [60, -1, 70, 8, 9], [50, 50, 50, 50, 50]),
    (100, 4100, 300, [7, 30, -5, 90, 20], [7, 30, 30, 90, 90]),
    (2000, 1000, 520, [-2 ** 31, 900, 300, 2 ** 31 - 1], [0, 900, 900, 2000]),
    (16000, 1030, 1290, [-9, 9000, 4000, 1 << 20], [0, 9000, 9000, 16000])])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_offsets_out_of_order_are_a_clamped_split(rows, n, k, bad, split, out):
    """The whole product is that of the clamped ascending split, from the tile of few rows
    to the largest; nothing around it is written."""
    import sparse_mixture_experts_gate_amd as M
    lin = M.MX4Linear.from_weight(_rand(1, len(bad) - 1, n, k, dt="bf16"))
    codes, scales = M.mx4_quantize(_rand(2, rows, k, dt="bf16"))
    desc = M.MoeMx4GemmDesc(rows=rows, n_groups=len(bad) - 1, n=n, k=k, ld_y=n + 3,
                            out_dtype=M.MOE_DT_BF16 if out == "bf16" else M.MOE_DT_F32)
    got = []
    for off in (bad, split):
        wide = torch.full((rows + 600, n + 3), 7.0, dtype=DT[out], device=DEV)
        M.moe_mx4_gemm(desc, codes, scales, lin.codes, lin.scales,
                       torch.tensor(off, dtype=torch.int32, device=DEV), wide[300:-300, 1:1 + n])
        inside = wide[300:-300, 1:1 + n]
        got.append(inside.clone())
        inside[split[0]:split[-1]] = 7.0
        assert bool((wide == 7).all())
    assert torch.equal(*got)
