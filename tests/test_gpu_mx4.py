"""Microscaled 4-bit values on the GPU. Codes, scales and values are compared for
equality: scaling by a power of two is exact and every rounding has one answer.

Products: an instruction multiplies 64 values exactly and adds them to an fp32 sum;
with k / 64 instructions one after the other, and a sum that may drop bits below its
last (2^-23 of the terms' magnitude each) rather than round, the result is off by (k
/ 64 + 8) 2^-23 of the sum of the terms' magnitudes, and bf16 outputs by 2^-8 of the
value more."""
import numpy as np
import pytest
import torch

import oracle.token_ops as B
from parity_util import host

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
RND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
DEV = "cuda:0"


def _rand(seed, *shape, dt="f32", spread=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    v = torch.randn(*shape, generator=g, device=DEV)
    if spread:
        v = v * torch.exp2((torch.randn(*shape[:-1], 1, generator=g, device=DEV) * spread).round())
    return v.to(DT[dt])


def _same(codes, scales, v):
    c, b = B.mx4_encode(host(v))
    assert np.array_equal(host(codes), B.mx4_pack(c))
    assert np.array_equal(host(scales), B.mx4_words(b))
    return c, b


SHAPES = [(1, 1), (1, 7168), (3, 31), (5, 32), (2, 33), (9, 128), (7, 129), (33, 500), (40, 513),
          (31, 1407), (2, 5, 70), (3, 33, 600), (1, 1, 2048)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_and_back(shape, dt):
    import sparse_mixture_experts_gate_amd as M
    v = _rand(1, *shape, dt=dt, spread=8.0)
    codes, scales = M.mx4_quantize(v)
    c, b = _same(codes, scales, v)
    for out in ("bf16", "f32"):
        got = M.mx4_dequantize(codes, scales, shape[-1], DT[out])
        assert got.dtype is DT[out] and got.shape == v.shape
        assert np.array_equal(host(got), B.mx4_decode(c, b, shape[-1]))


@pytest.mark.parametrize("rows,k", [(40000, 32), (4100, 4096), (1100, 16384)])
def test_many_blocks(rows, k):
    """Past the choice of 32 rows per workgroup, ragged at its end."""
    import sparse_mixture_experts_gate_amd as M
    v = _rand(2, rows, k, dt="bf16", spread=2.0)
    codes, scales = M.mx4_quantize(v)
    pick = np.r_[0:70, rows // 2:rows // 2 + 40, rows - 70:rows]
    c, b = B.mx4_encode(host(v[torch.from_numpy(pick).to(DEV)]))
    assert np.array_equal(host(codes)[pick], B.mx4_pack(c))
    assert np.array_equal(host(scales)[:, pick], B.mx4_words(b))


def test_every_rounding():
    """All halves between codes, both signs, past 6, at every scale that fp32 has,
    denormal numbers and the largest ones among them."""
    import sparse_mixture_experts_gate_amd as M
    a = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    near = np.r_[a, np.nextafter(a, 9, dtype=np.float32), np.nextafter(a, -9, dtype=np.float32)]
    block = np.zeros((3, 32), np.float32)
    for i in range(3):  # each of them beside a largest value of 4 .. 8
        block[i, :16], block[i, 16:31] = near[16 * i:16 * i + 16], -near[16 * i:16 * i + 15]
        block[i, 31] = 4.0
    e = np.arange(-146, 126)
    v = np.ldexp(block[None].astype(np.float64), e[:, None, None]).astype(np.float32).reshape(-1, 32)
    t = torch.from_numpy(v).to(DEV)
    codes, scales = M.mx4_quantize(t)
    _same(codes, scales, t)


def test_every_code_and_scale_back():
    import sparse_mixture_experts_gate_amd as M
    c = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    byte = np.arange(256, dtype=np.uint8)[:, None]
    for out in ("bf16", "f32"):
        got = host(M.mx4_dequantize(torch.from_numpy(B.mx4_pack(c)).to(DEV),
                                    torch.from_numpy(np.ascontiguousarray(B.mx4_words(byte))).to(DEV),
                                    32, DT[out])).astype(np.float64)
        want = B.mx4_decode(c, byte, 32)
        # 6 * 2^127 and its like are past the largest number
        want = np.where(np.abs(want) > 3.4e38, np.sign(want) * np.inf, want)
        assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nan_infinity_and_zeros(dt):
    import sparse_mixture_experts_gate_amd as M
    v = _rand(3, 6, 200, dt=dt)
    v[0, 5], v[1, 40], v[2, 199] = float("nan"), float("inf"), float("-inf")
    v[3] = 0.0
    v[4, 32:64] = -0.0
    codes, scales = M.mx4_quantize(v)
    c, b = _same(codes, scales, v)
    assert b[0, 0] == b[1, 1] == b[2, 6] == 255 and not b[3].any()
    got = host(M.mx4_dequantize(codes, scales, 200))
    assert np.array_equal(got, B.mx4_decode(c, b, 200), equal_nan=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_by_permutation_and_strides(dt):
    """Rows through perm, zeros for entries outside; rows of a wider matrix."""
    import sparse_mixture_experts_gate_amd as M
    x = _rand(4, 20, 311, dt=dt)[:, 7:7 + 300]
    perm = torch.tensor([3, 3, -1, 19, 0, 20, 7, 2 ** 31 - 1, 5], dtype=torch.int32, device=DEV)
    hp = host(perm).astype(np.int64)
    want = np.where(((hp >= 0) & (hp < 20))[:, None], host(x)[np.clip(hp, 0, 19)], 0.0)
    codes, scales = M.mx4_quantize(x, perm)
    assert codes.shape == (9, 160)
    _same(codes, scales, torch.from_numpy(want))
    _same(*M.mx4_quantize(x), x)


@pytest.mark.parametrize("k", [1, 31, 96, 513])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_swiglu(k, dt):
    """What is quantized is silu(gate) * up in fp32, off by 8 units of 2^-24 or so
    (exp, quotient, two products): a code is the nearest, or its neighbour where that
    decides. Blocks whose largest value is next to a power of two are left out."""
    import sparse_mixture_experts_gate_amd as M
    x = _rand(5, 30, 2 * k, dt=dt, spread=1.0)
    x[3, 0] = -200.0
    got = host(M.mx4_dequantize(*M.mx4_quantize(x, act="swiglu"), k, torch.float32)).astype(np.float64)
    v = B.swiglu(host(x))
    pad = np.zeros((30, -(-k // 32) * 32))
    pad[:, :k] = v
    amax = np.abs(pad.reshape(30, -1, 32)).max(-1)
    m, e = np.frexp(amax)
    clear = (np.abs(m - 0.5) > 1e-5) & (np.abs(m - 1.0) > 1e-5)
    unit = np.repeat(2.0 ** (e - 3.0), 32, 1)[:, :k]
    a = np.abs(v) / unit
    half = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, np.maximum(1.0, a - 6)))
    # exp(-gate) past 2^128, the end of fp32, gives 0 for a value below |gate| 2^-128
    # |up|, and no gate here is past 2^8 in magnitude
    under = 2.0 ** -120 * np.abs(host(x).astype(np.float64)[:, k:])
    ok = np.abs(got - v) <= unit * (half + 1e-5) + under
    assert (ok | ~np.repeat(clear, 32, 1)[:, :k]).all()


def _offsets(rows, G, seed, first=0, last=None):
    g = np.random.default_rng(seed)
    cut = np.sort(g.integers(first, (rows if last is None else last) + 1, size=G - 1))
    return np.r_[first, cut, rows if last is None else last].astype(np.int32)


def _check_product(rows, G, n, k, dt="bf16", out="bf16", seed=0, first=0, last=None, act=None):
    import sparse_mixture_experts_gate_amd as M
    w = _rand(seed + 1, G, n, k, dt="bf16", spread=2.0)
    x = _rand(seed + 2, rows, 2 * k if act else k, dt=dt, spread=2.0)
    off = _offsets(rows, G, seed, first, last)
    lin = M.MX4Linear.from_weight(w)
    y = lin.forward(x, torch.from_numpy(off).to(DEV), act=act, out_dtype=DT[out])
    q = host(M.mx4_dequantize(*M.mx4_quantize(x, act=act), k, torch.float32)).astype(np.float64)
    ref, mag = B.mx4_product(q, host(lin.values()).astype(np.float64), off)
    inside = np.zeros(rows, bool)
    inside[off[0]:off[-1]] = True
    got = host(y).astype(np.float64)[inside]
    tol = (k / 64 + 8) * 2.0 ** -23 * mag[inside] + RND[out] * np.abs(ref[inside])
    bad = ~(np.abs(got - ref[inside]) <= tol)
    assert y.shape == (rows, n) and not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[:4],
                                                    got[bad][:4], ref[inside][bad][:4])


@pytest.mark.parametrize("rows,G,n,k", [
    (1, 1, 1, 1), (1, 1, 32, 64), (32, 1, 32, 64), (1, 3, 70, 33), (5, 2, 128, 256), (17, 4, 200, 300),
    (40, 3, 129, 257), (64, 1, 256, 512), (100, 7, 96, 1000), (128, 1, 128, 2048), (130, 64, 64, 128),
    (9, 512, 40, 70)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_product(rows, G, n, k, out):
    _check_product(rows, G, n, k, out=out)


@pytest.mark.parametrize("rows,G,n,k", [
    (700, 2, 300, 500), (2000, 3, 1000, 520), (1030, 1, 2050, 264), (1500, 5, 4096, 256),
    (4099, 3, 2048, 300), (6000, 2, 4100, 130), (8200, 9, 4096, 768)])
def test_larger_products(rows, G, n, k):
    """128 x 128 and 256 x 256 tiles, ragged on every side."""
    _check_product(rows, G, n, k, out="f32", seed=3)


@pytest.mark.parametrize("rows,G,n,k", [(50, 3, 70, 90), (5000, 3, 4096, 200)])
def test_rows_outside_the_groups_are_not_written(rows, G, n, k):
    import sparse_mixture_experts_gate_amd as M
    _check_product(rows, G, n, k, first=7, last=rows - 11)
    x, lin = _rand(1, rows, k), M.MX4Linear.from_weight(_rand(2, G, n, k))
    off = torch.from_numpy(_offsets(rows, G, 0, 7, rows - 11)).to(DEV)
    wide = torch.full((rows, n + 5), 7.0, device=DEV)
    desc = M.MoeMx4GemmDesc(rows=rows, n_groups=G, n=n, k=k, out_dtype=M.MOE_DT_F32, ld_y=n + 5)
    codes, scales = M.mx4_quantize(x)
    M.moe_mx4_gemm(desc, codes, scales, lin.codes, lin.scales, off, wide[:, 2:2 + n])
    want = lin.forward(x, off, out_dtype=torch.float32)
    assert torch.equal(wide[7:rows - 11, 2:2 + n], want[7:rows - 11])
    assert bool((wide[:7] == 7).all()) and bool((wide[rows - 11:] == 7).all())
    assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 2 + n:] == 7).all())


def test_types_activation_and_permutation():
    import sparse_mixture_experts_gate_amd as M
    _check_product(60, 3, 100, 333, dt="f32", out="f32")
    _check_product(60, 3, 100, 333, act="swiglu")
    x, lin = _rand(1, 20, 130, dt="bf16"), M.MX4Linear.from_weight(_rand(2, 2, 40, 130))
    perm = torch.tensor([4, 4, 19, -1, 0, 3, 7], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 3, 7], dtype=torch.int32, device=DEV)
    rows = x[perm.clamp(min=0).long()]
    rows[3] = 0
    assert torch.equal(lin.forward(x, off, perm=perm), lin.forward(rows, off))


def test_offsets_out_of_order_stay_inside():
    """Clamped to a valid split: groups before the bad one keep their products."""
    import sparse_mixture_experts_gate_amd as M
    x, lin = _rand(1, 50, 64), M.MX4Linear.from_weight(_rand(2, 4, 40, 64))
    good = lin.forward(x, torch.tensor([0, 10, 20, 30, 50], dtype=torch.int32, device=DEV))
    bad = lin.forward(x, torch.tensor([-9, 10, 5, 2 ** 31 - 1, 3], dtype=torch.int32, device=DEV))
    assert torch.equal(good[:10], bad[:10])


def test_nan_stays_in_its_row_and_column():
    import sparse_mixture_experts_gate_amd as M
    x, w = _rand(1, 40, 1100), _rand(2, 2, 50, 1100)
    off = torch.tensor([0, 25, 40], dtype=torch.int32, device=DEV)
    good = M.MX4Linear.from_weight(w).forward(x, off)
    x[7, 1099] = float("nan")
    w[1, 0, 3], w[1, 49, 1000] = float("inf"), float("nan")
    bad = M.MX4Linear.from_weight(w).forward(x, off)
    want = torch.zeros(40, 50, dtype=torch.bool, device=DEV)
    want[7] = True
    want[25:, 0] = want[25:, 49] = True
    assert torch.equal(bad.isnan(), want) and torch.equal(bad[~want], good[~want])


def test_from_blocks_and_values():
    """Scales in row order; gradients through the map go by GroupedLinear."""
    import sparse_mixture_experts_gate_amd as M
    w = _rand(1, 3, 40, 200, dt="bf16")
    c, b = B.mx4_encode(host(w))
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    lin, ref = M.MX4Linear.from_blocks(t(B.mx4_pack(c)), t(b)), M.MX4Linear.from_weight(w)
    assert torch.equal(lin.scales, ref.scales) and lin.k == 224
    assert torch.equal(lin.values()[..., :200], ref.values())
    off = torch.tensor([0, 5, 5, 30], dtype=torch.int32, device=DEV)
    dx = M.GroupedLinear(ref.values()).input_grad(_rand(2, 30, 40, dt="bf16"), off)
    assert dx.shape == (30, 200) and bool(dx.isfinite().all())


def test_no_rows():
    import sparse_mixture_experts_gate_amd as M
    codes, scales = M.mx4_quantize(torch.empty(0, 100, device=DEV))
    assert codes.shape == (0, 64) and scales.shape == (1, 0, 4)
    assert M.mx4_dequantize(codes, scales, 100).shape == (0, 100)
    lin = M.MX4Linear.from_weight(_rand(1, 2, 30, 100))
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert lin.forward(torch.empty(0, 100, device=DEV), off).shape == (0, 30)
    assert lin.forward(_rand(1, 5, 100), off).shape == (5, 30)  # rows of no group


@pytest.mark.parametrize("rows,n,k", [(33, 300, 4096), (200, 130, 1408), (64, 4096, 96)])
def test_one_row_more_or_less_changes_no_other(rows, n, k):
    """A row's product does not depend on the rows beside it, nor on the tile."""
    import sparse_mixture_experts_gate_amd as M
    x, lin = _rand(1, 9000, k, dt="bf16"), M.MX4Linear.from_weight(_rand(2, 1, n, k))
    off = lambda m: torch.tensor([0, m], dtype=torch.int32, device=DEV)
    want = lin.forward(x, off(9000), out_dtype=torch.float32)
    for m in (1, rows, rows + 1, 1000):
        assert torch.equal(lin.forward(x[:m], off(m), out_dtype=torch.float32), want[:m])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_permutation_of_no_rows(dt):
    """A rank without tokens: every entry of perm is outside."""
    import sparse_mixture_experts_gate_amd as M
    x = torch.empty(0, 96, dtype=DT[dt], device=DEV)
    perm = torch.tensor([-1, 0, 5], dtype=torch.int32, device=DEV)
    codes, scales = M.mx4_quantize(x, perm)
    assert codes.shape == (3, 48) and not codes.any() and not scales.any()
    lin = M.MX4Linear.from_weight(_rand(1, 1, 40, 96))
    y = lin.forward(x, torch.tensor([0, 3], dtype=torch.int32, device=DEV), perm=perm)
    assert y.shape == (3, 40) and not y.any()


@pytest.mark.parametrize("a,b", [(-100, -40), (-126, -3), (-60, -84), (-120, -120), (120, 20)])
def test_products_at_the_ends_of_the_range(a, b):
    """Sums below the normal numbers keep their bits, past the range they are infinite:
    32 equal products of powers of two are one power."""
    import sparse_mixture_experts_gate_amd as M
    lin = M.MX4Linear.from_weight(torch.full((1, 40, 32), 2.0 ** b, device=DEV))
    off = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    y = host(lin.forward(torch.full((5, 32), 2.0 ** a, device=DEV), off, out_dtype=torch.float32))
    with np.errstate(over="ignore"):
        assert (y == np.float32(2.0 ** (a + b + 5))).all()


@pytest.mark.parametrize("rows,G,n,k", [
    (8, 8, 2816, 300), (64, 32, 1030, 257), (33, 4, 2817, 96), (100, 7, 2000, 1000), (40, 1, 5000, 70)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_products_of_few_rows_in_many_tiles(rows, G, n, k, out):
    """Past one 32 x 32 tile for each CU: 32 x 128 tiles."""
    _check_product(rows, G, n, k, out=out, seed=11)


@pytest.mark.parametrize("n", [4096, 4100, 9000])
def test_rows_outside_the_groups_of_few_rows(n):
    """Both tiles of 32 rows: rows and columns around the outputs are left as they were."""
    import sparse_mixture_experts_gate_amd as M
    rows, G, k = 40, 2, 520
    x, lin = _rand(1, rows, k), M.MX4Linear.from_weight(_rand(2, G, n, k))
    off = torch.tensor([3, 20, 37], dtype=torch.int32, device=DEV)
    codes, scales = M.mx4_quantize(x)
    for out, dt in ((M.MOE_DT_F32, torch.float32), (M.MOE_DT_BF16, torch.bfloat16)):
        wide = torch.full((rows, n + 5), 7.0, device=DEV, dtype=dt)
        desc = M.MoeMx4GemmDesc(rows=rows, n_groups=G, n=n, k=k, out_dtype=out, ld_y=n + 5)
        M.moe_mx4_gemm(desc, codes, scales, lin.codes, lin.scales, off, wide[:, 2:2 + n])
        want = lin.forward(x, off, out_dtype=dt)
        assert torch.equal(wide[3:37, 2:2 + n], want[3:37])
        wide[3:37, 2:2 + n] = 7.0
        assert bool((wide == 7).all())
