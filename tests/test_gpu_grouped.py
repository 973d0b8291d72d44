"""Products grouped by expert on the GPU against the fp64 definition.

Bounds, from the arithmetic: bf16 products are exact in fp32, the sum over K
terms in any order is off by at most K u of its absolute terms (u = 2^-24), and
a bf16 output adds half a unit in the last place (8 significant bits: up to
2^-8 of the value).
"""
import numpy as np
import pytest
import torch

import oracle.block_ops as B
from parity_util import host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda:0") * scale).bfloat16()


def _lens(rows, groups, skew, seed):
    rs = np.random.RandomState(seed)
    p = (np.arange(groups) + 1.0) ** -skew
    return rs.multinomial(rows, rs.permutation(p / p.sum()))


def _off(lens, first=0):
    o = np.concatenate([[0], np.cumsum(lens)]) + first
    return o, torch.tensor(o, dtype=torch.int32, device="cuda:0")


def _ws(desc, op):
    import sparse_mixture_experts_gate_amd as M
    n = M.moe_grouped_gemm_workspace_size(desc, op)
    return torch.empty(n, dtype=torch.uint8, device="cuda:0") if n else None


def _close(got, ref, mag, terms, rnd, what):
    got = host(got).astype(np.float64)
    bad = ~(np.abs(got - ref) <= rnd * np.abs(ref) + (terms + 2) * U * mag + 1e-30)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           got[bad][:4], ref[bad][:4])


def _check(x, w, dy, off_h, off, what):
    import sparse_mixture_experts_gate_amd as M
    lin = M.GroupedLinear(w)
    hx, hw, hdy = (host(t).astype(np.float64) for t in (x, w, dy))
    G, n, k = w.shape
    inside = slice(off_h[0], off_h[-1])
    ax, aw, ady = np.abs(hx), np.abs(hw), np.abs(hdy)
    for dt, rnd in ((torch.bfloat16, 2.0 ** -8), (torch.float32, U)):
        y = lin.forward(x, off, out_dtype=dt)
        _close(y[inside], B.grouped(hx, hw, off_h)[inside], B.grouped(ax, aw, off_h)[inside], k,
               rnd, what + " y")
        dx = lin.input_grad(dy, off, out_dtype=dt)
        _close(dx[inside], B.grouped_dgrad(hdy, hw, off_h)[inside],
               B.grouped_dgrad(ady, aw, off_h)[inside], n, rnd, what + " dx")
    dw = M.GroupedLinear.weight_grad(dy, x, off)
    ref, mag = B.grouped_wgrad(hdy, hx, off_h), B.grouped_wgrad(ady, ax, off_h)
    most = int(np.max(np.diff(off_h)))
    _close(dw, ref, mag, most, U, what + " dw")
    # accumulation: one more rounded sum
    base = torch.randn(G, n, k, device="cuda:0")
    acc = M.GroupedLinear.weight_grad(dy, x, off, into=base.clone())
    _close(acc, ref + host(base), mag + np.abs(host(base)), most, U, what + " dw accumulated")


CASES = [
    # rows, groups, n, k, skew
    (1, 1, 1, 1, 0.0), (1, 3, 8, 8, 0.0), (3, 2, 64, 64, 0.0), (17, 5, 72, 200, 0.5),
    (64, 4, 128, 64, 0.0), (65, 1, 33, 65, 0.0), (130, 7, 129, 257, 1.0), (300, 512, 16, 24, 0.3),
    (257, 3, 256, 128, 0.8), (777, 64, 136, 88, 1.1), (900, 2, 512, 320, 0.2),
    (1000, 9, 407, 213, 0.5), (40, 16, 264, 1416, 0.0), (600, 1, 1032, 520, 0.0),
    (2048, 8, 248, 72, 0.6),
    # enough tiles for the 256 x 256 kernels: forward, input gradient, weight gradient
    (6000, 3, 2056, 264, 0.4), (6000, 3, 264, 2056, 0.4), (1500, 3, 2056, 2056, 0.3),
    # and of any alignment: 128 x 256
    (6000, 3, 2057, 263, 0.4), (6000, 3, 263, 2057, 0.4),
    # long contractions of few outputs: partial sums of several workgroups
    (20, 1, 64, 4104, 0.0), (20, 1, 4104, 72, 0.0), (9000, 2, 136, 72, 0.5),
    (20, 3, 65, 4001, 0.0), (21, 2, 4001, 65, 0.0), (9000, 2, 133, 71, 0.5),
]


@pytest.mark.parametrize("rows,groups,n,k,skew", CASES)
def test_products(rows, groups, n, k, skew):
    off_h, off = _off(_lens(rows, groups, skew, rows))
    x, dy = _rand(1, rows, k), _rand(2, rows, n)
    w = _rand(3, groups, n, k, scale=0.1)
    _check(x, w, dy, off_h, off, f"{rows}x{groups}x{n}x{k}")


@pytest.mark.parametrize("n,k,lens", [
    (2048, 2048, [600, 1, 700, 900, 500, 799, 0, 1500]),
    # more tiles than expected of so many rows: the last round's are shared
    (2048, 3208, [577] * 5 + [769] * 3), (3208, 2048, [577] * 5 + [769] * 3),
])
def test_tiles_of_192_rows(n, k, lens):
    off_h, off = _off(lens)
    x, dy = _rand(1, sum(lens), k), _rand(2, sum(lens), n)
    _check(x, _rand(3, len(lens), n, k, scale=0.1), dy, off_h, off, f"{n}x{k}")


def test_empty_groups_and_rows_outside():
    """Empty groups at both ends and inside; rows before the first and past the
    last group keep what they held; no rows at all."""
    import sparse_mixture_experts_gate_amd as M
    for k in (96, 91):
        lens = [0, 5, 0, 0, 130, 1, 0]
        off_h, off = _off(lens, first=7)
        rows = 7 + sum(lens) + 9
        x, dy, w = _rand(1, rows, k), _rand(2, rows, 80), _rand(3, len(lens), 80, k)
        _check(x, w, dy, off_h, off, "empty groups")
        y = torch.full((rows, 80), 7.0, device="cuda:0")
        dx = torch.full((rows, k), 7.0, device="cuda:0")
        desc = M.MoeGroupedDesc(rows=rows, n_groups=len(lens), n=80, k=k, out_dtype=M.MOE_DT_F32)
        M.moe_grouped_gemm(desc, x, w, off, y, _ws(desc, M.MOE_GROUPED_FORWARD))
        M.moe_grouped_gemm_dgrad(desc, dy, w, off, dx, _ws(desc, M.MOE_GROUPED_DGRAD))
        for t in (y, dx):
            assert bool((t[:7] == 7).all()) and bool((t[7 + sum(lens):] == 7).all())
        none = torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda:0")
        assert not M.GroupedLinear.weight_grad(dy, x, none).any()
        assert not M.GroupedLinear.weight_grad(dy[:0], x[:0], none).any()
        assert M.GroupedLinear(w).forward(x[:0], none).shape == (0, 80)


@pytest.mark.parametrize("pad", [0, 5, 8])
@pytest.mark.parametrize("n,k", [(64, 128), (200, 72)])
def test_strides(pad, n, k):
    """Operands and outputs inside wider buffers whose other columns hold NaN:
    none of it enters a product, and it is not overwritten."""
    import sparse_mixture_experts_gate_amd as M
    rows, G = 150, 3
    off_h, off = _off(_lens(rows, G, 0.4, 1))
    ldk, ldn = k + 2 * pad, n + 2 * pad
    nan = float("nan")
    X = torch.full((rows, ldk), nan, device="cuda:0").bfloat16()
    DY = torch.full((rows, ldn), nan, device="cuda:0").bfloat16()
    X[:, pad:pad + k], DY[:, pad:pad + n] = _rand(1, rows, k), _rand(2, rows, n)
    x, dy, w = X[:, pad:pad + k], DY[:, pad:pad + n], _rand(3, G, n, k)
    _check(x, w, dy, off_h, off, f"pad {pad}")
    Y = torch.full((rows, ldn), 7.0, device="cuda:0").bfloat16()
    desc = M.MoeGroupedDesc(rows=rows, n_groups=G, n=n, k=k, out_dtype=M.MOE_DT_BF16, ld_k=ldk,
                            ld_n=ldn)
    M.moe_grouped_gemm(desc, x, w, off, Y[:, pad:pad + n], _ws(desc, M.MOE_GROUPED_FORWARD))
    assert torch.equal(Y[:, pad:pad + n], M.GroupedLinear(w).forward(x, off))
    assert bool((Y[:, :pad] == 7).all()) and bool((Y[:, pad + n:] == 7).all())


def test_nan_stays_in_its_row_and_group():
    import sparse_mixture_experts_gate_amd as M
    for n, k in ((136, 192), (75, 61)):
        off_h, off = _off([40, 3, 200])
        x, w, dy = _rand(1, 243, k), _rand(2, 3, n, k), _rand(3, 243, n)
        y0 = M.GroupedLinear(w).forward(x, off)
        dw0 = M.GroupedLinear.weight_grad(dy, x, off)
        x[41, k // 2] = float("inf")
        x[100, 0] = float("nan")
        y = M.GroupedLinear(w).forward(x, off)
        rows = torch.ones(243, dtype=torch.bool, device="cuda:0")
        rows[41] = rows[100] = False
        assert torch.equal(y[rows], y0[rows])
        assert bool(torch.isnan(y[100]).all()) and not bool(torch.isfinite(y[41]).any())
        dw = M.GroupedLinear.weight_grad(dy, x, off)
        assert torch.equal(dw[0], dw0[0])
        assert bool(torch.isnan(dw[2, :, 0]).all()) and torch.equal(dw[2, :, 1:], dw0[2, :, 1:])
        w[1] = float("nan")
        y = M.GroupedLinear(w).forward(x, off)
        assert torch.equal(y[:40], y0[:40]) and bool(torch.isnan(y[40:43]).all())


def test_bad_offsets_are_clamped():
    """Offsets out of range or order are replaced by a valid split; groups
    before the first bad entry keep their products."""
    import sparse_mixture_experts_gate_amd as M
    x, w = _rand(1, 100, 64), _rand(2, 4, 96, 64)
    good = M.GroupedLinear(w).forward(x, torch.tensor([0, 30, 60, 60, 100], dtype=torch.int32,
                                                      device="cuda:0"))
    for bad in ([-5, 30, 60, 50, 1 << 30], [0, 30, 60, -7, 200]):
        o = torch.tensor(bad, dtype=torch.int32, device="cuda:0")
        y = M.GroupedLinear(w).forward(x, o)
        assert torch.equal(y, good)
        dw = M.GroupedLinear.weight_grad(y, x, o)
        assert bool(torch.isfinite(dw).all()) and not dw[2].any()


def test_gradients_against_differences():
    """<dx, e> and <dw, e> against differences of the forward, which is linear
    in each argument: exact but for the rounding of the terms."""
    import sparse_mixture_experts_gate_amd as M
    off_h, off = _off([9, 0, 40])
    x, w, dy = _rand(1, 49, 72), _rand(2, 3, 56, 72), _rand(3, 49, 56)
    ex, ew = _rand(4, 49, 72), _rand(5, 3, 56, 72)
    f = lambda x_, w_: M.GroupedLinear(w_).forward(x_, off, torch.float32).double()
    dx = M.GroupedLinear(w).input_grad(dy, off, torch.float32).double()
    dw = M.GroupedLinear.weight_grad(dy, x, off).double()
    for lhs, out in (((dx * ex).sum(), f(ex, w)), ((dw * ew).sum(), f(x, ew))):
        rhs = (out * dy.double()).sum()
        assert abs(float(lhs - rhs)) <= 200 * U * float((out.abs() * dy.double().abs()).sum()) + 1e-3


def test_streams_and_repeats_bit_for_bit():
    import sparse_mixture_experts_gate_amd as M
    off_h, off = _off(_lens(700, 6, 0.7, 2))
    x, w, dy = _rand(1, 700, 320), _rand(2, 6, 264, 320), _rand(3, 700, 264)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lin = M.GroupedLinear(w)
    one = lin.forward(x, off), lin.input_grad(dy, off), lin.weight_grad(dy, x, off)
    two = (lin.forward(x, off, stream=s), lin.input_grad(dy, off, stream=s),
           lin.weight_grad(dy, x, off, stream=s))
    s.synchronize()
    for a, b in zip(one, two):
        assert torch.equal(a, b)


def test_row_offsets_past_32_bits():
    """Rows whose byte offsets pass 2^32 in x, y and dy (strided rows), read
    and written at the right place."""
    import sparse_mixture_experts_gate_amd as M
    ld, rows = 1 << 20, 2200  # 2^21 bytes a row
    X = torch.zeros(rows, ld, dtype=torch.bfloat16, device="cuda:0")
    x = X[:, :64]
    x.copy_(_rand(1, rows, 64))
    w = _rand(2, 2, 64, 64)
    off_h, off = _off([5, rows - 5])
    y = M.GroupedLinear(w).forward(x, off, torch.float32)
    assert torch.equal(y, M.GroupedLinear(w).forward(x.contiguous(), off, torch.float32))
    desc = M.MoeGroupedDesc(rows=rows, n_groups=2, n=64, k=64, out_dtype=M.MOE_DT_BF16, ld_k=ld,
                            ld_n=ld)
    M.moe_grouped_gemm(desc, x, w, off, X[:, 128:192], _ws(desc, M.MOE_GROUPED_FORWARD))
    assert torch.equal(X[:, 128:192], y.bfloat16())
    dw = M.GroupedLinear.weight_grad(X[:, 128:192], x, off)
    ref = M.GroupedLinear.weight_grad(X[:, 128:192].contiguous(), x.contiguous(), off)
    assert torch.equal(dw, ref)
