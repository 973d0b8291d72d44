"""RMS norm on the GPU against the fp64 definition.

Bounds, from the arithmetic: every value is computed in fp32 (unit roundoff u =
2^-24). v is one rounding of x + residual; its squares are all positive, so their
sum of d terms, in a tree of depth <= log2(d) + d / 512 per lane, is off by that
many u of itself and rstd by half of it; o has two products more. 32 covers those
counts at the sizes here. bf16 outputs add half a unit in the last place, 2^-8 of
the value. Codes: the scaled value is off by the same few u, its rounding by 2^-4 of
the value, or half of 2^-9 below 2^-6.
"""
import numpy as np
import pytest
import torch

import oracle.token_ops as B
from oracle.moe_oracle import e4m3_decode
from parity_util import host

pytestmark = pytest.mark.gpu

U, C = 2.0 ** -24, 32.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
RND = {"bf16": 2.0 ** -8, "f32": U}
SHAPES = [(1, 1), (1, 7168), (3, 127), (5, 128), (2, 129), (7, 513), (4, 1000), (3, 2047),
          (2, 4096), (3, 7167), (2, 8193), (1, 16384), (2, 16385), (2, 20000)]


def _rand(seed, *shape, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda:0") * scale + shift


def _close(got, ref, tol, what):
    got, ref = host(got).astype(np.float64), np.asarray(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           got[bad][:3], ref[bad][:3])


def _check(o, x, r, w, eps, dt):
    y, v, rstd = B.rmsnorm(host(x), None if w is None else host(w), eps,
                           None if r is None else host(r))
    _close(o["rstd"], rstd, C * U * rstd, "rstd")
    if o["y"] is not None:
        _close(o["y"], y, (RND[dt] + C * U) * np.abs(y) + 1e-38, "y")
    if r is not None:
        _close(o["sum"], v, RND[dt] * np.abs(v) + U * np.abs(v) + 1e-38, "sum")
    if o["codes"] is not None:
        _, scale = B.tiles(y)
        _close(o["scale"], scale, C * U * scale, "scale")
        q = y / np.repeat(scale, 128, 1)[:, :y.shape[1]]
        got = e4m3_decode(host(o["codes"]))
        tol = np.maximum(2.0 ** -4 * np.abs(q), 2.0 ** -10) + 2 * C * U * np.abs(q)
        bad = ~(np.abs(got - q) <= tol)
        assert not bad.any(), (int(bad.sum()), got[bad][:3], q[bad][:3])


@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("res", [False, True])
def test_forward(n, d, dt, res):
    import sparse_mixture_experts_gate_amd as M
    x = _rand(1, n, d, scale=2.0).to(DT[dt])
    r = _rand(2, n, d).to(DT[dt]) if res else None
    norm = M.RMSNorm(_rand(3, d, scale=0.2, shift=1.0), 1e-5)
    both = norm.forward(x, r, codes=True)
    _check(both, x, r, norm.weight, 1e-5, dt)
    rows, codes = norm.forward(x, r), norm.forward(x, r, rows=False, codes=True)
    assert rows["codes"] is None and codes["y"] is None
    assert torch.equal(rows["y"], both["y"]) and torch.equal(codes["codes"], both["codes"])
    assert torch.equal(codes["scale"], both["scale"])


def _check_backward(o, dy, x, rstd, w, dr, dt):
    hx, hdy, hr = (host(t).astype(np.float64) for t in (x, dy, rstd))
    dx, dw = B.rmsnorm_backward(hdy, hx, hr, None if w is None else host(w),
                                None if dr is None else host(dr))
    g = np.abs(hdy * (1.0 if w is None else host(w).astype(np.float64)))
    z = np.abs(hx * hr[:, None])
    terms = hr[:, None] * (g + z * (g * z).mean(1, keepdims=True))
    if dr is not None:
        terms = terms + np.abs(host(dr))
    _close(o["dx"], dx, RND[dt] * np.abs(dx) + C * U * terms + 1e-38, "dx")
    depth = C + hx.shape[0] / 8.0  # a block adds its rows one after the other
    _close(o["dweight"], dw, depth * U * (np.abs(hdy) * z).sum(0) + 1e-38, "dweight")


@pytest.mark.parametrize("n,d", SHAPES + [(2500, 130), (1100, 1408), (700, 2050), (0, 64)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("res", [False, True])
def test_backward(n, d, dt, res):
    import sparse_mixture_experts_gate_amd as M
    x = _rand(1, n, d, scale=2.0).to(DT[dt])
    dy = _rand(5, n, d).to(DT[dt])
    dr = _rand(6, n, d).to(DT[dt]) if res else None
    op = M.RMSNorm(_rand(3, d, scale=0.2, shift=1.0))
    f = op.forward(x)
    o = op.backward(dy, x, f["rstd"], dr)
    if n == 0:
        assert not o["dweight"].any()
        return
    _check_backward(o, dy, x, f["rstd"], op.weight, dr, dt)


def test_gradient_against_differences():
    """dx and dweight of the kernels against central differences of the forward
    kernel. The loss has 96 terms of size 1; with h = 2^-6 its third derivative
    leaves h^2 / 6 of a few and the fp32 forward 96 u / h."""
    import sparse_mixture_experts_gate_amd as M
    x, w, dy = _rand(1, 4, 24), _rand(2, 24, shift=1.0), _rand(4, 4, 24)
    op = M.RMSNorm(w)
    o = op.backward(dy, x, op.forward(x)["rstd"])
    loss = lambda x_, w_: float((M.RMSNorm(w_).forward(x_)["y"].double() * dy.double()).sum())
    h = 2.0 ** -6
    for i in [(0, 0), (1, 7), (3, 23)]:
        e = torch.zeros_like(x); e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - float(o["dx"][i])) < 2e-3
    for j in (0, 11):
        e = torch.zeros_like(w); e[j] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - float(o["dweight"][j])) < 2e-3


@pytest.mark.parametrize("d", [96, 1000, 5000, 17000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strided_rows_in_place_and_no_weight(d, dt):
    """Row strides on every operand, outputs in place of inputs, no weight; the
    columns between rows stay as they were."""
    import sparse_mixture_experts_gate_amd as M
    n, ld = 5, d + 13
    big, rbig = _rand(1, n, ld).to(DT[dt]), _rand(2, n, ld).to(DT[dt])
    qbig = torch.full((n, ld), 99, dtype=torch.uint8, device="cuda:0")
    x, r, q = big[:, 3:3 + d], rbig[:, 5:5 + d], qbig[:, 1:1 + d]
    x0, r0 = x.clone(), r.clone()
    around = lambda: [t.clone() for t in (big[:, :3], big[:, 3 + d:], rbig[:, :5], rbig[:, 5 + d:],
                                          qbig[:, :1], qbig[:, 1 + d:])]
    edges = around()
    rstd = torch.empty(n, device="cuda:0")
    scale = torch.empty(n, -(-d // 128), device="cuda:0")
    desc = M.MoeRmsNormDesc(n=n, d=d, dtype=M.MOE_DT_BF16 if dt == "bf16" else M.MOE_DT_F32, eps=1e-6,
                            ld_x=ld, ld_r=ld, ld_y=ld, ld_s=ld, ld_q=ld)
    M.moe_rmsnorm_forward(desc, x, r, None, x, q, scale, r, rstd)  # y -> x, sum -> r
    _check({"y": x, "sum": r, "rstd": rstd, "codes": q.contiguous(), "scale": scale}, x0, r0, None,
           1e-6, dt)
    assert all(torch.equal(a, b) for a, b in zip(edges, around()))
    dbig = _rand(3, n, ld).to(DT[dt])
    dy, edges = dbig[:, 2:2 + d], dbig.clone()
    dy0 = dy.clone()
    dw = torch.empty(d, device="cuda:0")
    ws = torch.empty(M.moe_rmsnorm_backward_workspace_size(desc), dtype=torch.uint8, device="cuda:0")
    M.moe_rmsnorm_backward(desc, dy, r, None, rstd, None, dy, dw, ws)  # dx in place of dy
    _check_backward({"dx": dy, "dweight": dw}, dy0, r, rstd, None, None, dt)
    assert torch.equal(dbig[:, :2], edges[:, :2]) and torch.equal(dbig[:, 2 + d:], edges[:, 2 + d:])


@pytest.mark.parametrize("d", [200, 3000, 17000])
def test_zero_rows_tiny_values_nan_and_infinity(d):
    """A row of zeros and a tile below 2^-100 get scale 1 and zero codes; NaN and
    infinity stay in their own row, and their tiles' codes are NaN."""
    import sparse_mixture_experts_gate_amd as M
    x = _rand(1, 5, d)
    x[1] = 0
    x[2, 7], x[3, 150] = float("nan"), float("inf")
    w = torch.ones(d, device="cuda:0")
    w[128:] = 1e-35
    o = M.RMSNorm(w).forward(x, codes=True)
    y, codes, scale = host(o["y"]), host(o["codes"]), host(o["scale"])
    assert not y[1].any() and not codes[1].any() and (scale[1] == 1).all()
    assert (scale[[0, 4], 1:] == 1).all() and not codes[[0, 4], 128:].any()
    assert np.isnan(y[2]).all() and (codes[2] == 0x7f).all() and np.isnan(scale[2]).all()
    assert np.isnan(y[3, 150]) and (codes[3, 128:min(256, d)] == 0x7f).all()
    good = torch.tensor([0, 4], device="cuda:0")
    again = M.RMSNorm(w).forward(x[good].contiguous(), codes=True)
    for k in ("y", "codes", "scale", "rstd"):
        assert torch.equal(again[k], o[k][good])


def test_vectors_at_any_element():
    """Weight and statistics that do not start on 16 bytes."""
    import sparse_mixture_experts_gate_amd as M
    flat = _rand(1, 333, shift=1.0)
    x, dy = _rand(2, 6, 300), _rand(3, 6, 300)
    op, ref = M.RMSNorm(flat[1:301]), M.RMSNorm(flat[1:301].clone())
    a, b = op.forward(x), ref.forward(x)
    assert torch.equal(a["y"], b["y"])
    rstd = torch.cat([b["rstd"][:1], b["rstd"]])[1:]
    assert torch.equal(op.backward(dy, x, rstd)["dweight"], ref.backward(dy, x, b["rstd"])["dweight"])


def test_more_rows_than_a_launch_counts():
    """Rows of one value: 2^24 + 5 of them, past a launch of 2^22 blocks of 4."""
    import sparse_mixture_experts_gate_amd as M
    n = (1 << 24) + 5
    x = torch.full((n, 1), 3.0, dtype=torch.bfloat16, device="cuda:0")
    o = M.RMSNorm(None, 0.0).forward(x, codes=True)
    assert bool((o["y"] == 1).all()) and bool((o["codes"] == 0x7e).all())
    assert bool(((o["scale"] * 448 - 1).abs() <= 8 * U).all())
    d = M.RMSNorm(None, 0.0).backward(x, x, o["rstd"])
    # a row of one value: its norm does not move but for a few u of 3 * 1/3
    assert bool((d["dx"].abs() <= 16 * U).all())


@pytest.mark.parametrize("n", [511, 512, 513])
@pytest.mark.parametrize("d", [31, 700, 1500, 2300, 4500, 9000])
def test_both_ways_to_dweight(n, d):
    """From the rows' own launch and from partial rows; dresidual's place for dx."""
    import sparse_mixture_experts_gate_amd as M
    for dt in ("bf16", "f32"):
        x, dy, dr = (_rand(s, n, d).to(DT[dt]) for s in (1, 2, 3))
        op = M.RMSNorm(_rand(4, d, scale=0.2, shift=1.0))
        f = op.forward(x)
        o = op.backward(dy, x, f["rstd"], dr)
        _check_backward(o, dy, x, f["rstd"], op.weight, dr, dt)
        again = op.backward(dy, x, f["rstd"], dr)
        assert torch.equal(again["dweight"], o["dweight"])
        desc = op._desc(x)
        for place in (dr.clone(), dy.clone()):
            a, b = (place, dy) if torch.equal(place, dr) else (dr, place)
            dw = torch.empty(d, device="cuda:0")
            ws = torch.empty(M.moe_rmsnorm_backward_workspace_size(desc), dtype=torch.uint8,
                             device="cuda:0")
            M.moe_rmsnorm_backward(desc, b, x, op.weight, f["rstd"], a, place, dw, ws)
            assert torch.equal(place, o["dx"])
            _check_backward({"dx": place, "dweight": dw}, dy, x, f["rstd"], op.weight, dr, dt)
