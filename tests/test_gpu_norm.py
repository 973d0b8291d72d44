"""Layer norm on the GPU against the fp64 definition.

Bounds, from the arithmetic: every value is computed in fp32 (unit roundoff u =
2^-24) from exact inputs. v - mean carries at most a few u (|v| + |mean|), the
statistics a few u times the row's condition sqrt(1 + mean^2 / var); a sum of d
terms in a tree of depth <= log2(d) + d / 512 adds that many u of its absolute
terms. 32 covers those counts at the sizes here. bf16 outputs add half a unit
in the last place: with 8 significant bits up to 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import oracle.block_ops as B
from parity_util import host

pytestmark = pytest.mark.gpu

U, C = 2.0 ** -24, 32.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
RND = {"bf16": 2.0 ** -8, "f32": U}


def _rand(seed, *shape, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda:0") * scale + shift


def _close(got, ref, tol, what):
    got, ref = host(got).astype(np.float64), np.asarray(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           got[bad][:3], ref[bad][:3])


def _cond(v, mean, rstd):
    """Magnitude of the terms behind a normalized value (v, the terms of the
    mean, the terms of rstd), in units of it."""
    return (np.abs(v) + np.abs(v).mean(1, keepdims=True)) * rstd[:, None] + np.sqrt(
        1.0 + (mean * rstd) ** 2)[:, None] * np.abs((v - mean[:, None]) * rstd[:, None])


def _check_forward(o, x, r, w, b, eps, dt):
    y, v, mean, rstd = B.layernorm(host(x), None if w is None else host(w),
                                   None if b is None else host(b), eps,
                                   None if r is None else host(r))
    aw = 1.0 if w is None else np.abs(host(w))
    _close(o["mean"], mean, C * U * np.abs(v).mean(1) + 1e-30, "mean")
    _close(o["rstd"], rstd, C * U * rstd * np.sqrt(1.0 + (mean * rstd) ** 2), "rstd")
    if r is not None:
        _close(o["sum"], v, RND[dt] * np.abs(v) + U * np.abs(v), "sum")
    _close(o["y"], y, RND[dt] * np.abs(y) + C * U * (_cond(v, mean, rstd) * aw + np.abs(y)) + 1e-30,
           "y")


SHAPES = [(1, 1), (3, 2), (5, 7), (7, 512), (6, 513), (2, 1024), (3, 1409), (9, 2048), (2, 4095),
          (1, 7168), (3, 8193), (2, 16384), (2, 16385), (1, 20011)]


@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("res", [False, True])
def test_forward(n, d, dt, res):
    import sparse_mixture_experts_gate_amd as M
    x = _rand(1, n, d, scale=2.0, shift=0.5).to(DT[dt])
    r = _rand(2, n, d).to(DT[dt]) if res else None
    w, b = _rand(3, d, scale=0.2, shift=1.0), _rand(4, d, scale=0.1)
    o = M.LayerNorm(w, b, 1e-5).forward(x, r)
    _check_forward(o, x, r, w, b, 1e-5, dt)


def _check_backward(o, dy, x, mean, rstd, w, dr, dt):
    hx, hdy = host(x).astype(np.float64), host(dy).astype(np.float64)
    hm, hr = host(mean).astype(np.float64), host(rstd).astype(np.float64)
    dx, dw, db = B.layernorm_backward(hdy, hx, hm, hr, None if w is None else host(w),
                                      None if dr is None else host(dr))
    g = np.abs(hdy * (1.0 if w is None else host(w).astype(np.float64)))
    z = _cond(hx, hm, hr)
    terms = hr[:, None] * (g + g.mean(1, keepdims=True) + z * (g * z).mean(1, keepdims=True))
    if dr is not None:
        terms = terms + np.abs(host(dr))
    _close(o["dx"], dx, RND[dt] * np.abs(dx) + C * U * terms + 1e-30, "dx")
    depth = C + hx.shape[0] / 8.0  # a block adds its rows one after the other
    _close(o["dweight"], dw, depth * U * (np.abs(hdy) * z).sum(0) + 1e-30, "dweight")
    _close(o["dbias"], db, depth * U * np.abs(hdy).sum(0) + 1e-30, "dbias")


@pytest.mark.parametrize("n,d", SHAPES + [(2500, 130), (1100, 1408), (700, 2050), (0, 64)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("res", [False, True])
def test_backward(n, d, dt, res):
    import sparse_mixture_experts_gate_amd as M
    x = _rand(1, n, d, scale=2.0, shift=0.5).to(DT[dt])
    dy = _rand(5, n, d).to(DT[dt])
    dr = _rand(6, n, d).to(DT[dt]) if res else None
    w = _rand(3, d, scale=0.2, shift=1.0)
    op = M.LayerNorm(w, None)
    f = op.forward(x)
    o = op.backward(dy, x, f["mean"], f["rstd"], dr)
    if n == 0:
        assert not o["dweight"].any() and not o["dbias"].any()
        return
    _check_backward(o, dy, x, f["mean"], f["rstd"], w, dr, dt)


def test_gradient_against_differences():
    """dx, dweight and dbias of the kernels against central differences of the
    forward kernel. The loss has 96 terms of size 1; with h = 2^-6 its third
    derivative leaves h^2 / 6 of a few and the fp32 forward 96 u / h."""
    import sparse_mixture_experts_gate_amd as M
    x, w, b = _rand(1, 4, 24), _rand(2, 24, shift=1.0), _rand(3, 24)
    dy = _rand(4, 4, 24)
    op = M.LayerNorm(w, b)
    f = op.forward(x)
    o = op.backward(dy, x, f["mean"], f["rstd"])
    loss = lambda x_, w_, b_: float((M.LayerNorm(w_, b_).forward(x_)["y"].double() * dy.double()).sum())
    h = 2.0 ** -6
    for i in [(0, 0), (1, 7), (3, 23)]:
        e = torch.zeros_like(x); e[i] = h
        assert abs((loss(x + e, w, b) - loss(x - e, w, b)) / (2 * h) - float(o["dx"][i])) < 2e-3
    for j in (0, 11):
        e = torch.zeros_like(w); e[j] = h
        assert abs((loss(x, w + e, b) - loss(x, w - e, b)) / (2 * h) - float(o["dweight"][j])) < 2e-3
        assert abs((loss(x, w, b + e) - loss(x, w, b - e)) / (2 * h) - float(o["dbias"][j])) < 2e-3


@pytest.mark.parametrize("d", [96, 1000, 5000, 17000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strided_rows_in_place_and_no_weights(d, dt):
    """Row strides on every operand, outputs in place of inputs, no weight or
    bias; the columns between rows stay as they were."""
    import sparse_mixture_experts_gate_amd as M
    n, ld = 5, d + 13
    big = _rand(1, n, ld).to(DT[dt])
    rbig = _rand(2, n, ld).to(DT[dt])
    x, r = big[:, 3:3 + d], rbig[:, 5:5 + d]
    x0, r0 = x.clone(), r.clone()
    edges = [t.clone() for t in (big[:, :3], big[:, 3 + d:], rbig[:, :5], rbig[:, 5 + d:])]
    mean, rstd = torch.empty(n, device="cuda:0"), torch.empty(n, device="cuda:0")
    desc = M.MoeNormDesc(n=n, d=d, dtype=M.MOE_DT_BF16 if dt == "bf16" else M.MOE_DT_F32, eps=1e-6,
                         ld_x=ld, ld_r=ld, ld_y=ld, ld_s=ld)
    M.moe_layernorm_forward(desc, x, r, None, None, x, r, mean, rstd)  # y -> x, sum -> r
    _check_forward({"y": x, "sum": r, "mean": mean, "rstd": rstd}, x0, r0, None, None, 1e-6, dt)
    for t, e in zip((big[:, :3], big[:, 3 + d:], rbig[:, :5], rbig[:, 5 + d:]), edges):
        assert torch.equal(t, e)
    # backward: dx in place of dy
    dbig = _rand(3, n, ld).to(DT[dt])
    dy = dbig[:, 1:1 + d]
    dy0 = dy.clone()
    ws = torch.empty(M.moe_layernorm_backward_workspace_size(desc), dtype=torch.uint8,
                     device="cuda:0")
    dw, db = torch.empty(d, device="cuda:0"), torch.empty(d, device="cuda:0")
    M.moe_layernorm_backward(desc, dy, r, None, mean, rstd, x, dy, dw, db, ws)
    _check_backward({"dx": dy, "dweight": dw, "dbias": db}, dy0, r, mean, rstd, None, x, dt)
    # one of the column sums alone
    db2 = torch.empty(d, device="cuda:0")
    dx2 = torch.empty(n, ld, device="cuda:0", dtype=DT[dt])[:, :d]
    M.moe_layernorm_backward(desc, dy0.new_empty(n, ld)[:, :d].copy_(dy0), r, None, mean, rstd, x,
                             dx2, None, db2, ws)
    assert torch.equal(db2, db) and torch.equal(dx2, dy)


def test_special_rows():
    """A constant row has variance zero (y = bias), a large mean keeps its
    spread, and NaN or infinity stays in its own row."""
    import sparse_mixture_experts_gate_amd as M
    for d in (40, 3000, 17000):
        x = _rand(1, 6, d)
        x[0] = 3.0
        x[1] += 1.0e4
        x[2, d // 2] = float("nan")
        x[3, d - 1] = float("inf")
        w, b = _rand(3, d, shift=1.0), _rand(4, d)
        o = M.LayerNorm(w, b).forward(x)
        y = o["y"]
        # the mean of equal values is off by at most a few roundings of 3
        assert float((y[0] - b).abs().max()) <= 8 * 3 * U * float(o["rstd"][0]) * float(w.abs().max())
        assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())
        keep = [1, 4, 5]
        _check_forward({k: o[k][keep] for k in ("y", "mean", "rstd")}, x[keep], None, w, b, 1e-5,
                       "f32")


def test_stream_and_repeat_bit_for_bit():
    import sparse_mixture_experts_gate_amd as M
    x, dy = _rand(1, 1000, 1408).bfloat16(), _rand(2, 1000, 1408).bfloat16()
    op = M.LayerNorm(_rand(3, 1408), _rand(4, 1408))
    f = op.forward(x)
    a = op.backward(dy, x, f["mean"], f["rstd"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    f2 = op.forward(x, stream=s)
    b = op.backward(dy, x, f2["mean"], f2["rstd"], stream=s)
    s.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k])
    assert torch.equal(f["y"], f2["y"])
