"""Rows that end inside a lane's eight values, at every length near a multiple of
eight, in buffers of NaN that neither reads nor writes may touch.

Each result of bf16 rows is compared with that of the same values as fp32 rows, whose
ends take other accesses, and the fp32 one's with the definition in 64 bits. The fp32
arithmetic is the same for both, but for where products and sums are fused: 8 roundings
(2^-24 each) of the terms' magnitude for a value, d / 8 + 16 for a sum over a row's d
values, besides the one rounding to bf16 (2^-8 of the value)."""
import numpy as np
import pytest
import torch

import oracle.token_ops as B
from parity_util import host

pytestmark = pytest.mark.gpu

DEV, U = "cuda:0", 2.0 ** -24
LENGTHS = [*range(1, 26), *range(505, 522), 1023, 1025, 2041, 2047, 4089, 4095, 7165, 8191, 8199]


def _in_nan(t, gap=3):
    """t's values as rows that start at any element, NaN around them."""
    n, d = t.shape
    wide = torch.full((n + 2, d + 2 * gap + 1), float("nan"), dtype=t.dtype, device=DEV)
    rows = wide[1:1 + n, gap:gap + d]
    rows.copy_(t)
    return rows


def _untouched(rows, gap=3):
    n, d = rows.shape
    wide = rows._base if rows._base is not None else rows
    keep = torch.ones(wide.shape, dtype=torch.bool, device=DEV)
    keep[1:1 + n, gap:gap + d] = False
    return bool(torch.isnan(wide[keep]).all()) and not bool(torch.isnan(rows).any())


def _values(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).bfloat16()


def _near(got, ref, mag, what, n=8.0):
    """bf16 `got` is fp32 `ref`, rounded, but for n roundings of the terms' magnitude."""
    got, ref, mag = (host(t).astype(np.float64) for t in (got, ref, mag))
    bad = ~(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * n * U * mag)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3],
                           ref[bad][:3])


@pytest.mark.parametrize("d", LENGTHS)
def test_norms(d):
    import sparse_mixture_experts_gate_amd as M
    n = 5
    x, r, dy = (_values(s, n, d) for s in (1, 2, 3))
    w, b = _values(4, d).float(), _values(5, d).float()
    xs, rs, dys = (_in_nan(t) for t in (x, r, dy))
    f = lambda t: t.float()
    for N in (M.RMSNorm(w), M.LayerNorm(w, b)):
        lo, hi = N.forward(xs, rs), N.forward(f(x), f(r))
        s = hi["sum"].abs().amax(1, keepdim=True).expand(n, d)
        _near(lo["sum"], hi["sum"], hi["sum"].abs(), "sum", 1.0)
        rstd = hi["rstd"][:, None]
        _near(lo["y"], hi["y"], (d / 8 + 16) * (s * rstd * w.abs() + b.abs()), "y")
        stats = [hi[k] for k in ("mean", "rstd") if k in hi]
        v = _in_nan(hi["sum"].bfloat16())
        lo, hi = N.backward(dys, v, *stats, rs), N.backward(f(dy), f(v), *stats, f(r))
        g = (dy.abs().amax(1, keepdim=True) * w.abs().max()).float().expand(n, d)
        z = 1 + 2 * s * rstd
        _near(lo["dx"], hi["dx"], (d / 8 + 16) * rstd * g * z * z + r.abs(), "dx")
        dw, ref = (host(o["dweight"]).astype(np.float64) for o in (lo, hi))
        top = host((f(dy).abs() * z).sum(0)).astype(np.float64)
        assert (np.abs(dw - ref) <= 16 * U * top).all()
    y, _, rstd = B.rmsnorm(host(f(x)), host(w), 1e-6, host(f(r)))
    got = host(M.RMSNorm(w).forward(f(x), f(r))["y"]).astype(np.float64)
    assert (np.abs(got - y) <= 32 * U * np.abs(y) + 1e-38).all()
    assert all(_untouched(t) for t in (xs, rs, dys))


@pytest.mark.parametrize("d", LENGTHS)
def test_dispatch_and_return(d):
    import sparse_mixture_experts_gate_amd as M
    T, K, E = 6, 3, 4
    g = torch.Generator(device=DEV)
    g.manual_seed(d)
    idx = torch.randint(-1, E, (T, K), generator=g, device=DEV, dtype=torch.int32)
    x, base, dy = (_values(s, T, d) for s in (1, 2, 3))
    w = torch.rand(T, K, generator=g, device=DEV)
    s = M.TokenDispatch(E).forward(_in_nan(x), idx)
    kept = int(s["offsets"][-1])
    perm = s["perm"][:kept].long()
    assert torch.equal(s["rows"][:kept], x[perm]) and kept == int((idx >= 0).sum())
    rows = torch.full((T * K, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    rows[:kept] = s["rows"][:kept]
    y = M.TokenDispatch.combine(_in_nan(rows), s["inv"], w, base)
    full = rows.float().nan_to_num()
    ref = M.TokenDispatch.combine(full, s["inv"], w, base.float())
    picked = torch.where((idx >= 0)[..., None], x[:, None].float(), 0.0)
    mag = (w[..., None] * picked.abs()).sum(1) + base.float().abs()
    _near(y, ref, mag, "return")
    exact = host((w.double()[..., None] * picked.double()).sum(1) + base.double())
    assert (np.abs(host(ref) - exact) <= 8 * U * host(mag)).all()
    dys, into = _in_nan(dy), torch.full_like(rows, 3.0)
    lo = M.TokenDispatch.combine_grad(dys, rows, s["inv"], w, into)
    hi = M.TokenDispatch.combine_grad(dy.float(), full, s["inv"], w)
    assert torch.equal(lo["drows"][:kept], hi["drows"][:kept].bfloat16())
    assert (lo["drows"][kept:] == 3.0).all() and _untouched(dys)
    top = host((picked.abs() * dy.float().abs()[:, None]).sum(2))
    diff = np.abs(host(lo["dweight"]) - host(hi["dweight"]))
    assert (diff <= 2 * (d / 8 + 16) * U * top).all()


@pytest.mark.parametrize("d", [*LENGTHS, 127, 129, 255, 257])
@pytest.mark.parametrize("rows", [3, 70])
def test_4bit_values(d, rows):
    import sparse_mixture_experts_gate_amd as M
    x = _values(1, rows, d)
    xs = _in_nan(x)
    perm = torch.tensor([rows - 1, -1, 0, rows, 1], dtype=torch.int32, device=DEV)
    picked = torch.where(((perm >= 0) & (perm < rows))[:, None], x[perm.clamp(0, rows - 1).long()],
                         torch.zeros_like(x[:1]))
    for args, v in (((xs,), x), ((xs, perm), picked), ((x[None].repeat(3, 1, 1),), None)):
        codes, scales = M.mx4_quantize(*args)
        if v is None:
            codes, scales, v = codes[1], scales[1], x
        c, b = B.mx4_encode(host(v))
        assert np.array_equal(host(codes), B.mx4_pack(c))
        assert np.array_equal(host(scales), B.mx4_words(b))
        for out in (torch.bfloat16, torch.float32):
            back = M.mx4_dequantize(codes.contiguous(), scales.contiguous(), d, out)
            assert np.array_equal(host(back), B.mx4_decode(c, b, d))
    wide = _in_nan(_values(2, rows, 2 * d))
    lo = M.mx4_dequantize(*M.mx4_quantize(wide, act="swiglu"), d, torch.float32)
    hi = M.mx4_dequantize(*M.mx4_quantize(wide.float(), act="swiglu"), d, torch.float32)
    assert torch.equal(lo, hi)


@pytest.mark.parametrize("k", [31, 128, 129, 256, 257])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_4bit_values_of_many_narrow_rows(k, dt):
    """More rows than the choice of fewer per workgroup, ragged ends of several matrices."""
    import sparse_mixture_experts_gate_amd as M
    v = _values(3, 3, 30011, k).to(dt)
    codes, scales = M.mx4_quantize(v)
    pick = np.r_[0:70, 15000:15040, 30011 - 70:30011]
    c, b = B.mx4_encode(host(v[:, torch.from_numpy(pick).to(DEV)]))
    assert np.array_equal(host(codes)[:, pick], B.mx4_pack(c))
    assert np.array_equal(host(scales)[:, :, pick], B.mx4_words(b))
    back = M.mx4_dequantize(codes, scales, k, dt)
    assert np.array_equal(host(back)[:, pick], B.mx4_decode(c, b, k))
