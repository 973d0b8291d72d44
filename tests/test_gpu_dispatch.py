"""Tokens sorted by expert and returned, on the GPU. Places and moved rows are
compared for equality. Sums: y adds K products in fp32, each addition off by u =
2^-24 of the terms; dweight's sum of d products runs 32 deep per lane and sweep of
8192 values (one of 2048 or 1024 at smaller widths), then over 64 lanes and 4 waves:
48 + d / 128 additions at most. bf16 outputs add 2^-8 of the value."""
import numpy as np
import pytest
import torch

import oracle.token_ops as B
from parity_util import host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.uint8}
RND = {"bf16": 2.0 ** -8, "f32": U}
DEV = "cuda:0"


def _idx(seed, T, K, E, gone=0.0, lowest=-1):
    """Selections, some of them of no expert here; duplicates within a token too."""
    g = np.random.default_rng(seed)
    idx = g.integers(0, E, size=(T, K)).astype(np.int32)
    idx[g.random((T, K)) < gone] = lowest
    return idx


def _rows(seed, n, d, dt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if dt == "fp8":
        return torch.randint(0, 255, (n, d), generator=g, device=DEV, dtype=torch.uint8)
    return torch.randn(n, d, generator=g, device=DEV).to(DT[dt])


def _place(idx, E, rows=None):
    """The sort in whole-array steps, checked against the oracle's pairs in its pins."""
    T, K = idx.shape
    flat = idx.reshape(-1)
    there = (flat >= 0) & (flat < E)
    order = np.flatnonzero(there)[np.argsort(flat[there], kind="stable")]
    rows = T * K if rows is None else rows
    perm, inv = np.full(rows, -1, np.int32), np.full(T * K, -1, np.int32)
    kept = order[:rows]
    perm[:len(kept)], inv[kept] = kept // K, np.arange(len(kept))
    off = np.minimum(np.searchsorted(flat[order], np.arange(E + 1)), rows).astype(np.int32)
    return off, perm, inv.reshape(T, K)


def test_whole_array_sort_is_the_oracles():
    for seed, (T, K, E, gone, rows) in enumerate([(9, 3, 4, 0.3, None), (9, 3, 4, 0.0, 10),
                                                  (1, 1, 1, 0.0, None), (5, 2, 7, 1.0, None)]):
        idx = _idx(seed, T, K, E, gone)
        for a, b in zip(_place(idx, E, rows), B.dispatch(idx, E, rows)):
            assert np.array_equal(a, b)


CASES = [  # T, K, E, gone, d, rows
    (1, 1, 1, 0.0, 1, None), (1, 8, 256, 0.0, 7168, None), (16, 8, 256, 0.0, 100, None),
    (16, 8, 32, 0.875, 7168, None), (33, 5, 3, 0.2, 33, 50), (7, 64, 512, 0.1, 17, None),
    (64, 2, 2, 1.0, 64, None), (300, 8, 64, 0.0, 130, 1000), (512, 8, 512, 0.3, 65, None),
    (513, 8, 512, 0.3, 65, None), (8192, 1, 7, 0.0, 3, None), (2000, 6, 64, 0.0, 1408, None),
    (3001, 7, 100, 0.5, 1025, 9000), (20000, 8, 65, 0.0, 5, None), (5000, 64, 257, 0.0, 2, 1),
    (1100, 3, 129, 1.0, 20, None)]


@pytest.mark.parametrize("T,K,E,gone,d,rows", CASES)
@pytest.mark.parametrize("dt", ["bf16", "f32", "fp8"])
def test_dispatch(T, K, E, gone, d, rows, dt):
    import sparse_mixture_experts_gate_amd as M
    idx = _idx(T + K, T, K, E, gone, lowest=E if T % 2 else -1)
    off, perm, inv = _place(idx, E, rows)
    x = _rows(1, T, d, dt)
    scale = _rows(2, T, -(-d // 128), "f32") if dt == "fp8" else None
    n = len(perm)
    into = _rows(3, n, d, dt)
    before = into.clone()
    o = M.TokenDispatch(E, rows).forward(x, torch.from_numpy(idx).to(DEV), scale, into)
    assert np.array_equal(host(o["offsets"]), off)
    assert np.array_equal(host(o["perm"]), perm)
    assert np.array_equal(host(o["inv"]), inv)
    kept = int(off[-1])
    src = torch.from_numpy(perm[:kept].astype(np.int64)).to(DEV)
    assert o["rows"] is into and torch.equal(into[:kept], x[src])
    assert torch.equal(into[kept:], before[kept:])
    if scale is not None:
        assert torch.equal(o["scale"][:kept], scale[src])
    s = M.TokenDispatch(E, rows).forward(None, torch.from_numpy(idx).to(DEV))
    assert s["rows"] is None and all(torch.equal(s[k], o[k]) for k in ("offsets", "perm", "inv"))


def test_no_tokens():
    import sparse_mixture_experts_gate_amd as M
    idx = torch.empty(0, 4, dtype=torch.int32, device=DEV)
    o = M.TokenDispatch(3).forward(torch.empty(0, 8, device=DEV), idx)
    assert o["offsets"].tolist() == [0, 0, 0, 0] and o["rows"].shape == (0, 8)
    y = M.TokenDispatch.combine(torch.empty(0, 8, device=DEV), o["inv"])
    assert y.shape == (0, 8)
    g = M.TokenDispatch.combine_grad(y, o["rows"], o["inv"], torch.empty(0, 4, device=DEV))
    assert g["drows"].shape == (0, 8) and g["dweight"].shape == (0, 4)


def _check_return(T, K, d, dt, idx, E, rows, weight, base):
    import sparse_mixture_experts_gate_amd as M
    _, perm, inv = _place(idx, E, rows)
    r = _rows(4, len(perm), d, dt)
    r[perm < 0] = float("nan")  # rows behind the last place are never read
    w = torch.rand(T, K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)) if weight else None
    if weight:
        w[torch.from_numpy(inv < 0).to(DEV)] = float("nan")  # nor weights without a place
    b = _rows(6, T, d, dt) if base else None
    dy = _rows(7, T, d, dt)
    ti = torch.from_numpy(inv).to(DEV)
    y = M.TokenDispatch.combine(r, ti, w, b)
    hr, hw = host(r).astype(np.float64), None if w is None else host(w).astype(np.float64)
    hb, hdy = None if b is None else host(b).astype(np.float64), host(dy).astype(np.float64)
    ok = inv >= 0
    picked = np.where(ok[..., None], hr[np.maximum(inv, 0)], 0.0)
    wt = np.where(ok, 1.0 if hw is None else hw, 0.0)
    ref = np.einsum("tk,tkd->td", wt, picked) + (0 if hb is None else hb)
    mag = np.einsum("tk,tkd->td", np.abs(wt), np.abs(picked)) + (0 if hb is None else np.abs(hb))
    got = host(y).astype(np.float64)
    assert (np.abs(got - ref) <= RND[dt] * np.abs(ref) + K * U * mag + 1e-38).all()
    before = r.clone()
    before[perm < 0] = 3.0
    o = M.TokenDispatch.combine_grad(dy, r, ti, w, into=before.clone())
    want = (wt[..., None] * hdy[:, None])[ok]
    got = host(o["drows"]).astype(np.float64)
    assert (np.abs(got[inv[ok]] - want) <= (RND[dt] + U) * np.abs(want) + 1e-38).all()
    assert (got[perm < 0] == 3.0).all()
    if weight:
        dw, mag = np.einsum("tkd,td->tk", picked, hdy), np.einsum("tkd,td->tk", np.abs(picked), np.abs(hdy))
        got = host(o["dweight"]).astype(np.float64)
        assert (np.abs(got - dw) <= (48 + d / 128) * U * mag + 1e-38).all()
        assert (got[~ok] == 0).all()
    else:
        assert o["dweight"] is None


@pytest.mark.parametrize("T,K,E,gone,d,rows", [
    (1, 1, 1, 0.0, 1, None), (1, 8, 256, 0.0, 7168, None), (16, 8, 32, 0.875, 7168, None),
    (33, 5, 3, 0.2, 33, 50), (7, 64, 512, 0.1, 17, None), (64, 2, 2, 1.0, 64, None),
    (100, 6, 64, 0.0, 2048, None), (50, 7, 9, 0.5, 1025, 200), (3, 3, 4, 0.0, 8193, None),
    (2, 4, 4, 0.0, 20001, None), (40, 16, 64, 0.3, 1407, None), (9, 15, 20, 0.0, 513, None)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("weight,base", [(True, True), (False, False), (True, False)])
def test_return_and_its_gradients(T, K, E, gone, d, rows, dt, weight, base):
    _check_return(T, K, d, dt, _idx(T + K, T, K, E, gone), E, rows, weight, base)


def test_same_expert_twice_in_a_token():
    idx = np.zeros((5, 4), np.int32)
    idx[2] = [1, 0, 1, 1]
    _check_return(5, 4, 100, "f32", idx, 2, None, True, True)


@pytest.mark.parametrize("T", [5, 3000])
def test_selections_of_any_value(T):
    """Everything outside 0 .. E - 1 is no expert, the type's ends among it."""
    import sparse_mixture_experts_gate_amd as M
    bad = np.array([-2 ** 31, 2 ** 31 - 1, -1, 4, 513, 1 << 9], np.int32)
    idx = np.random.default_rng(T).integers(0, 4, (T, 4)).astype(np.int32)
    idx[1::2, 1:3] = bad[np.arange(T // 2 * 2).reshape(-1, 2) % 6]
    off, perm, inv = _place(idx, 4)
    o = M.TokenDispatch(4).forward(None, torch.from_numpy(idx).to(DEV))
    for k, v in (("offsets", off), ("perm", perm), ("inv", inv)):
        assert np.array_equal(host(o[k]), v), k


def test_bad_places_are_left_out():
    """inv outside the sorted rows reads and writes nothing."""
    import sparse_mixture_experts_gate_amd as M
    inv = torch.tensor([[0, 7], [-5, 2 ** 31 - 1], [6, 1]], dtype=torch.int32, device=DEV)
    r = torch.arange(6.0, device=DEV).reshape(6, 1).expand(6, 40).contiguous()[:6]
    w = torch.full((3, 2), 2.0, device=DEV)
    y = M.TokenDispatch.combine(r, inv, w)
    assert y[:, 0].tolist() == [0.0, 0.0, 2.0]
    o = M.TokenDispatch.combine_grad(torch.ones(3, 40, device=DEV), r, inv, w, into=r.clone())
    assert o["drows"][:, 39].tolist() == [2.0, 2.0, 2.0, 3.0, 4.0, 5.0]
    assert o["dweight"].tolist() == [[0.0, 0.0], [0.0, 0.0], [0.0, 40.0]]


@pytest.mark.parametrize("d", [40, 1100, 3001])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strided_rows_and_places_of_inputs(d, dt):
    """Row strides of every matrix, y in base's place, drows in the rows' place."""
    import sparse_mixture_experts_gate_amd as M
    T, K, E = 21, 3, 5
    idx = torch.from_numpy(_idx(1, T, K, E, 0.3)).to(DEV)
    dtype = M.MOE_DT_BF16 if dt == "bf16" else M.MOE_DT_F32
    wide = lambda s, n: _rows(s, n, d + 9, dt)
    bx, bp, bb = wide(1, T), wide(2, T * K), wide(3, T)
    x, p, b = (t[:, 1:1 + d] for t in (bx, bp, bb))
    edges = [(t, t.clone()) for t in (bp, bb)]
    desc = M.MoeDispatchDesc(T=T, d=d, n_experts=E, top_k=K, dtype=dtype, ld_t=d + 9, ld_p=d + 9)
    i32 = dict(dtype=torch.int32, device=DEV)
    off, perm, inv = torch.empty(E + 1, **i32), torch.empty(T * K, **i32), torch.empty(T, K, **i32)
    M.moe_token_dispatch(desc, idx, x, None, off, perm, inv, p, None)
    ref = M.TokenDispatch(E).forward(x.contiguous(), idx)
    kept = int(off[-1])
    assert torch.equal(p[:kept], ref["rows"][:kept]) and torch.equal(inv, ref["inv"])
    w = torch.rand(T, K, device=DEV)
    want = M.TokenDispatch.combine(ref["rows"], inv, w, b.contiguous())
    grad = M.TokenDispatch.combine_grad(x.contiguous(), ref["rows"], inv, w)
    M.moe_token_combine(desc, p, inv, w, b, b)
    assert torch.equal(b, want)
    dw = torch.empty(T, K, device=DEV)
    M.moe_token_combine_backward(desc, x, p, inv, w, p, dw)
    assert torch.equal(p[:kept], grad["drows"][:kept]) and torch.equal(dw, grad["dweight"])
    for t, e in edges:
        assert torch.equal(t[:, :1], e[:, :1]) and torch.equal(t[:, 1 + d:], e[:, 1 + d:])


def test_gradients_against_differences():
    """Linear maps, so differences of any step are exact but for rounding: fp32
    sums of 60 terms of size 1."""
    import sparse_mixture_experts_gate_amd as M
    idx = torch.tensor([[0, 1], [1, -1], [2, 0]], dtype=torch.int32, device=DEV)
    d = 20
    x, w, dy = _rows(1, 3, d, "f32"), torch.rand(3, 2, device=DEV), _rows(2, 3, d, "f32")
    disp = M.TokenDispatch(3)

    def loss(x_, w_):
        o = disp.forward(x_, idx, into=torch.zeros(6, d, device=DEV))
        return float((M.TokenDispatch.combine(o["rows"], o["inv"], w_).double() * dy.double()).sum())

    o = disp.forward(x, idx, into=torch.zeros(6, d, device=DEV))
    g = M.TokenDispatch.combine_grad(dy, o["rows"], o["inv"], w)
    dx = M.TokenDispatch.combine(g["drows"], o["inv"])
    for i in [(0, 0), (1, 5), (2, 19)]:
        e = torch.zeros_like(x); e[i] = 1.0
        assert abs(loss(x + e, w) - loss(x - e, w) - 2 * float(dx[i])) < 1e-4
    for i in [(0, 0), (1, 1), (2, 1)]:
        e = torch.zeros_like(w); e[i] = 1.0
        assert abs(loss(x, w + e) - loss(x, w - e) - 2 * float(g["dweight"][i])) < 1e-4


@pytest.mark.parametrize("T,K", [(256, 8), (257, 8), (1024, 2), (1025, 1), (1024, 1), (30, 9), (3, 33)])
def test_both_sides_of_one_launch(T, K):
    """Pairs that one launch places and the next size up, rows of a wave and of a block."""
    import sparse_mixture_experts_gate_amd as M
    idx = _idx(T, T, K, 40, 0.1)
    off, perm, inv = _place(idx, 40)
    for d in (512, 520):
        x = _rows(2, T, d, "bf16")
        o = M.TokenDispatch(40).forward(x, torch.from_numpy(idx).to(DEV))
        assert np.array_equal(host(o["offsets"]), off) and np.array_equal(host(o["perm"]), perm)
        assert np.array_equal(host(o["inv"]), inv)
        n = int(off[-1])
        assert torch.equal(o["rows"][:n], x[torch.from_numpy(perm[:n].astype(np.int64)).to(DEV)])
        _check_return(T, K, d, "f32", idx, 40, None, True, False)


@pytest.mark.parametrize("T,d", [(256, 2056), (257, 2056), (260, 7168), (300, 4099), (20, 2049)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_long_rows_by_few_and_by_more_tokens(T, d, dt):
    """A token's row by 1024 lanes and by 256."""
    _check_return(T, 5, d, dt, _idx(T, T, 5, 30, 0.3), 30, None, True, True)


@pytest.mark.parametrize("d", [100, 513, 2056, 4099, 7168, 8192, 8200])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_token_s_gradients_do_not_depend_on_the_others(d, dt):
    import sparse_mixture_experts_gate_amd as M
    T, K = 300, 4
    inv = torch.randperm(T * K, device=DEV).int().reshape(T, K)
    rows, dy = _rows(1, T * K, d, dt), _rows(2, T, d, dt)
    w = torch.rand(T, K, device=DEV)
    many = M.TokenDispatch.combine_grad(dy, rows, inv, w)
    y = M.TokenDispatch.combine(rows, inv, w)
    for n in (1, 7, 256):
        some = inv[:n].reshape(-1).long()
        own = torch.arange(n * K, device=DEV).int().reshape(n, K)
        few = M.TokenDispatch.combine_grad(dy[:n], rows[some], own, w[:n].contiguous())
        assert torch.equal(few["dweight"], many["dweight"][:n])
        assert torch.equal(few["drows"], many["drows"][some])
        assert torch.equal(M.TokenDispatch.combine(rows[some], own, w[:n].contiguous()), y[:n])
