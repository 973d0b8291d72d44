"""The operators on a token's way together, as a program uses them: 4-bit experts of
one rank behind norm and router, E4M3 tiles into the layer's FP8 experts, a training
step; and their calls under graph capture, from several threads, on other streams and
past 2^32 bytes."""
import threading

import numpy as np
import pytest
import torch

import oracle as O
import oracle.token_ops as B
import sparse_mixture_experts_gate_amd as M
from parity_util import TOL, host, row_rel_err
from sparse_mixture_experts_gate_amd.workloads import CONFIGS, Workload, make_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U8 = 2.0 ** -8


def _rand(seed, *shape, dt=torch.float32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dt)


def _h64(t):
    return host(t).astype(np.float64)


def _product_close(y, q, w, off, k, kept):
    """The bound of a 4-bit product: (k / 64 + 8) 2^-23 of the terms, one rounding."""
    ref, mag = B.mx4_product(_h64(q), _h64(w), off)
    d = np.abs(_h64(y)[:kept] - ref[:kept])
    assert (d <= (k / 64 + 8) * 2.0 ** -23 * mag[:kept] + U8 * np.abs(ref[:kept])).all()


def test_4bit_experts_of_one_rank():
    """norm -> router -> sort (half of the experts are elsewhere) -> gate and up product
    of the sorted, quantized rows -> down product of the quantized activation -> return
    with gates onto the residual sum. Every step against its definition on the step's
    own inputs."""
    wl = CONFIGS["small_bf16"].with_(name="chain", T=150, d=256, E=8, K=3, I=160, Is=0, G=1, M=1,
                                     n_clusters=4)
    P = make_inputs(wl.with_(I=192), DEV)
    layer = M.MoELayer(wl.with_(I=192), P)
    x, r = P["x"], _rand(1, 150, 256, dt=torch.bfloat16)
    norm = M.RMSNorm(_rand(2, 256) * 0.1 + 1.0)
    f = norm.forward(x, r)
    route = layer.forward(f["y"])
    here = torch.where(route["topk_idx"] < 4, route["topk_idx"], -1).contiguous()
    plan = M.TokenDispatch(4).forward(None, here)
    w13, w2 = _rand(3, 4, 320, 256) * 0.05, _rand(4, 4, 256, 160) * 0.05
    up, down = M.MX4Linear.from_weight(w13), M.MX4Linear.from_weight(w2)
    gu = up.forward(f["y"], plan["offsets"], perm=plan["perm"])
    rows = down.forward(gu, plan["offsets"], act="swiglu")
    out = M.TokenDispatch.combine(rows, plan["inv"], route["topk_gate"], f["sum"])

    off, perm, inv = B.dispatch(host(here), 4)
    kept = int(off[-1])
    assert 0 < kept < 450 and np.array_equal(host(plan["perm"]), perm)
    q = M.mx4_dequantize(*M.mx4_quantize(f["y"][plan["perm"][:kept].long()].contiguous()), 256)
    _product_close(gu[:kept], q, up.values(), off, 256, kept)
    q = M.mx4_dequantize(*M.mx4_quantize(gu[:kept], act="swiglu"), 160)
    _product_close(rows[:kept], q, down.values(), off, 160, kept)
    g = host(route["topk_gate"])
    want = B.combine(np.nan_to_num(_h64(rows)), inv, g, _h64(f["sum"]))
    mag = B.combine(np.abs(np.nan_to_num(_h64(rows))), inv, g, np.abs(_h64(f["sum"])))
    assert (np.abs(_h64(out) - want) <= U8 * np.abs(want) + 3 * 2.0 ** -24 * mag).all()


def test_norm_tiles_into_the_fp8_experts():
    """The norm's E4M3 tiles, moved to their experts by the dispatch, are what
    moe_expert_ffn reads; its outputs against the oracle's on the same codes."""
    T = 200
    wl = Workload("tiles", T=T, d=256, E=16, K=4, I=256, Is=256, G=4, M=2, topn=2, act="bf16",
                  w="fp8", x_kind="normal", bias_kind="uniform", bias_amp=0.05, w_std=0.05, seed=21)
    P = make_inputs(wl, DEV)
    layer = M.MoELayer(wl, P)
    f = M.RMSNorm(_rand(2, 256) * 0.1 + 1.0).forward(P["x"], codes=True)
    route = layer.forward(f["y"])
    p = M.TokenDispatch(16).forward(f["codes"], route["topk_idx"], f["scale"])
    yp = torch.empty(T * 4, 256, dtype=torch.bfloat16, device=DEV)
    ysh = torch.empty(T, 256, dtype=torch.bfloat16, device=DEV)
    M.moe_expert_ffn(layer.desc(T), layer.weights, f["y"], p["perm"], p["rows"], p["scale"],
                     p["offsets"], yp, ysh, layer.workspace(T))
    y = M.TokenDispatch.combine(yp, p["inv"], route["topk_gate"], ysh)
    q13 = [O.quantize_blocks_128(host(w)) for w in P["w13"]]
    q2 = [O.quantize_blocks_128(host(w)) for w in P["w2"]]
    x = B.tile_values(host(f["codes"]), host(f["scale"]))
    off, perm, inv = B.dispatch(host(route["topk_idx"]), 16)
    ref = np.zeros((T * 4, 256))
    for e in range(16):
        s = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            ref[s] = O.moe_oracle._fp8_expert(x[perm[s]], *q13[e], *q2[e])
    assert row_rel_err(host(yp), ref) <= TOL["fp8"]
    want = B.combine(_h64(yp), inv, host(route["topk_gate"]), _h64(ysh))
    assert row_rel_err(host(y), want) <= 2 * U8


def test_training_step_against_autograd():
    """norm -> dispatch -> two maps per expert -> return, and back. Ten tensors on the
    way are rounded to bf16, 2^-8 of themselves at most each; rounding errors pass the
    linear steps like the values they sit on."""
    T, d, n, E, K = 96, 192, 128, 4, 2
    bf = torch.bfloat16
    x, r = _rand(1, T, d, dt=bf), _rand(2, T, d, dt=bf)
    wn, dout = _rand(3, d) * 0.2 + 1.0, _rand(4, T, d, dt=bf)
    w1, w2 = (_rand(5, E, n, d) * d ** -0.5).to(bf), (_rand(6, E, d, n) * n ** -0.5).to(bf)
    idx = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(i))[:K]
                       for i in range(T)]).int().to(DEV)
    gate = torch.softmax(_rand(7, T, K), 1)
    norm, disp = M.RMSNorm(wn), M.TokenDispatch(E)
    up, down = M.GroupedLinear(w1), M.GroupedLinear(w2)
    f = norm.forward(x, r)
    p = disp.forward(f["y"], idx)
    off = p["offsets"]
    h = up.forward(p["rows"], off)
    y = down.forward(h, off)
    out = disp.combine(y, p["inv"], gate, f["sum"])
    g = disp.combine_grad(dout, y, p["inv"], gate)
    dh = down.input_grad(g["drows"], off)
    drows = up.input_grad(dh, off)
    dy = disp.combine(drows, p["inv"])
    b = norm.backward(dy, f["sum"], f["rstd"], dout)
    got = {"out": out, "dx": b["dx"], "dweight": b["dweight"], "dgate": g["dweight"],
           "dw1": up.weight_grad(dh, p["rows"], off), "dw2": down.weight_grad(g["drows"], h, off)}

    leaf = lambda t: t.double().cpu().requires_grad_()
    X, WN, W1, W2, G = leaf(x.float() + r.float()), leaf(wn), leaf(w1), leaf(w2), leaf(gate)
    o = X * torch.rsqrt(X.square().mean(1, keepdim=True) + 1e-6) * WN
    ref, ci = [], idx.cpu().long()
    for t in range(T):
        ref.append(X[t] + sum(G[t, k] * (W2[ci[t, k]] @ (W1[ci[t, k]] @ o[t])) for k in range(K)))
    ref = torch.stack(ref)
    (ref * dout.double().cpu()).sum().backward()
    want = {"out": ref.detach(), "dx": X.grad, "dweight": WN.grad, "dgate": G.grad, "dw1": W1.grad,
            "dw2": W2.grad}
    for k, v in want.items():
        err = float((got[k].double().cpu() - v).norm() / v.norm())
        assert err <= 10 * U8, (k, err)


# ---- captured calls, streams, threads ----------------------------------------------

class _Work:
    """Calls of every operator, both forms of the dispatch and two product tiles."""

    def __init__(self):
        bf, d = torch.bfloat16, 300
        self.norm = M.RMSNorm(_rand(1, d))
        self.few, self.many = M.TokenDispatch(5), M.TokenDispatch(70)
        self.x, self.r = _rand(2, 20, d, dt=bf), _rand(3, 20, d, dt=bf)
        self.big = _rand(4, 3000, 64)
        g = torch.Generator(device=DEV).manual_seed(5)
        self.i0 = torch.randint(0, 5, (20, 3), generator=g, device=DEV).int()
        self.i1 = torch.randint(0, 70, (3000, 4), generator=g, device=DEV).int()
        self.w0, self.w1 = torch.rand(20, 3, device=DEV), torch.rand(3000, 4, device=DEV)
        self.lin = M.MX4Linear.from_weight(_rand(6, 5, 40, d))
        self.wide = M.MX4Linear.from_weight(_rand(7, 70, 256, 64))

    def inputs(self):
        return [(t, s) for t, s in ((self.x, 10), (self.r, 20), (self.big, 30))]

    def __call__(self, stream=None):
        s = dict(stream=stream)
        f = self.norm.forward(self.x, self.r, codes=True, **s)
        p = self.few.forward(f["y"], self.i0, **s)
        q = self.few.forward(f["codes"], self.i0, f["scale"], **s)
        y = self.lin.forward(p["rows"], p["offsets"], **s)
        back = M.TokenDispatch.combine(p["rows"], p["inv"], self.w0, self.x, **s)
        g = M.TokenDispatch.combine_grad(back, p["rows"], p["inv"], self.w0, **s)
        b = self.norm.backward(back, f["sum"], f["rstd"], self.x, **s)
        m = self.many.forward(self.big, self.i1, **s)
        z = self.wide.forward(m["rows"], m["offsets"], out_dtype=torch.float32, **s)
        k = M.TokenDispatch.combine(z, m["inv"], self.w1, **s)
        v = M.mx4_dequantize(*M.mx4_quantize(self.big, **s), 64, **s)
        outs = [*f.values(), *p.values(), *q.values(), y, back, *g.values(), *b.values(),
                *m.values(), z, k, v]
        return [t for t in outs if t is not None]


def test_captured_calls_replay_with_new_inputs():
    work = _Work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = work()
    with torch.cuda.stream(side):  # larger eager calls replace the stream's buffers
        M.TokenDispatch(512).forward(None, torch.zeros(40000, 8, dtype=torch.int32, device=DEV))
        M.MX4Linear.from_weight(_rand(1, 1, 64, 4096)).forward(
            _rand(2, 5000, 4096), torch.tensor([0, 5000], dtype=torch.int32, device=DEV))
        junk = [torch.full((s,), float("nan"), device=DEV) for s in (1 << 12, 1 << 16, 1 << 20)
                for _ in range(8)]
    side.synchronize()
    for i in range(4):
        for t, seed in work.inputs():
            t.copy_(_rand(seed + i, *t.shape))
        work.i0.copy_(work.i0.roll(1, 0))
        work.i1.copy_(work.i1.roll(1, 0))
        want = [t.clone() for t in work()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (i, j)
        assert all(bool(torch.isnan(t).all()) for t in junk)


def test_other_streams():
    """stream= and a current stream other than the default: the same results."""
    work = _Work()
    want = work()
    torch.cuda.synchronize()
    s, c = torch.cuda.Stream(), torch.cuda.Stream()
    a = work(s)
    with torch.cuda.stream(c):
        b = work()
    torch.cuda.synchronize()
    for j, (w, x, y) in enumerate(zip(want, a, b)):
        assert torch.equal(w, x) and torch.equal(w, y), j


def test_threads_on_one_stream():
    works = [_Work(), _Work()]
    for t, seed in works[1].inputs():
        t.copy_(_rand(seed + 9, *t.shape))
    want = [w() for w in works]
    torch.cuda.synchronize()
    bad = []

    def calls(i):
        for n in range(12):
            bad.extend((i, n, j) for j, (a, b) in enumerate(zip(works[i](), want[i]))
                       if not torch.equal(a, b))

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]


# ---- past 2^32 bytes -------------------------------------------------------------------

def test_rows_past_4_gib():
    """Rows behind 2^32 bytes of every row matrix against a call on those rows alone."""
    T, d, bf = 40000, 32768, torch.bfloat16
    x = torch.randint(-100, 100, (T, d), device=DEV, dtype=torch.int16).to(bf)
    idx = torch.stack([torch.zeros(T), torch.ones(T)], 1).int().to(DEV)
    o = M.TokenDispatch(2).forward(x, idx)
    assert o["rows"].numel() * 2 > 2 ** 32
    pick = torch.tensor([0, 1, 12345, T - 2, T - 1], device=DEV)
    for k in range(2):
        assert torch.equal(o["inv"][pick, k], (pick + k * T).int())
        assert torch.equal(o["rows"][pick + k * T], x[pick])
    y = M.TokenDispatch.combine(o["rows"], o["inv"])
    assert torch.equal(y[pick], (x[pick].float() * 2).to(bf))
    w = torch.full((T, 2), 0.5, device=DEV)
    g = M.TokenDispatch.combine_grad(x, o["rows"], o["inv"], w)
    assert torch.equal(g["drows"][pick + T], (x[pick].float() / 2).to(bf))
    small = M.TokenDispatch.combine_grad(x[pick], x[pick], torch.arange(5, device=DEV).int()[:, None],
                                         w[:5, :1].contiguous())
    assert torch.equal(g["dweight"][pick, 1], small["dweight"][:, 0])
    del g, y
    for width in (d, 8192):  # rows read again, rows in registers
        v = o["rows"].reshape(-1, width)
        norm = M.RMSNorm(None)
        a = norm.forward(v, codes=True)
        tail = v[-3:].contiguous()
        b = norm.forward(tail, codes=True)
        for key in ("y", "codes", "scale", "rstd"):
            assert torch.equal(a[key][-3:], b[key]), (width, key)
        da = norm.backward(v, v, a["rstd"])["dx"]
        assert torch.equal(da[-3:], norm.backward(tail, tail, b["rstd"])["dx"])
        del a, da


def test_4bit_codes_past_2_gib():
    rows, k = 70001, 65536
    x = torch.randint(-100, 100, (rows, k), device=DEV, dtype=torch.int8).to(torch.bfloat16)
    codes, scales = M.mx4_quantize(x)
    assert codes.numel() > 2 ** 31
    tail = x[-5:].contiguous()
    c, s = M.mx4_quantize(tail)
    assert torch.equal(codes[-5:], c) and torch.equal(scales[:, -5:], s)
    assert torch.equal(M.mx4_dequantize(codes, scales, k)[-5:], M.mx4_dequantize(c, s, k))
    lin = M.MX4Linear.from_weight(_rand(1, 1, 48, k))
    off = lambda n: torch.tensor([0, n], dtype=torch.int32, device=DEV)
    y = lin.forward(x, off(rows), out_dtype=torch.float32)
    assert torch.equal(y[-5:], lin.forward(tail, off(5), out_dtype=torch.float32))


def test_weights_past_4_gib():
    """Codes of the last expert behind 2^32 bytes, and its scales."""
    G, n, k = 9, 16384, 65536
    codes = torch.randint(0, 256, (G, n, k // 2), device=DEV, dtype=torch.uint8)
    scales = torch.randint(120, 130, (G, k // 128, n, 4), device=DEV, dtype=torch.uint8)
    assert codes.numel() > 2 ** 32
    x = _rand(1, 40, k)
    lin = M.MX4Linear(codes, scales, k)
    off = torch.tensor([0] * 9 + [40], dtype=torch.int32, device=DEV)
    last = M.MX4Linear(codes[8:].clone(), scales[8:].clone(), k)
    one = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    assert torch.equal(lin.forward(x, off), last.forward(x, one))
