"""Host-only checks of the entry points of dsmoe_tokens.h: exported symbols and
refusals, each before anything reaches a GPU; and what the objects refuse."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sparse_mixture_experts_gate_amd", "libdsmoe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libdsmoe.so not built")

P = 0x1000  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def T():
    from sparse_mixture_experts_gate_amd import _token_ops
    return _token_ops


def test_every_declared_symbol_is_exported_and_bound(T):
    names = T.header_symbols()
    assert set(names) == {
        "moe_rmsnorm_forward", "moe_rmsnorm_backward_workspace_size", "moe_rmsnorm_backward",
        "moe_token_dispatch_workspace_size", "moe_token_dispatch", "moe_token_combine",
        "moe_token_combine_backward", "moe_mx4_quantize", "moe_mx4_dequantize", "moe_mx4_gemm"}
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    import sparse_mixture_experts_gate_amd as M
    for n in names:
        assert n in exported and callable(getattr(M, n))


def _norm(T, **kw):
    return T.MoeRmsNormDesc(**{**dict(n=4, d=64, dtype=1, eps=1e-5), **kw})


def test_rmsnorm_refusals(T):
    lib = T.lib()

    def fwd(desc, **kw):
        a = {**dict(x=P, r=None, w=P, y=P, q=None, sc=None, s=None, rstd=P), **kw}
        return lib.moe_rmsnorm_forward(None if desc is None else ctypes.byref(desc), a["x"], a["r"],
                                       a["w"], a["y"], a["q"], a["sc"], a["s"], a["rstd"], None)

    assert fwd(None) == 1
    n = ctypes.c_size_t()
    for kw, st in [(dict(n=-1), 1), (dict(n=1 << 31), 2), (dict(d=0), 1), (dict(d=(1 << 20) + 1), 2),
                   (dict(dtype=2), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
                   (dict(eps=float("inf")), 1), (dict(ld_x=63), 1), (dict(ld_r=-1), 1),
                   (dict(ld_y=1 << 31), 1), (dict(ld_s=1), 1), (dict(ld_q=63), 1)]:
        assert fwd(_norm(T, **kw)) == st, kw
        assert lib.moe_rmsnorm_backward_workspace_size(ctypes.byref(_norm(T, **kw)),
                                                       ctypes.byref(n)) == st
    for kw, st in [(dict(x=None), 1), (dict(y=None), 1), (dict(r=P), 1), (dict(s=P), 1),
                   (dict(q=P), 1), (dict(sc=P), 1), (dict(y=None, q=P), 1), (dict(x=P + 1), 3),
                   (dict(w=P + 4), 3), (dict(rstd=P + 8), 3), (dict(q=P, sc=P + 4), 3)]:
        assert fwd(_norm(T), **kw) == st, kw
    assert fwd(_norm(T, dtype=0), x=P + 2) == 3
    assert fwd(_norm(T, n=0), x=None, y=None) == 0
    d = _norm(T)
    assert lib.moe_rmsnorm_backward_workspace_size(ctypes.byref(d), None) == 1
    assert lib.moe_rmsnorm_backward_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
    assert n.value >= 64 * 4
    back = lambda ws, size, dw=P, dy=P: lib.moe_rmsnorm_backward(
        ctypes.byref(d), dy, P, P, P, None, P, dw, ws, size, None)
    assert back(P, n.value - 1) == 4 and back(None, n.value) == 1 and back(P + 4, n.value) == 3
    assert back(P, n.value, dy=None) == 1 and back(P, n.value, dw=P + 4) == 3


def _disp(mod, **kw):
    return mod.MoeDispatchDesc(**{**dict(T=5, d=64, n_experts=4, top_k=2, dtype=1), **kw})


BAD_DISP = [(dict(T=-1), 1), (dict(d=0), 1), (dict(d=1 << 29), 2), (dict(n_experts=0), 1),
            (dict(n_experts=513), 2), (dict(top_k=0), 1), (dict(top_k=65), 2),
            (dict(T=1 << 30, top_k=2), 2), (dict(dtype=3), 2), (dict(rows=11), 1), (dict(rows=-1), 1),
            (dict(ld_t=63), 1), (dict(ld_p=1 << 31), 1)]


def test_dispatch_refusals(T):
    lib = T.lib()

    def run(desc, **kw):
        a = {**dict(idx=P, x=P, xs=None, off=P, perm=P, inv=P, xp=P, xps=None, ws=P, n=1 << 40), **kw}
        return lib.moe_token_dispatch(None if desc is None else ctypes.byref(desc), a["idx"], a["x"],
                                      a["xs"], a["off"], a["perm"], a["inv"], a["xp"], a["xps"],
                                      a["ws"], a["n"], None)

    n = ctypes.c_size_t()
    size = lib.moe_token_dispatch_workspace_size
    assert run(None) == 1 and size(None, ctypes.byref(n)) == 1
    for kw, st in BAD_DISP:
        assert run(_disp(T, **kw)) == st, kw
        assert size(ctypes.byref(_disp(T, **kw)), ctypes.byref(n)) == st
    d = _disp(T)
    for kw, st in [(dict(idx=None), 1), (dict(off=None), 1), (dict(perm=None), 1),
                   (dict(inv=None), 1), (dict(xp=None), 1), (dict(x=None), 1), (dict(xs=P), 1),
                   (dict(xps=P), 1), (dict(idx=P + 2), 3), (dict(off=P + 1), 3), (dict(x=P + 1), 3),
                   (dict(xp=P + 1), 3), (dict(x=None, xp=None, xs=P, xps=P), 1)]:
        assert run(d, **kw) == st, kw
    f8 = _disp(T, dtype=2)
    assert run(f8) == run(f8, xs=P) == run(f8, xps=P) == 1
    assert run(f8, xs=P + 2, xps=P) == 3
    assert size(ctypes.byref(d), None) == 1
    assert size(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value == 0
    many = _disp(T, T=1 << 14)
    assert size(ctypes.byref(many), ctypes.byref(n)) == 0 and n.value > 0
    assert run(many, n=n.value - 1) == 4 and run(many, ws=None, n=n.value) == 1
    assert run(many, ws=P + 8) == 3


def test_combine_refusals(T):
    lib = T.lib()

    def fwd(desc, **kw):
        a = {**dict(yp=P, inv=P, w=P, b=P, y=P), **kw}
        return lib.moe_token_combine(None if desc is None else ctypes.byref(desc), a["yp"],
                                     a["inv"], a["w"], a["b"], a["y"], None)

    def bwd(desc, **kw):
        a = {**dict(dy=P, yp=P, inv=P, w=P, dyp=P, dw=P), **kw}
        return lib.moe_token_combine_backward(None if desc is None else ctypes.byref(desc), a["dy"],
                                              a["yp"], a["inv"], a["w"], a["dyp"], a["dw"], None)

    for f in (fwd, bwd):
        assert f(None) == 1
        for kw, st in BAD_DISP + [(dict(dtype=2), 2)]:
            assert f(_disp(T, **kw)) == st, kw
        assert f(_disp(T, T=0), inv=None, yp=None) == 0
    d = _disp(T)
    for kw, st in [(dict(yp=None), 1), (dict(inv=None), 1), (dict(y=None), 1), (dict(yp=P + 1), 3),
                   (dict(inv=P + 2), 3), (dict(w=P + 1), 3), (dict(b=P + 1), 3), (dict(y=P + 1), 3)]:
        assert fwd(d, **kw) == st, kw
    for kw, st in [(dict(dy=None), 1), (dict(yp=None), 1), (dict(inv=None), 1),
                   (dict(dyp=None, dw=None), 1), (dict(dy=P + 1), 3), (dict(dw=P + 2), 3),
                   (dict(dyp=P + 1), 3)]:
        assert bwd(d, **kw) == st, kw


def test_mx4_refusals(T):
    lib = T.lib()
    mk = lambda **kw: T.MoeMx4Desc(**{**dict(n_mats=1, rows=8, k=64, dtype=1, n_src=8), **kw})
    q = lambda d, src=P, perm=None, c=P, s=P: lib.moe_mx4_quantize(
        None if d is None else ctypes.byref(d), src, perm, c, s, None)
    dq = lambda d, c=P, s=P, out=P: lib.moe_mx4_dequantize(
        None if d is None else ctypes.byref(d), c, s, out, None)
    for f in (q, dq):
        assert f(None) == 1
        for kw, st in [(dict(n_mats=-1), 1), (dict(rows=-1), 1), (dict(k=0), 1),
                       (dict(k=(1 << 20) + 1), 2), (dict(n_mats=1 << 20, rows=1 << 11), 2),
                       (dict(rows=1 << 31), 2), (dict(n_mats=1 << 40, rows=0), 2),
                       (dict(dtype=2), 2), (dict(act=2), 1), (dict(ld=63), 1), (dict(ld=1 << 31), 1)]:
            assert f(mk(**kw)) == st, kw
        assert f(mk(rows=0)) == 0 and f(mk(n_mats=0)) == 0
    assert q(mk(n_src=-1)) == 1 and q(mk(act=1, ld=127)) == 1 and dq(mk(act=1)) == 1
    assert q(mk(n_mats=2), perm=P) == 1
    assert q(mk(), src=None) == q(mk(), c=None) == q(mk(), s=None) == 1
    assert q(mk(), src=P + 1) == q(mk(), c=P + 4) == q(mk(), s=P + 4) == q(mk(), perm=P + 2) == 3
    assert dq(mk(), c=None) == dq(mk(), s=None) == dq(mk(), out=None) == 1
    assert dq(mk(), out=P + 1) == dq(mk(), c=P + 8) == 3
    g = lambda **kw: T.MoeMx4GemmDesc(**{**dict(rows=16, n_groups=4, n=32, k=64, out_dtype=1), **kw})
    run = lambda d, *a: lib.moe_mx4_gemm(None if d is None else ctypes.byref(d),
                                         *(a or [P] * 6), None)
    assert run(None) == 1
    for kw, st in [(dict(rows=-1), 1), (dict(rows=1 << 28), 2), (dict(rows=1 << 24, k=1 << 13), 2),
                   (dict(n_groups=0), 1), (dict(n_groups=513), 2), (dict(n=0), 1), (dict(k=0), 1),
                   (dict(n=(1 << 20) + 1), 2), (dict(k=(1 << 20) + 1), 2),
                   (dict(n=1 << 20, k=1 << 12), 2), (dict(rows=1 << 27, k=1, n=1 << 17), 2),
                   (dict(out_dtype=2), 2), (dict(ld_y=31), 1), (dict(ld_y=1 << 31), 1)]:
        assert run(g(**kw)) == st, kw
    for i in range(6):
        args = [P] * 6
        args[i] = None
        assert run(g(), *args) == 1
        args[i] = P + 1
        assert run(g(), *args) == 3
    assert run(g(rows=0), *[None] * 6) == 0


def test_objects_check_shapes_and_types():
    import sparse_mixture_experts_gate_amd as M
    bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    z = lambda *s, dt=f32: torch.zeros(*s, dtype=dt)
    norm, disp, back = M.RMSNorm(z(8)), M.TokenDispatch(4), M.TokenDispatch
    idx, inv = z(3, 2, dt=i32), z(3, 2, dt=i32)
    lin = M.MX4Linear(z(2, 4, 32, dt=u8), z(2, 1, 4, 4, dt=u8), 40)
    off = z(3, dt=i32)
    bad = [
        lambda: norm.forward(z(2, 9)), lambda: norm.forward(z(8)),
        lambda: norm.forward(z(2, 8, dt=torch.float16)), lambda: norm.forward(z(2, 8), z(3, 8)),
        lambda: norm.forward(z(2, 8), rows=False), lambda: norm.forward(z(8, 2).t()),
        lambda: norm.backward(z(2, 8, dt=bf), z(2, 8), z(2)),
        lambda: norm.backward(z(2, 8), z(2, 8), z(3)),
        lambda: norm.backward(z(2, 8), z(2, 8), z(2), z(2, 7)),
        lambda: disp.forward(z(3, 8), z(3, 2)), lambda: disp.forward(z(4, 8), idx),
        lambda: disp.forward(z(3, 8, dt=torch.float16), idx), lambda: disp.forward(z(3, 8), idx[0]),
        lambda: disp.forward(z(3, 8), idx, z(3, 1)), lambda: disp.forward(z(3, 8, dt=u8), idx),
        lambda: disp.forward(z(3, 8, dt=u8), idx, z(3, 2)),
        lambda: disp.forward(z(3, 8), idx, into=z(5, 8)),
        lambda: disp.forward(z(3, 8), idx, scale_into=z(6, 1)),
        lambda: disp.forward(None, idx, into=z(6, 8)),
        lambda: M.TokenDispatch(4, rows=0).forward(z(3, 8), idx),
        lambda: back.combine(z(7, 8), inv), lambda: back.combine(z(6, 8, dt=u8), inv),
        lambda: back.combine(z(6, 8), inv, z(3, 3)), lambda: back.combine(z(6, 8), inv, None, z(3, 7)),
        lambda: back.combine(z(6, 8), inv, None, z(3, 8, dt=bf)), lambda: back.combine(z(6, 8), inv[0]),
        lambda: back.combine(z(0, 8), inv), lambda: back.combine(z(6, 8), inv.long()),
        lambda: back.combine_grad(z(3, 8), z(6, 7), inv), lambda: back.combine_grad(z(2, 8), z(6, 8), inv),
        lambda: back.combine_grad(z(3, 8), z(6, 8), inv, None, z(5, 8)),
        lambda: M.mx4_quantize(z(8)), lambda: M.mx4_quantize(z(8, 64, dt=torch.float16)),
        lambda: M.mx4_quantize(z(8, 63), act="swiglu"), lambda: M.mx4_quantize(z(8, 64), act="gelu"),
        lambda: M.mx4_quantize(z(2, 8, 64), z(8, dt=i32)), lambda: M.mx4_quantize(z(8, 64), z(8)),
        lambda: M.mx4_quantize(z(8, 2, 64).transpose(0, 1)),
        lambda: M.mx4_dequantize(z(4, 32, dt=u8), z(1, 4, 4, dt=u8), 65),
        lambda: M.mx4_dequantize(z(4, 32, dt=u8), z(4, 4, dt=u8), 64),
        lambda: M.mx4_dequantize(z(4, 32, dt=u8), z(1, 4, 4, dt=u8), 64, torch.float16),
        lambda: M.MX4Linear(z(2, 4, 32, dt=u8), z(2, 1, 4, 4, dt=u8), 65),
        lambda: M.MX4Linear(z(2, 4, 32), z(2, 1, 4, 4, dt=u8), 64),
        lambda: M.MX4Linear(z(260, dt=u8)[4:].reshape(2, 4, 32), z(2, 1, 4, 4, dt=u8), 64),
        lambda: M.MX4Linear.from_blocks(z(2, 4, 32, dt=u8), z(2, 4, 3, dt=u8)),
        lambda: M.MX4Linear.from_weight(z(4, 64)),
        lambda: lin.forward(z(5, 39), off), lambda: lin.forward(z(5, 40), off.long()),
        lambda: lin.forward(z(5, 40), z(4, dt=i32)), lambda: lin.forward(z(5, 40), off, act="swiglu"),
        lambda: lin.forward(z(5, 40), off, out_dtype=torch.float16),
        lambda: lin.forward(z(1, 5, 40), off),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_tensors_of_the_host_are_refused():
    """Every tensor that a kernel would read, by itself on the host."""
    import sparse_mixture_experts_gate_amd as M

    class OnGpu(torch.Tensor):
        """A host tensor that says it is on the current GPU."""
        get_device = lambda self: 0

    gpu = lambda t: t.as_subclass(OnGpu)
    i32, u8, z = torch.int32, torch.uint8, torch.zeros
    idx = z(3, 2, dtype=i32)
    D, k = M.TokenDispatch, 40
    calls = {
        "norm": (lambda w, x, r: M.RMSNorm(w).forward(x, r), [z(8), z(2, 8), z(2, 8)]),
        "norm backward": (lambda w, dy, x, s, r: M.RMSNorm(w).backward(dy, x, s, r),
                          [z(8), z(2, 8), z(2, 8), z(2), z(2, 8)]),
        "dispatch": (lambda x, i, s, a, b: D(4).forward(x, i, s, a, b),
                     [z(3, 8, dtype=u8), idx, z(3, 1), z(6, 8, dtype=u8), z(6, 1)]),
        "combine": (D.combine, [z(6, 8), idx, z(3, 2), z(3, 8)]),
        "combine gradient": (D.combine_grad, [z(3, 8), z(6, 8), idx, z(3, 2), z(6, 8)]),
        "quantize": (M.mx4_quantize, [z(4, 8), z(3, dtype=i32)]),
        "dequantize": (lambda c, s: M.mx4_dequantize(c, s, k),
                       [z(4, 32, dtype=u8), z(1, 4, 4, dtype=u8)]),
        "product": (lambda c, s, x, o, p: M.MX4Linear(c, s, k).forward(x, o, perm=p),
                    [z(2, 4, 32, dtype=u8), z(2, 1, 4, 4, dtype=u8), z(5, k), z(3, dtype=i32),
                     z(5, dtype=i32)]),
    }
    for name, (call, args) in calls.items():
        for i in range(len(args)):
            with pytest.raises(ValueError, match="GPU"):
                call(*(t if j == i else gpu(t) for j, t in enumerate(args)))
