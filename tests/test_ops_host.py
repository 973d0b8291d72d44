"""Host-only checks of the operators' C entry points: exported symbols and
refusals, each before anything reaches a GPU."""
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
def O():
    from sparse_mixture_experts_gate_amd import _ops
    return _ops


def test_every_declared_symbol_is_exported_and_bound(O):
    names = O.header_symbols()
    assert set(names) == {
        "moe_layernorm_forward", "moe_layernorm_backward_workspace_size", "moe_layernorm_backward",
        "moe_grouped_gemm", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad",
        "moe_grouped_gemm_workspace_size", "moe_orthogonalize_workspace_size", "moe_orthogonalize"}
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    import sparse_mixture_experts_gate_amd as M
    for n in names:
        assert n in exported and callable(getattr(M, n))


def _norm(O, **kw):
    return O.MoeNormDesc(**{**dict(n=4, d=64, dtype=1, eps=1e-5), **kw})


def _fwd(O, desc, **kw):
    a = {**dict(x=P, r=None, w=P, b=P, y=P, s=None, mean=P, rstd=P), **kw}
    return O.lib().moe_layernorm_forward(None if desc is None else ctypes.byref(desc), a["x"],
                                         a["r"], a["w"], a["b"], a["y"], a["s"], a["mean"],
                                         a["rstd"], None)


def test_norm_refusals(O):
    assert _fwd(O, None) == 1
    for kw, st in [(dict(n=-1), 1), (dict(n=1 << 31), 2), (dict(d=0), 1), (dict(d=(1 << 20) + 1), 2),
                   (dict(dtype=2), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
                   (dict(eps=float("inf")), 1), (dict(ld_x=63), 1), (dict(ld_r=-1), 1),
                   (dict(ld_y=1 << 31), 1), (dict(ld_s=1), 1)]:
        assert _fwd(O, _norm(O, **kw)) == st, kw
        n = ctypes.c_size_t()
        assert O.lib().moe_layernorm_backward_workspace_size(
            ctypes.byref(_norm(O, **kw)), ctypes.byref(n)) == st
    for kw, st in [(dict(x=None), 1), (dict(y=None), 1), (dict(r=P), 1), (dict(s=P), 1),
                   (dict(mean=None), 1), (dict(rstd=None), 1), (dict(x=P + 1), 3),
                   (dict(w=P + 4), 3), (dict(mean=P + 8), 3)]:
        assert _fwd(O, _norm(O), **kw) == st, kw
    assert _fwd(O, _norm(O, dtype=0), x=P + 2) == 3
    assert _fwd(O, _norm(O, n=0), x=None, y=None) == 0
    lib, d = O.lib(), _norm(O)
    n = ctypes.c_size_t()
    assert lib.moe_layernorm_backward_workspace_size(ctypes.byref(d), None) == 1
    assert lib.moe_layernorm_backward_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
    assert n.value >= 2 * 64 * 4
    back = lambda ws, size, dw=P, dy=P: lib.moe_layernorm_backward(
        ctypes.byref(d), dy, P, P, P, P, None, P, dw, P, ws, size, None)
    assert back(P, n.value - 1) == 4 and back(None, n.value) == 1 and back(P + 4, n.value) == 3
    assert back(P, n.value, dy=None) == 1 and back(P, n.value, dw=P + 4) == 3


def _grouped(O, **kw):
    return O.MoeGroupedDesc(**{**dict(rows=16, n_groups=4, n=32, k=64, out_dtype=1), **kw})


def test_grouped_refusals(O):
    lib = O.lib()
    fns = [lib.moe_grouped_gemm, lib.moe_grouped_gemm_dgrad, lib.moe_grouped_gemm_wgrad]
    for f in fns:
        assert f(None, P, P, P, P, P, 1 << 40, None) == 1
        for kw, st in [(dict(rows=-1), 1), (dict(rows=(1 << 31) - 1), 2), (dict(n_groups=0), 1),
                       (dict(n_groups=513), 2), (dict(n=0), 1), (dict(k=0), 1),
                       (dict(n=1 << 15, k=1 << 14), 2), (dict(ld_k=63), 1), (dict(ld_n=31), 1),
                       (dict(ld_k=1 << 21), 2), (dict(ld_n=1 << 21), 2)]:
            assert f(ctypes.byref(_grouped(O, **kw)), P, P, P, P, P, 1 << 40, None) == st, kw
        d = _grouped(O)
        for i in range(4):
            args = [P] * 4
            args[i] = None
            assert f(ctypes.byref(d), *args, P, 1 << 40, None) == 1
            args[i] = P + 1
            assert f(ctypes.byref(d), *args, P, 1 << 40, None) == 3
    for f in fns[:2]:
        assert f(ctypes.byref(_grouped(O, out_dtype=2)), P, P, P, P, P, 1 << 40, None) == 2
        assert f(ctypes.byref(_grouped(O, out_dtype=0)), P, P, P, P + 2, P, 1 << 40, None) == 3
        assert f(ctypes.byref(_grouped(O, rows=0)), None, None, None, None, None, 0, None) == 0
    assert b"" != lib.moe_last_error()
    # few outputs of a long contraction: partial sums need a workspace
    d, n = _grouped(O, rows=4, n_groups=1, n=64, k=8192), ctypes.c_size_t()
    size = lib.moe_grouped_gemm_workspace_size
    assert size(ctypes.byref(d), 0, ctypes.byref(n)) == 0 and n.value > 0
    assert size(ctypes.byref(d), 3, ctypes.byref(n)) == size(ctypes.byref(d), -1, ctypes.byref(n)) == 1
    assert size(None, 0, ctypes.byref(n)) == size(ctypes.byref(d), 0, None) == 1
    run = lambda ws, b: lib.moe_grouped_gemm(ctypes.byref(d), P, P, P, P, ws, b, None)
    assert run(P, n.value - 1) == 4 and run(None, n.value) == 1 and run(P + 4, n.value) == 3


def test_orthogonalize_refusals(O):
    lib = O.lib()
    mk = lambda **kw: O.MoeOrthDesc(**{**dict(n_mats=2, rows=32, cols=640, grad_dtype=0, steps=5,
                                              momentum=0.95, nesterov=1), **kw})
    n = ctypes.c_size_t()
    assert lib.moe_orthogonalize_workspace_size(None, ctypes.byref(n)) == 1
    for kw, st in [(dict(n_mats=-1), 1), (dict(n_mats=65536), 2), (dict(rows=0), 1),
                   (dict(cols=0), 1), (dict(rows=16385), 2), (dict(grad_dtype=2), 2),
                   (dict(steps=0), 1), (dict(steps=17), 1), (dict(momentum=1.0), 1),
                   (dict(momentum=-0.1), 1), (dict(momentum=float("nan")), 1),
                   (dict(nesterov=2), 1)]:
        assert lib.moe_orthogonalize_workspace_size(ctypes.byref(mk(**kw)), ctypes.byref(n)) == st, kw
    d = mk()
    assert lib.moe_orthogonalize_workspace_size(ctypes.byref(d), None) == 1
    assert lib.moe_orthogonalize_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
    run = lambda g=P, mi=None, mo=None, out=P, ws=P, size=n.value: lib.moe_orthogonalize(
        ctypes.byref(d), g, mi, mo, out, ws, size, None)
    assert run(size=n.value - 1) == 4
    assert run(g=None) == run(out=None) == run(ws=None) == run(mi=P) == run(mo=P) == 1
    assert run(g=P + 4) == run(ws=P + 8) == 3
    # small matrices are worked on in LDS
    small = ctypes.c_size_t(1)
    assert lib.moe_orthogonalize_workspace_size(ctypes.byref(mk(cols=64)), ctypes.byref(small)) == 0
    assert small.value == 0 and n.value > 0
    assert lib.moe_orthogonalize(ctypes.byref(mk(n_mats=0)), None, None, None, None, None, 0,
                                 None) == 0


def test_wrappers_check_shapes_and_types():
    import sparse_mixture_experts_gate_amd as M
    bf, f32 = torch.bfloat16, torch.float32
    z = lambda *s, dt=f32: torch.zeros(*s, dtype=dt)
    norm = M.LayerNorm(z(8), z(8))
    for bad in (lambda: norm.forward(z(2, 9)), lambda: norm.forward(z(8)),
                lambda: norm.forward(z(2, 8, dt=torch.float16)),
                lambda: norm.forward(z(2, 8), z(3, 8)), lambda: norm.forward(z(2, 8), z(2, 8, dt=bf)),
                lambda: norm.forward(z(8, 2).t()), lambda: norm.forward(z(1, 8).expand(2, 8)),
                lambda: norm.backward(z(2, 8, dt=bf), z(2, 8), z(2), z(2)),
                lambda: norm.backward(z(2, 8), z(2, 8), z(3), z(2))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError):
        M.GroupedLinear(z(2, 4, 8))
    lin = M.GroupedLinear(z(2, 4, 8, dt=bf))
    off = z(3, dt=torch.int32)
    for bad in (lambda: lin.forward(z(5, 8), off), lambda: lin.forward(z(5, 7, dt=bf), off),
                lambda: lin.forward(z(5, 8, dt=bf), z(4, dt=torch.int32)),
                lambda: lin.forward(z(5, 8, dt=bf), z(3, dt=torch.int64)),
                lambda: lin.forward(z(5, 8, dt=bf), off, out_dtype=torch.float16),
                lambda: lin.input_grad(z(5, 8, dt=bf), off),
                lambda: lin.weight_grad(z(5, 4, dt=bf), z(6, 8, dt=bf), off),
                lambda: lin.weight_grad(z(5, 4, dt=bf), z(5, 8, dt=bf), off, into=z(2, 4, 9))):
        with pytest.raises(ValueError):
            bad()
    muon = M.Muon()
    for bad in (lambda: muon.direction(z(8)), lambda: muon.direction(z(4, 8, dt=torch.float16)),
                lambda: muon.direction(z(4, 8).t()), lambda: muon.direction(z(4, 8), z(4, 9)),
                lambda: muon.direction(z(4, 8), z(4, 8, dt=bf)),
                lambda: muon.direction(z(4, 8), None, z(4, 8))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(M.MoeError):
        M.Muon(momentum=1.5).direction(z(4, 8))
