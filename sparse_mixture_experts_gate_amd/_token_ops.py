"""ctypes binding of include/dsmoe_tokens.h: one Python function per C entry
point, with the same name (argument marshalling only, as in ``_ops``)."""
from __future__ import annotations

import ctypes
import os
import re

from . import _lib as L
from ._ops import _nbytes, _p, _rows, _stream

HEADER = os.path.join(os.path.dirname(L.PKG), "include", "dsmoe_tokens.h")

MOE_MX4_PLAIN, MOE_MX4_SWIGLU = 0, 1


class MoeRmsNormDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("ld_x", ctypes.c_int64), ("ld_r", ctypes.c_int64),
                ("ld_y", ctypes.c_int64), ("ld_s", ctypes.c_int64), ("ld_q", ctypes.c_int64)]


class MoeDispatchDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("dtype", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("ld_t", ctypes.c_int64), ("ld_p", ctypes.c_int64)]


class MoeMx4Desc(ctypes.Structure):
    _fields_ = [("n_mats", ctypes.c_int64), ("rows", ctypes.c_int64), ("k", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("ld", ctypes.c_int64),
                ("n_src", ctypes.c_int64)]


class MoeMx4GemmDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("n_groups", ctypes.c_int32), ("n", ctypes.c_int32),
                ("k", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("ld_y", ctypes.c_int64)]


def header_symbols() -> list[str]:
    """Names of the functions that include/dsmoe_tokens.h declares."""
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"^moe_status\s+(\w+)\s*\(", txt, re.M)))


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        l = L.lib()
        P, Z = ctypes.c_void_p, ctypes.c_size_t
        S = ctypes.POINTER(Z)
        N, D, X, G = (ctypes.POINTER(t) for t in (MoeRmsNormDesc, MoeDispatchDesc, MoeMx4Desc,
                                                  MoeMx4GemmDesc))
        sig = {
            "moe_rmsnorm_forward": [N, P, P, P, P, P, P, P, P, P],
            "moe_rmsnorm_backward_workspace_size": [N, S],
            "moe_rmsnorm_backward": [N, P, P, P, P, P, P, P, P, Z, P],
            "moe_token_dispatch_workspace_size": [D, S],
            "moe_token_dispatch": [D, P, P, P, P, P, P, P, P, P, Z, P],
            "moe_token_combine": [D, P, P, P, P, P, P],
            "moe_token_combine_backward": [D, P, P, P, P, P, P, P],
            "moe_mx4_quantize": [X, P, P, P, P, P],
            "moe_mx4_dequantize": [X, P, P, P, P],
            "moe_mx4_gemm": [G, P, P, P, P, P, P, P],
        }
        for name, args in sig.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        _lib = l
    return _lib


def call(name: str, desc, *args) -> None:
    """The entry point `name` with addresses and plain values, for callers that
    have checked their tensors."""
    status = getattr(_lib or lib(), name)(ctypes.byref(desc), *args)
    if status:
        L._check(status, name)


def _size(name: str, desc) -> int:
    n = ctypes.c_size_t(0)
    call(name, desc, ctypes.byref(n))
    return n.value


def moe_rmsnorm_forward(desc, x, residual, weight, y, codes, scale, sum, rstd, stream=None):
    L._check(lib().moe_rmsnorm_forward(ctypes.byref(desc), _rows(x), _rows(residual), _p(weight),
                                       _rows(y), _rows(codes), _p(scale), _rows(sum), _p(rstd),
                                       _stream(stream)), "moe_rmsnorm_forward")


def moe_rmsnorm_backward_workspace_size(desc) -> int:
    return _size("moe_rmsnorm_backward_workspace_size", desc)


def moe_rmsnorm_backward(desc, dy, x, weight, rstd, dresidual, dx, dweight, ws, stream=None):
    L._check(lib().moe_rmsnorm_backward(ctypes.byref(desc), _rows(dy), _rows(x), _p(weight),
                                        _p(rstd), _rows(dresidual), _rows(dx), _p(dweight), _p(ws),
                                        _nbytes(ws), _stream(stream)), "moe_rmsnorm_backward")


def moe_token_dispatch_workspace_size(desc) -> int:
    return _size("moe_token_dispatch_workspace_size", desc)


def moe_token_dispatch(desc, topk_idx, x, x_scale, offsets, perm, inv, x_perm, x_perm_scale,
                       ws=None, stream=None):
    L._check(lib().moe_token_dispatch(ctypes.byref(desc), _p(topk_idx), _rows(x), _p(x_scale),
                                      _p(offsets), _p(perm), _p(inv), _rows(x_perm),
                                      _p(x_perm_scale), _p(ws), _nbytes(ws), _stream(stream)),
             "moe_token_dispatch")


def moe_token_combine(desc, y_perm, inv, weight, base, y, stream=None):
    L._check(lib().moe_token_combine(ctypes.byref(desc), _rows(y_perm), _p(inv), _p(weight),
                                     _rows(base), _rows(y), _stream(stream)), "moe_token_combine")


def moe_token_combine_backward(desc, dy, y_perm, inv, weight, dy_perm, dweight, stream=None):
    L._check(lib().moe_token_combine_backward(ctypes.byref(desc), _rows(dy), _rows(y_perm),
                                              _p(inv), _p(weight), _rows(dy_perm), _p(dweight),
                                              _stream(stream)), "moe_token_combine_backward")


def moe_mx4_quantize(desc, src, perm, codes, scales, stream=None):
    L._check(lib().moe_mx4_quantize(ctypes.byref(desc), _rows(src), _p(perm), _p(codes),
                                    _p(scales), _stream(stream)), "moe_mx4_quantize")


def moe_mx4_dequantize(desc, codes, scales, dst, stream=None):
    L._check(lib().moe_mx4_dequantize(ctypes.byref(desc), _p(codes), _p(scales), _rows(dst),
                                      _stream(stream)), "moe_mx4_dequantize")


def moe_mx4_gemm(desc, x_codes, x_scales, w_codes, w_scales, offsets, y, stream=None):
    L._check(lib().moe_mx4_gemm(ctypes.byref(desc), _p(x_codes), _p(x_scales), _p(w_codes),
                                _p(w_scales), _p(offsets), _rows(y), _stream(stream)),
             "moe_mx4_gemm")
