"""ctypes binding of include/dsmoe_ops.h: one Python function per C entry
point, with the same name (argument marshalling only, as in ``_lib``)."""
from __future__ import annotations

import ctypes
import os
import re

import torch

from . import _lib as L

HEADER = os.path.join(os.path.dirname(L.PKG), "include", "dsmoe_ops.h")


class MoeNormDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("ld_x", ctypes.c_int64), ("ld_r", ctypes.c_int64),
                ("ld_y", ctypes.c_int64), ("ld_s", ctypes.c_int64)]


class MoeGroupedDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("n_groups", ctypes.c_int32), ("n", ctypes.c_int32),
                ("k", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("ld_k", ctypes.c_int64),
                ("ld_n", ctypes.c_int64), ("accumulate", ctypes.c_int32)]


class MoeOrthDesc(ctypes.Structure):
    _fields_ = [("n_mats", ctypes.c_int64), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("steps", ctypes.c_int32),
                ("momentum", ctypes.c_float), ("nesterov", ctypes.c_int32)]


def header_symbols() -> list[str]:
    """Names of the functions that include/dsmoe_ops.h declares."""
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"^moe_status\s+(\w+)\s*\(", txt, re.M)))


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        l = L.lib()
        P, Z = ctypes.c_void_p, ctypes.c_size_t
        N, G, O = (ctypes.POINTER(t) for t in (MoeNormDesc, MoeGroupedDesc, MoeOrthDesc))
        sig = {
            "moe_layernorm_forward": [N, P, P, P, P, P, P, P, P, P],
            "moe_layernorm_backward_workspace_size": [N, ctypes.POINTER(Z)],
            "moe_layernorm_backward": [N, P, P, P, P, P, P, P, P, P, P, Z, P],
            "moe_grouped_gemm_workspace_size": [G, ctypes.c_int32, ctypes.POINTER(Z)],
            "moe_grouped_gemm": [G, P, P, P, P, P, Z, P],
            "moe_grouped_gemm_dgrad": [G, P, P, P, P, P, Z, P],
            "moe_grouped_gemm_wgrad": [G, P, P, P, P, P, Z, P],
            "moe_orthogonalize_workspace_size": [O, ctypes.POINTER(Z)],
            "moe_orthogonalize": [O, P, P, P, P, P, Z, P],
        }
        for name, args in sig.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        _lib = l
    return _lib


def _p(t) -> int | None:
    """Device pointer of a contiguous tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _rows(t) -> int | None:
    """Device pointer of a row matrix. Its rows may be strided, as the
    descriptor says, and counted by several leading dimensions."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if not t.is_contiguous() and not _one_row_stride(t.shape, t.stride()):
        raise ValueError("row matrices passed to the library must have contiguous columns and "
                         "one row stride")
    return t.data_ptr()


def _one_row_stride(shape, stride) -> bool:
    return (len(shape) > 1 and 1 in (shape[-1], stride[-1]) and
            all(shape[i] == 1 or stride[i] == stride[i + 1] * shape[i + 1]
                for i in range(len(shape) - 2)))


def _stream(stream) -> int:
    """Handle of a torch stream, or of the current one."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def moe_layernorm_forward(desc, x, residual, weight, bias, y, sum, mean, rstd, stream=None):
    L._check(lib().moe_layernorm_forward(ctypes.byref(desc), _rows(x), _rows(residual),
                                         _p(weight), _p(bias), _rows(y), _rows(sum), _p(mean),
                                         _p(rstd), _stream(stream)), "moe_layernorm_forward")


def moe_layernorm_backward_workspace_size(desc) -> int:
    n = ctypes.c_size_t(0)
    L._check(lib().moe_layernorm_backward_workspace_size(ctypes.byref(desc), ctypes.byref(n)),
             "moe_layernorm_backward_workspace_size")
    return n.value


def moe_layernorm_backward(desc, dy, x, weight, mean, rstd, dresidual, dx, dweight, dbias, ws,
                           stream=None):
    L._check(lib().moe_layernorm_backward(ctypes.byref(desc), _rows(dy), _rows(x), _p(weight),
                                          _p(mean), _p(rstd), _rows(dresidual), _rows(dx),
                                          _p(dweight), _p(dbias), _p(ws), _nbytes(ws),
                                          _stream(stream)),
             "moe_layernorm_backward")


MOE_GROUPED_FORWARD, MOE_GROUPED_DGRAD, MOE_GROUPED_WGRAD = 0, 1, 2


def moe_grouped_gemm_workspace_size(desc, op) -> int:
    n = ctypes.c_size_t(0)
    L._check(lib().moe_grouped_gemm_workspace_size(ctypes.byref(desc), op, ctypes.byref(n)),
             "moe_grouped_gemm_workspace_size")
    return n.value


def moe_grouped_gemm(desc, x, w, offsets, y, ws=None, stream=None):
    L._check(lib().moe_grouped_gemm(ctypes.byref(desc), _rows(x), _p(w), _p(offsets), _rows(y),
                                    _p(ws), _nbytes(ws), _stream(stream)), "moe_grouped_gemm")


def moe_grouped_gemm_dgrad(desc, dy, w, offsets, dx, ws=None, stream=None):
    L._check(lib().moe_grouped_gemm_dgrad(ctypes.byref(desc), _rows(dy), _p(w), _p(offsets),
                                          _rows(dx), _p(ws), _nbytes(ws), _stream(stream)),
             "moe_grouped_gemm_dgrad")


def moe_grouped_gemm_wgrad(desc, dy, x, offsets, dw, ws=None, stream=None):
    L._check(lib().moe_grouped_gemm_wgrad(ctypes.byref(desc), _rows(dy), _rows(x), _p(offsets),
                                          _p(dw), _p(ws), _nbytes(ws), _stream(stream)),
             "moe_grouped_gemm_wgrad")


def moe_orthogonalize_workspace_size(desc) -> int:
    n = ctypes.c_size_t(0)
    L._check(lib().moe_orthogonalize_workspace_size(ctypes.byref(desc), ctypes.byref(n)),
             "moe_orthogonalize_workspace_size")
    return n.value


def moe_orthogonalize(desc, grad, m_in, m_out, out, ws, stream=None):
    L._check(lib().moe_orthogonalize(ctypes.byref(desc), _p(grad), _p(m_in), _p(m_out), _p(out),
                                     _p(ws), _nbytes(ws), _stream(stream)), "moe_orthogonalize")
