"""Objects over the operators of ``include/dsmoe_ops.h``: layer norm, linear
maps grouped by expert, and the orthogonalized update. They check shapes,
allocate outputs and keep the workspace; all arithmetic is the library's."""
from __future__ import annotations

import contextlib
import threading

import torch

from . import _lib as L
from . import _ops as O

_DT = {torch.float32: L.MOE_DT_F32, torch.bfloat16: L.MOE_DT_BF16}


_CURRENT = contextlib.nullcontext()


def _on(stream):
    """Allocate on the stream that the call runs on."""
    return _CURRENT if stream is None else torch.cuda.stream(stream)


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, n: int, d: int) -> int:
    """Row stride of a row matrix [n, d], checked."""
    if t.dtype is not dtype or t.shape != (n, d):
        raise ValueError(f"{name}: expected {dtype} [{n}, {d}], got {t.dtype} {list(t.shape)}")
    if n <= 1 or t.is_contiguous():
        if d > 1 and n and t.stride(1) != 1:
            raise ValueError(f"{name}: columns must be contiguous")
        return d
    rows, cols = t.stride()
    if d > 1 and cols != 1:
        raise ValueError(f"{name}: columns must be contiguous")
    if rows < d:
        raise ValueError(f"{name}: rows overlap (stride {rows} < {d})")
    return rows


def _vector(t, name: str, dtype: torch.dtype, n: int) -> None:
    if t is not None and (t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous()):
        raise ValueError(f"{name}: expected contiguous {dtype} [{n}], got {t.dtype} "
                         f"{list(t.shape)}")


def _aligned(t):
    """t, or a copy of it where it does not start on 16 bytes as the library
    asks of vectors (a view of a flat parameter buffer, a slice of the rows'
    statistics)."""
    return t if t is None or not t.data_ptr() & 15 else t.clone()


def _on_gpu(stream, first, *others) -> None:
    """Refuse tensors (None: not given) that are not on the GPU the call runs
    on: a kernel that reads a host address or another GPU's faults."""
    at = first.get_device()
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError("expected all tensors on one GPU")
    if at < 0 or at != (torch._C._cuda_getDevice() if stream is None else stream.device_index):
        raise ValueError("expected tensors on the GPU of the call's stream")


class _Workspace:
    """One buffer per stream and host thread, grown as calls need it. Two
    threads that use one stream have a buffer each: a call's kernels meet in
    its workspace, and the other thread's may be enqueued between them. A call
    that is being captured gets a buffer of its own from the graph's memory
    pool, since replays write to that address whatever eager calls do later."""

    def __init__(self):
        self._local = threading.local()

    @property
    def _bufs(self) -> dict:
        """The calling thread's buffers."""
        try:
            return self._local.bufs
        except AttributeError:
            self._local.bufs = {}
            return self._local.bufs

    def get(self, need: int, device, stream) -> torch.Tensor:
        """A buffer of at least `need` bytes; called with `stream` current."""
        if torch.cuda.is_current_stream_capturing():
            return torch.empty(need, dtype=torch.uint8, device=device)
        bufs, key = self._bufs, (device, O._stream(stream))
        buf = bufs.get(key)
        if buf is None or buf.numel() < need:
            buf = bufs[key] = torch.empty(need, dtype=torch.uint8, device=device)
        return buf


class LayerNorm:
    """Layer norm over the last dimension with fp32 weight and bias (either
    may be None), for bf16 or fp32 rows (moe_layernorm_forward)."""

    def __init__(self, weight: torch.Tensor | None, bias: torch.Tensor | None = None,
                 eps: float = 1e-5):
        self.weight, self.bias, self.eps = weight, bias, eps
        self._ws = _Workspace()
        for t, name in ((weight, "weight"), (bias, "bias")):
            if t is not None:
                _vector(t, name, torch.float32, t.numel())
        self.dims = {t.numel() for t in (weight, bias) if t is not None}

    def _desc(self, x: torch.Tensor) -> O.MoeNormDesc:
        if x.dim() != 2 or x.dtype not in _DT:
            raise ValueError(f"x: expected bf16 or fp32 [n, d], got {x.dtype} {list(x.shape)}")
        n, d = x.shape
        for v in self.dims:
            if v != d:
                raise ValueError(f"x: rows of {d} values, weight and bias have {sorted(self.dims)}")
        return O.MoeNormDesc(n, d, _DT[x.dtype], self.eps, _rows(x, "x", x.dtype, n, d))

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None,
                stream=None) -> dict:
        """y = norm(x + residual) with the row statistics, and the sum itself
        when there is a residual: {"y", "mean", "rstd", "sum"}; "sum" is what
        the backward takes as x (x itself without a residual)."""
        desc = self._desc(x)
        n, d = x.shape
        if residual is not None:
            desc.ld_r = _rows(residual, "residual", x.dtype, n, d)
        _on_gpu(stream, x, residual, self.weight, self.bias)
        with _on(stream):
            y = x.new_empty(n, d)
            total = x.new_empty(n, d) if residual is not None else None
            mean = x.new_empty(n, dtype=torch.float32)
            rstd = x.new_empty(n, dtype=torch.float32)
            weight, bias = _aligned(self.weight), _aligned(self.bias)
        O.moe_layernorm_forward(desc, x, residual, weight, bias, y, total, mean, rstd, stream)
        return {"y": y, "mean": mean, "rstd": rstd, "sum": x if residual is None else total}

    def backward(self, dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                 dresidual: torch.Tensor | None = None, stream=None) -> dict:
        """{"dx", "dweight", "dbias"} for the forward's normalized rows x
        (its "sum"); dresidual is added to dx."""
        desc = self._desc(x)
        n, d = x.shape
        desc.ld_y = _rows(dy, "dy", x.dtype, n, d)
        if dresidual is not None:
            desc.ld_r = _rows(dresidual, "dresidual", x.dtype, n, d)
        _vector(mean, "mean", torch.float32, n)
        _vector(rstd, "rstd", torch.float32, n)
        _on_gpu(stream, dy, x, self.weight, mean, rstd, dresidual)
        with _on(stream):
            dx = torch.empty(n, d, dtype=x.dtype, device=x.device)
            dw = torch.empty(d, dtype=torch.float32, device=x.device)
            db = torch.empty_like(dw)
            need = O.moe_layernorm_backward_workspace_size(desc)
            ws = self._ws.get(need, x.device, stream) if need else None
            weight, mean, rstd = _aligned(self.weight), _aligned(mean), _aligned(rstd)
        O.moe_layernorm_backward(desc, dy, x, weight, mean, rstd, dresidual, dx, dw, db, ws, stream)
        return {"dx": dx, "dweight": dw, "dbias": db}


class GroupedLinear:
    """One linear map per expert, weight [groups, n, k] bf16, over rows sorted
    by expert (``moe_permute``'s order) with ``offsets`` [groups + 1] int32 on
    the device: group g owns rows offsets[g] .. offsets[g + 1] - 1. Rows
    outside the groups are not written."""

    def __init__(self, weight: torch.Tensor):
        if weight.dim() != 3 or weight.dtype != torch.bfloat16 or not weight.is_contiguous():
            raise ValueError(f"weight: expected contiguous bf16 [groups, n, k], got "
                             f"{weight.dtype} {list(weight.shape)}")
        self.weight = weight

    # partial sums of few outputs, shared by all maps of a stream and thread
    _ws = _Workspace()

    @staticmethod
    def _workspace(desc, op, device, stream):
        need = O.moe_grouped_gemm_workspace_size(desc, op)
        return GroupedLinear._ws.get(need, device, stream) if need else None

    @staticmethod
    def _desc(rows, groups, n, k, offsets, out_dtype=torch.float32) -> O.MoeGroupedDesc:
        _vector(offsets, "offsets", torch.int32, groups + 1)
        if out_dtype not in _DT:
            raise ValueError(f"out_dtype: bf16 or fp32, got {out_dtype}")
        return O.MoeGroupedDesc(rows=rows, n_groups=groups, n=n, k=k, out_dtype=_DT[out_dtype])

    def forward(self, x: torch.Tensor, offsets: torch.Tensor, out_dtype=torch.bfloat16,
                stream=None) -> torch.Tensor:
        """y [rows, n] = x W_g^T (moe_grouped_gemm)."""
        G, n, k = self.weight.shape
        desc = self._desc(x.shape[0], G, n, k, offsets, out_dtype)
        desc.ld_k = _rows(x, "x", torch.bfloat16, x.shape[0], k)
        _on_gpu(stream, x, self.weight, offsets)
        with _on(stream):
            y = torch.empty(x.shape[0], n, dtype=out_dtype, device=x.device)
            ws = self._workspace(desc, O.MOE_GROUPED_FORWARD, x.device, stream)
        O.moe_grouped_gemm(desc, x, self.weight, offsets, y, ws, stream)
        return y

    def input_grad(self, dy: torch.Tensor, offsets: torch.Tensor, out_dtype=torch.bfloat16,
                   stream=None) -> torch.Tensor:
        """dx [rows, k] = dy W_g (moe_grouped_gemm_dgrad)."""
        G, n, k = self.weight.shape
        desc = self._desc(dy.shape[0], G, n, k, offsets, out_dtype)
        desc.ld_n = _rows(dy, "dy", torch.bfloat16, dy.shape[0], n)
        _on_gpu(stream, dy, self.weight, offsets)
        with _on(stream):
            dx = torch.empty(dy.shape[0], k, dtype=out_dtype, device=dy.device)
            ws = self._workspace(desc, O.MOE_GROUPED_DGRAD, dy.device, stream)
        O.moe_grouped_gemm_dgrad(desc, dy, self.weight, offsets, dx, ws, stream)
        return dx

    @staticmethod
    def weight_grad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                    into: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """dw [groups, n, k] fp32 = dy_g^T x_g (moe_grouped_gemm_wgrad), added
        to ``into`` when given (gradient accumulation)."""
        G = offsets.shape[0] - 1
        rows, n, k = dy.shape[0], dy.shape[1], x.shape[1]
        desc = GroupedLinear._desc(rows, G, n, k, offsets)
        desc.ld_n = _rows(dy, "dy", torch.bfloat16, rows, n)
        desc.ld_k = _rows(x, "x", torch.bfloat16, rows, k)
        desc.accumulate = into is not None
        if into is not None and (into.dtype != torch.float32 or into.shape != (G, n, k)
                                 or not into.is_contiguous()):
            raise ValueError(f"into: expected contiguous fp32 [{G}, {n}, {k}], got {into.dtype} "
                             f"{list(into.shape)}")
        _on_gpu(stream, dy, x, offsets, into)
        with _on(stream):
            if into is None:
                into = torch.empty(G, n, k, dtype=torch.float32, device=dy.device)
            ws = GroupedLinear._workspace(desc, O.MOE_GROUPED_WGRAD, dy.device, stream)
        O.moe_grouped_gemm_wgrad(desc, dy, x, offsets, into, ws, stream)
        return into


class Muon:
    """Momentum and Newton-Schulz orthogonalization of weight updates
    (moe_orthogonalize) for matrices [..., rows, cols], all at once."""

    def __init__(self, momentum: float = 0.95, nesterov: bool = True, steps: int = 5):
        self.momentum, self.nesterov, self.steps = momentum, nesterov, steps
        self._ws = _Workspace()

    def direction(self, grad: torch.Tensor, momentum: torch.Tensor | None = None,
                  out_momentum: torch.Tensor | None = None, stream=None) -> tuple:
        """(out, momentum'): the orthogonalized direction in bf16 and the new
        fp32 momentum, written to ``out_momentum`` (which may be
        ``momentum``). Without momentum: (out, None)."""
        if grad.dim() < 2 or grad.dtype not in _DT or not grad.is_contiguous():
            raise ValueError(f"grad: expected contiguous bf16 or fp32 [..., rows, cols], got "
                             f"{grad.dtype} {list(grad.shape)}")
        rows, cols = grad.shape[-2:]
        for t, name in ((momentum, "momentum"), (out_momentum, "out_momentum")):
            if t is not None and (t.dtype != torch.float32 or t.shape != grad.shape
                                  or not t.is_contiguous()):
                raise ValueError(f"{name}: expected contiguous fp32 {list(grad.shape)}, got "
                                 f"{t.dtype} {list(t.shape)}")
        if momentum is None and out_momentum is not None:
            raise ValueError("out_momentum without momentum")
        desc = O.MoeOrthDesc(n_mats=grad.numel() // (rows * cols) if rows * cols else 0, rows=rows,
                             cols=cols, grad_dtype=_DT[grad.dtype], steps=self.steps,
                             momentum=self.momentum, nesterov=int(self.nesterov))
        need = O.moe_orthogonalize_workspace_size(desc)
        _on_gpu(stream, grad, momentum, out_momentum)
        with _on(stream):
            out = torch.empty(grad.shape, dtype=torch.bfloat16, device=grad.device)
            if momentum is not None and out_momentum is None:
                out_momentum = torch.empty_like(momentum)
            ws = self._ws.get(need, grad.device, stream) if need else None
        O.moe_orthogonalize(desc, grad, momentum, out_momentum, out, ws, stream)
        return out, out_momentum
