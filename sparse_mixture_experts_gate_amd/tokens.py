"""Objects over the operators of ``include/dsmoe_tokens.h``: RMS norm, tokens
sorted by expert and returned, linear maps with 4-bit weights. They check shapes,
allocate outputs and keep the workspace; all arithmetic is the library's."""
from __future__ import annotations

import torch

from . import _lib as L
from . import _token_ops as T
from ._ops import _stream
from .blocks import _DT, _aligned, _on, _on_gpu, _rows, _vector, _Workspace

_ACT = {None: T.MOE_MX4_PLAIN, "swiglu": T.MOE_MX4_SWIGLU}


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _matrix(t, name: str, dtype, *shape) -> None:
    if t is not None and (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{name}: expected contiguous {dtype} {list(shape)}, got {t.dtype} "
                         f"{list(t.shape)}")


class RMSNorm:
    """RMS norm over the last dimension with fp32 weight (or None), for bf16 or
    fp32 rows (moe_rmsnorm_forward)."""

    def __init__(self, weight: torch.Tensor | None, eps: float = 1e-6):
        self.weight, self.eps = weight, eps
        self._ws = _Workspace()
        if weight is not None:
            _vector(weight, "weight", torch.float32, weight.numel())

    def _desc(self, x: torch.Tensor) -> T.MoeRmsNormDesc:
        if x.dim() != 2 or x.dtype not in _DT:
            raise ValueError(f"x: expected bf16 or fp32 [n, d], got {x.dtype} {list(x.shape)}")
        n, d = x.shape
        if self.weight is not None and self.weight.numel() != d:
            raise ValueError(f"x: rows of {d} values, weight has {self.weight.numel()}")
        return T.MoeRmsNormDesc(n, d, _DT[x.dtype], self.eps, _rows(x, "x", x.dtype, n, d))

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None, rows: bool = True,
                codes: bool = False, stream=None) -> dict:
        """o = norm(x + residual): with ``rows`` "y" in x's type; with ``codes``
        "codes" (uint8, E4M3) and "scale" of its 1x128 tiles; "rstd"; and "sum",
        what the backward takes as x (x itself without a residual)."""
        desc = self._desc(x)
        n, d = x.shape
        if residual is not None:
            desc.ld_r = _rows(residual, "residual", x.dtype, n, d)
        if not rows and not codes:
            raise ValueError("rows and codes: at least one")
        _on_gpu(stream, x, residual, self.weight)
        with _on(stream):
            y = x.new_empty(n, d) if rows else None
            q = x.new_empty(n, d, dtype=torch.uint8) if codes else None
            scale = x.new_empty(n, -(-d // 128), dtype=torch.float32) if codes else None
            total = x.new_empty(n, d) if residual is not None else None
            rstd = x.new_empty(n, dtype=torch.float32)
            weight = _aligned(self.weight)
        T.call("moe_rmsnorm_forward", desc, x.data_ptr(), _ptr(residual), _ptr(weight), _ptr(y),
               _ptr(q), _ptr(scale), _ptr(total), rstd.data_ptr(), _stream(stream))
        return {"y": y, "codes": q, "scale": scale, "rstd": rstd,
                "sum": x if residual is None else total}

    def backward(self, dy: torch.Tensor, x: torch.Tensor, rstd: torch.Tensor,
                 dresidual: torch.Tensor | None = None, stream=None) -> dict:
        """{"dx", "dweight"} for the forward's normalized rows x (its "sum");
        dresidual is added to dx."""
        desc = self._desc(x)
        n, d = x.shape
        desc.ld_y = _rows(dy, "dy", x.dtype, n, d)
        if dresidual is not None:
            desc.ld_r = _rows(dresidual, "dresidual", x.dtype, n, d)
        _vector(rstd, "rstd", torch.float32, n)
        _on_gpu(stream, dy, x, self.weight, rstd, dresidual)
        with _on(stream):
            dx = torch.empty(n, d, dtype=x.dtype, device=x.device)
            dw = torch.empty(d, dtype=torch.float32, device=x.device)
            need = T.moe_rmsnorm_backward_workspace_size(desc)
            ws = self._ws.get(need, x.device, stream) if need else None
            weight, rstd = _aligned(self.weight), _aligned(rstd)
        T.call("moe_rmsnorm_backward", desc, dy.data_ptr(), x.data_ptr(), _ptr(weight),
               rstd.data_ptr(), _ptr(dresidual), dx.data_ptr(), dw.data_ptr(), _ptr(ws), need,
               _stream(stream))
        return {"dx": dx, "dweight": dw}


class TokenDispatch:
    """Sorts tokens by the experts they selected and brings expert outputs back
    (moe_token_dispatch, moe_token_combine). ``rows``: places of the sorted
    matrices; None: one for every pair."""

    _DT = {**_DT, torch.uint8: L.MOE_DT_FP8_E4M3}
    # the sort's tables, shared by all dispatches of a stream and thread
    _ws = _Workspace()

    def __init__(self, n_experts: int, rows: int | None = None):
        self.n_experts, self.rows = n_experts, rows

    def forward(self, x: torch.Tensor | None, topk_idx: torch.Tensor,
                scale: torch.Tensor | None = None, into: torch.Tensor | None = None,
                scale_into: torch.Tensor | None = None, stream=None) -> dict:
        """{"rows", "scale", "offsets", "perm", "inv"} for selections topk_idx [T,
        K] int32 (outside 0 .. n_experts - 1: no place). x [T, d] bf16, fp32, or
        uint8 (E4M3) with the scales of its tiles; None sorts only. Rows go to
        ``into`` where given; those behind the last place are not written."""
        if topk_idx.dim() != 2:
            raise ValueError(f"topk_idx: expected int32 [T, K], got {list(topk_idx.shape)}")
        n, K = topk_idx.shape
        _matrix(topk_idx, "topk_idx", torch.int32, n, K)
        places = n * K if self.rows is None else min(self.rows, n * K)
        desc = T.MoeDispatchDesc(T=n, d=1, n_experts=self.n_experts, top_k=K, dtype=L.MOE_DT_F32,
                                 rows=places)
        if self.rows is not None and self.rows < 1:
            raise ValueError(f"rows: expected at least 1, got {self.rows}")
        tiles = 0
        if x is None:
            if scale is not None or into is not None or scale_into is not None:
                raise ValueError("rows or scales without x")
        else:
            if x.dim() != 2 or x.dtype not in self._DT:
                raise ValueError(f"x: expected bf16, fp32 or uint8 [T, d], got {x.dtype} "
                                 f"{list(x.shape)}")
            d = desc.d = x.shape[1]
            desc.dtype = self._DT[x.dtype]
            desc.ld_t = _rows(x, "x", x.dtype, n, d)
            if into is not None:
                desc.ld_p = _rows(into, "into", x.dtype, places, d)
            if (scale is None) != (x.dtype is not torch.uint8):
                raise ValueError("scale: with E4M3 rows, and only with them")
            if scale is not None:
                tiles = -(-d // 128)
                _matrix(scale, "scale", torch.float32, n, tiles)
                _matrix(scale_into, "scale_into", torch.float32, places, tiles)
            elif scale_into is not None:
                raise ValueError("scale_into without scale")
        _on_gpu(stream, topk_idx, x, scale, into, scale_into)
        with _on(stream):
            i32 = dict(dtype=torch.int32, device=topk_idx.device)
            offsets = torch.empty(self.n_experts + 1, **i32)
            perm, inv = torch.empty(places, **i32), torch.empty(n, K, **i32)
            if x is not None and into is None:
                into = x.new_empty(places, desc.d)
            if tiles and scale_into is None:
                scale_into = scale.new_empty(places, tiles)
            need = T.moe_token_dispatch_workspace_size(desc)
            ws = self._ws.get(need, topk_idx.device, stream) if need else None
        T.call("moe_token_dispatch", desc, topk_idx.data_ptr(), _ptr(x), _ptr(scale),
               offsets.data_ptr(), perm.data_ptr(), inv.data_ptr(), _ptr(into), _ptr(scale_into),
               _ptr(ws), need, _stream(stream))
        return {"rows": into, "scale": scale_into, "offsets": offsets, "perm": perm, "inv": inv}

    @staticmethod
    def _back(t, name, inv, rows, weight):
        """Descriptor of a return between token rows t and sorted rows."""
        if inv.dim() != 2 or t.dim() != 2 or t.dtype not in _DT:
            raise ValueError(f"expected inv int32 [T, K] and {name} bf16 or fp32 rows, got "
                             f"{list(inv.shape)} and {t.dtype} {list(t.shape)}")
        n, K = inv.shape
        _matrix(inv, "inv", torch.int32, n, K)
        _matrix(weight, "weight", torch.float32, n, K)
        if not 0 < rows <= n * K and n:
            raise ValueError(f"sorted rows: expected 1 .. T * K = {n * K}, got {rows}")
        return T.MoeDispatchDesc(T=n, d=t.shape[1], n_experts=1, top_k=K, dtype=_DT[t.dtype],
                                 rows=rows)

    @staticmethod
    def combine(rows: torch.Tensor, inv: torch.Tensor, weight: torch.Tensor | None = None,
                base: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """y [T, d] = base + sum_k weight[:, k] rows[inv[:, k]] (moe_token_combine);
        with weight None the gradient of ``forward`` in x, for rows = its "rows"'
        gradient."""
        desc = TokenDispatch._back(rows, "rows", inv, rows.shape[0], weight)
        n, d = inv.shape[0], rows.shape[1]
        desc.ld_p = _rows(rows, "rows", rows.dtype, rows.shape[0], d)
        if base is not None:
            _matrix(base, "base", rows.dtype, n, d)
        _on_gpu(stream, rows, inv, weight, base)
        with _on(stream):
            y = torch.empty(n, d, dtype=rows.dtype, device=rows.device)
        T.call("moe_token_combine", desc, rows.data_ptr(), inv.data_ptr(), _ptr(weight),
               _ptr(base), y.data_ptr(), _stream(stream))
        return y

    @staticmethod
    def combine_grad(dy: torch.Tensor, rows: torch.Tensor, inv: torch.Tensor,
                     weight: torch.Tensor | None = None, into: torch.Tensor | None = None,
                     stream=None) -> dict:
        """{"drows", "dweight"} of ``combine`` (moe_token_combine_backward; the
        gradient in base is dy): drows in ``into`` where given, rows that no pair
        has are not written; dweight None without weights."""
        desc = TokenDispatch._back(dy, "dy", inv, rows.shape[0], weight)
        n, d = inv.shape[0], dy.shape[1]
        desc.ld_t = _rows(dy, "dy", dy.dtype, n, d)
        # rows and drows share a stride: both contiguous
        _matrix(rows, "rows", dy.dtype, rows.shape[0], d)
        _matrix(into, "into", dy.dtype, rows.shape[0], d)
        _on_gpu(stream, dy, rows, inv, weight, into)
        with _on(stream):
            if into is None:
                into = torch.empty(rows.shape[0], d, dtype=dy.dtype, device=dy.device)
            dw = None if weight is None else torch.empty(inv.shape, dtype=torch.float32,
                                                         device=dy.device)
        T.call("moe_token_combine_backward", desc, dy.data_ptr(),
               None if dw is None else rows.data_ptr(), inv.data_ptr(), _ptr(weight),
               into.data_ptr(), _ptr(dw), _stream(stream))
        return {"drows": into, "dweight": dw}


def _mx4_bytes(mats: int, rows: int, k: int) -> tuple:
    """Bytes of a row's codes and words of its scales; both buffers' shapes."""
    kb = -(-k // 32)
    return (mats, rows, kb * 16), (mats, -(-kb // 4), rows, 4)


def _mx4_desc(x, k, act, perm) -> T.MoeMx4Desc:
    if x.dim() not in (2, 3) or x.dtype not in _DT:
        raise ValueError(f"x: expected bf16 or fp32 [rows, k] or [n, rows, k], got {x.dtype} "
                         f"{list(x.shape)}")
    if act not in _ACT:
        raise ValueError(f"act: None or 'swiglu', got {act!r}")
    if perm is not None:
        if x.dim() != 2:
            raise ValueError("perm: for one matrix")
        _vector(perm, "perm", torch.int32, perm.numel())
    n, rows = (1, x.shape[0]) if x.dim() == 2 else x.shape[:2]
    width = x.shape[-1]
    if act and width % 2:
        raise ValueError(f"x: rows of gate and up halves, got {width} values")
    if k is not None and width != k * (2 if act else 1):
        raise ValueError(f"x: expected rows of {k * (2 if act else 1)} values, got {width}")
    ld = width
    if x.dim() == 2:
        ld = _rows(x, "x", x.dtype, rows, width)
    elif not x.is_contiguous():
        raise ValueError("x: expected contiguous matrices")
    return T.MoeMx4Desc(n_mats=n, rows=rows if perm is None else perm.shape[0],
                        k=width // 2 if act else width, dtype=_DT[x.dtype], act=_ACT[act], ld=ld,
                        n_src=rows)


def mx4_quantize(x: torch.Tensor, perm: torch.Tensor | None = None, act: str | None = None,
                 stream=None) -> tuple:
    """(codes, scales) of x [rows, k] or [n, rows, k] (moe_mx4_quantize): uint8 [...,
    rows, ceil(k / 32) * 16] and [..., ceil(k / 128), rows, 4]. perm: of x[perm],
    zeros for entries outside x. act "swiglu": of silu(gate) * up, x = gate | up."""
    desc = _mx4_desc(x, None, act, perm)
    _on_gpu(stream, x, perm)
    cs, ss = _mx4_bytes(desc.n_mats, desc.rows, desc.k)
    with _on(stream):
        codes = torch.empty(cs[-x.dim():] if x.dim() == 3 else cs[1:], dtype=torch.uint8,
                            device=x.device)
        scales = torch.empty(ss if x.dim() == 3 else ss[1:], dtype=torch.uint8, device=x.device)
    T.call("moe_mx4_quantize", desc, x.data_ptr(), _ptr(perm), codes.data_ptr(),
           scales.data_ptr(), _stream(stream))
    return codes, scales


def mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, k: int, dtype=torch.bfloat16,
                   stream=None) -> torch.Tensor:
    """The values [..., rows, k] of mx4_quantize's codes and scales
    (moe_mx4_dequantize)."""
    if codes.dim() not in (2, 3) or dtype not in _DT:
        raise ValueError(f"expected codes [rows, bytes] or [n, rows, bytes] and bf16 or fp32 out, "
                         f"got {list(codes.shape)} and {dtype}")
    mats, rows = (1, codes.shape[0]) if codes.dim() == 2 else codes.shape[:2]
    cs, ss = _mx4_bytes(mats, rows, k)
    cut = 3 - codes.dim()
    _matrix(codes, "codes", torch.uint8, *cs[cut:])
    _matrix(scales, "scales", torch.uint8, *ss[cut:])
    _on_gpu(stream, codes, scales)
    desc = T.MoeMx4Desc(n_mats=mats, rows=rows, k=k, dtype=_DT[dtype])
    with _on(stream):
        codes, scales = _aligned(codes), _aligned(scales)
        out = torch.empty(*codes.shape[:-1], k, dtype=dtype, device=codes.device)
    T.call("moe_mx4_dequantize", desc, codes.data_ptr(), scales.data_ptr(), out.data_ptr(),
           _stream(stream))
    return out


class MX4Linear:
    """One linear map per expert with 4-bit weights, codes and scales of [groups,
    n, k] as mx4_quantize writes them, over rows sorted by expert with ``offsets``
    [groups + 1] int32 (moe_mx4_gemm). Rows outside the groups are not written.
    For gradients through the map, GroupedLinear takes ``values()``."""

    # quantized rows, shared by all maps of a stream and thread
    _ws = _Workspace()

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, k: int):
        if codes.dim() != 3 or k < 1:
            raise ValueError(f"codes: expected uint8 [groups, n, bytes], got {list(codes.shape)}")
        cs, ss = _mx4_bytes(*codes.shape[:2], k)
        _matrix(codes, "codes", torch.uint8, *cs)
        _matrix(scales, "scales", torch.uint8, *ss)
        if (codes.data_ptr() | scales.data_ptr()) & 15:
            raise ValueError("codes and scales must start on 16 bytes")
        self.codes, self.scales, self.k = codes, scales, k

    @classmethod
    def from_weight(cls, weight: torch.Tensor, stream=None) -> "MX4Linear":
        """Quantizes weight [groups, n, k], bf16 or fp32."""
        if weight.dim() != 3:
            raise ValueError(f"weight: expected [groups, n, k], got {list(weight.shape)}")
        return cls(*mx4_quantize(weight, stream=stream), weight.shape[2])

    @classmethod
    def from_blocks(cls, codes: torch.Tensor, scales: torch.Tensor, k: int | None = None,
                    stream=None) -> "MX4Linear":
        """From scales in row order, uint8 [groups, n, blocks]; rows of k values (all
        of the blocks' without it)."""
        if scales.dim() != 3:
            raise ValueError(f"scales: expected uint8 [groups, n, blocks], got {list(scales.shape)}")
        G, n, kb = scales.shape
        _matrix(codes, "codes", torch.uint8, G, n, kb * 16)
        if k is None:
            k = kb * 32
        if -(-k // 32) != kb:
            raise ValueError(f"k: expected {kb * 32 - 31} .. {kb * 32} for {kb} blocks, got {k}")
        with _on(stream):
            words = torch.nn.functional.pad(scales, (0, -kb % 4)).reshape(G, n, -1, 4)
            words = words.transpose(1, 2).contiguous()
        return cls(codes, words, k)

    def values(self, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
        """The weights [groups, n, k] that the codes stand for."""
        return mx4_dequantize(self.codes, self.scales, self.k, dtype, stream)

    def forward(self, x: torch.Tensor, offsets: torch.Tensor, act: str | None = None,
                perm: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                stream=None) -> torch.Tensor:
        """y [rows, n] = q(x) W_g^T for x [rows, k] bf16 or fp32; act and perm as in
        mx4_quantize (rows = perm's)."""
        G, n = self.codes.shape[:2]
        if x.dim() != 2:
            raise ValueError(f"x: expected [rows, k], got {list(x.shape)}")
        desc = _mx4_desc(x, self.k, act, perm)
        _vector(offsets, "offsets", torch.int32, G + 1)
        if out_dtype not in _DT:
            raise ValueError(f"out_dtype: bf16 or fp32, got {out_dtype}")
        _on_gpu(stream, x, self.codes, self.scales, offsets, perm)
        rows = desc.rows
        kb = -(-self.k // 32)
        first = (rows * kb * 16 + 255) // 256 * 256
        g = T.MoeMx4GemmDesc(rows=rows, n_groups=G, n=n, k=self.k, out_dtype=_DT[out_dtype])
        with _on(stream):
            y = torch.empty(rows, n, dtype=out_dtype, device=x.device)
            ws = self._ws.get(first + -(-kb // 4) * rows * 4, x.device, stream) if rows else None
        if rows:
            codes, at = ws.data_ptr(), _stream(stream)
            T.call("moe_mx4_quantize", desc, x.data_ptr(), _ptr(perm), codes, codes + first, at)
            T.call("moe_mx4_gemm", g, codes, codes + first, self.codes.data_ptr(),
                   self.scales.data_ptr(), offsets.data_ptr(), y.data_ptr(), at)
        return y
