"""Timed cases of the operators on a token's way through an expert layer: RMS
norm with the residual sum and an 8-bit output (forward and backward), tokens
sorted by expert and returned with weights (forward and gradients), and
microscaled 4-bit weights (quantization and products grouped by expert).

`listed()` and `draw()` give cases, `prepare()` makes one case's inputs on the
GPU, `run()` is one pass: the plain torch form in 32 bits, or with `own` the
package's entry points. `exact()` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4, "fp8": 1}
EPS = 1e-6
TILE = 128            # values that share a scale in 8 bits
BLOCK = 32            # values that share a scale in 4 bits

# widths of the repository's workloads
WIDTHS = (128, 256, 1408, 2048, 2816, 4096, 7168)
DEV = "cuda:0"


def listed():
    return [
        # one sequence decodes one token: residual sum, norm and FP8 tiles of a single row
        dict(name="rms_fwd_one_token", op="rms_fwd", n=1, d=7168, dtype="bf16", residual=True,
             out="both"),
        # a prefill batch in front of an FP8 layer: rows for the router, tiles for the experts
        dict(name="rms_fwd_prefill", op="rms_fwd", n=8192, d=7168, dtype="bf16", residual=True,
             out="both"),
        # fp32 layer of an odd width, a ragged number of tokens
        dict(name="rms_bwd_odd_f32", op="rms_bwd", n=1003, d=1407, dtype="f32", residual=False),
        # training step: norm gradient plus the residual stream's gradient
        dict(name="rms_bwd_train", op="rms_bwd", n=8192, d=7168, dtype="bf16", residual=True),
        # decode, 16 tokens x top-8 of 256 experts
        dict(name="dispatch_decode", op="dispatch", tokens=16, experts=256, k=8, d=7168,
             dtype="bf16", local=1.0),
        # prefill of the FP8 layer: E4M3 rows and their tile scales to the experts
        dict(name="dispatch_prefill_fp8", op="dispatch", tokens=8192, experts=256, k=8, d=7168,
             dtype="fp8", local=1.0),
        # one expert-parallel rank of eight: most pairs belong to experts elsewhere
        dict(name="return_rank", op="return", tokens=4096, experts=32, k=8, d=7168, dtype="bf16",
             local=0.125, weight=True, base=True, grad=False),
        # training step of the 64-expert layer, 4096 tokens x top-6: return and its gradients
        dict(name="return_train", op="return", tokens=4096, experts=64, k=6, d=2048, dtype="bf16",
             local=1.0, weight=True, base=True, grad=True),
        # a small odd-sized matrix: blocks that end inside a row, unaligned pitches
        dict(name="mx4_weights_odd", op="mx4_weights", mats=3, rows=613, k=1407, dtype="bf16"),
        # gate and up matrices of 32 experts, once per weight set
        dict(name="mx4_weights_load", op="mx4_weights", mats=32, rows=4096, k=7168, dtype="bf16"),
        # decode, 16 tokens x top-8 over 256 experts: streams the touched weights
        dict(name="mx4_product_decode", op="mx4_product", rows=128, groups=256, n=4096, k=7168,
             skew=0.0, act=False),
        # prefill of one expert-parallel rank (32 experts), loads skewed like a Zipf law
        dict(name="mx4_product_prefill", op="mx4_product", rows=8192, groups=32, n=4096, k=7168,
             skew=0.7, act=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width of the workloads, or (one in three) any odd one of the range."""
    if rng.random() < 1 / 3:
        return min(_log(rng, lo, hi) | 1, hi - 1)
    return rng.choice([w for w in WIDTHS if lo <= w <= hi])


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_bwd", "dispatch", "return", "mx4_weights", "mx4_product"])
    if op in ("rms_fwd", "rms_bwd"):
        c = dict(op=op, n=_log(rng, 1, 8192), d=_width(rng, 65, 7168),
                 dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.5)
        if op == "rms_fwd":
            c["out"] = rng.choice(["rows", "codes", "both"])
        return c
    if op in ("dispatch", "return"):
        d, k = _width(rng, 65, 7168), rng.choice([1, 2, 4, 6, 8, 8])
        dtype = rng.choice(["bf16", "bf16", "f32"] + ["fp8"] * (op == "dispatch"))
        grad = rng.random() < 0.5
        most = 4.0e8 / (k * d * SIZE[dtype])
        c = dict(op=op, tokens=max(1, min(_log(rng, 1, 16384), int(most))),
                 experts=_log(rng, max(k, 2), 512), k=k, d=d, dtype=dtype,
                 local=rng.choice([1.0, 1.0, round(rng.uniform(0.05, 0.9), 2)]))
        if op == "return":
            c.update(weight=rng.random() < 0.75, base=rng.random() < 0.5, grad=grad)
        return c
    if op == "mx4_weights":
        rows, k = _width(rng, 65, 4096), _width(rng, 65, 7168)
        return dict(op=op, mats=max(1, min(_log(rng, 1, 64), int(4.0e8 / (rows * k)))), rows=rows,
                    k=k, dtype=rng.choice(["bf16", "f32"]))
    n, k = _width(rng, 65, 4096), _width(rng, 65, 4096)
    rows = min(_log(rng, 1, 32768), int(2.0e11 / (n * k)))
    return dict(op=op, rows=rows, groups=_log(rng, 1, 128), n=n, k=k,
                skew=round(rng.uniform(0.0, 1.1), 2), act=rng.random() < 0.3)


def _tiles(d, t):
    return (d + t - 1) // t


def work(case):
    op = case["op"]
    if op in ("rms_fwd", "rms_bwd"):
        n, d, s, r = case["n"], case["d"], SIZE[case["dtype"]], int(case["residual"])
        if op == "rms_bwd":  # dy, x, dx (and the residual's gradient); weight, dweight; rstd
            return {"bytes": n * d * s * (3 + r) + 8 * d + 4 * n, "flops": n * d * (9 + r)}
        # x (and residual, sum), rows, codes and scales; weight; rstd
        b = n * d * s * (1 + 2 * r) + 4 * d + 4 * n
        f = n * d * (4 + r)
        if case["out"] != "codes":
            b += n * d * s
        if case["out"] != "rows":
            b += n * d + 4 * n * _tiles(d, TILE)
            f += 3 * n * d
        return {"bytes": b, "flops": f}
    if op in ("dispatch", "return"):
        t, k, s = case["tokens"], case["k"], SIZE[case["dtype"]]
        row = case["d"] * s + (4 * _tiles(case["d"], TILE) if case["dtype"] == "fp8" else 0)
        pairs = t * k * case["local"]
        if op == "dispatch":  # rows in, sorted rows out; selections, offsets, perm, inv
            return {"bytes": row * (t + pairs) + 12 * t * k + 4 * case["experts"], "flops": t * k}
        b = row * (t * (1 + int(case["base"])) + pairs) + t * k * (4 + 4 * int(case["weight"]))
        f = 2 * pairs * case["d"]
        if case["grad"]:  # dy, the rows again for dweight, drows
            b += row * (t + pairs) + 4 * t * k * int(case["weight"])
            f += (3 if case["weight"] else 1) * pairs * case["d"]
        return {"bytes": b, "flops": f}
    if op == "mx4_weights":  # values in; codes and scales; the values they stand for
        m, r, k = case["mats"], case["rows"], case["k"]
        return {"bytes": m * r * (k * (SIZE[case["dtype"]] + 2) + 17 * _tiles(k, BLOCK)),
                "flops": 4 * m * r * k}
    rows, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
    touched = float(np.sum(1.0 - (1.0 - _shares(case)) ** rows))  # expected groups with a row
    return {"bytes": rows * (2 * k * (2 if case["act"] else 1) + 2 * n)
            + touched * n * 17 * _tiles(k, BLOCK), "flops": 2 * rows * n * k}


def _shares(case):
    w = (np.arange(case["groups"]) + 1.0) ** -case["skew"]
    return w / w.sum()


# ---- inputs ----------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _selections(g, case):
    """Distinct experts per token, popular ones among them; those past the rank's
    own experts (`local` of them are its) count as none."""
    t, e, k = case["tokens"], case["experts"], case["k"]
    every = max(e, int(round(e / case["local"])))
    every = max(every, k)
    score = torch.rand(t, every, generator=g, device=DEV) + 0.3 * torch.rand(
        1, every, generator=g, device=DEV)
    idx = score.topk(k, dim=1).indices
    return torch.where(idx < e, idx, -1).int().contiguous()


def _sorted(idx, e):
    """offsets, perm, inv of the stable sort of the pairs by expert; pairs without
    an expert come last, without a place."""
    flat = idx.reshape(-1).long()
    key = torch.where(flat < 0, e, flat)
    order = torch.sort(key, stable=True).indices
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.bincount(key, minlength=e + 1)[:e].cumsum(0).int()
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=DEV)
    there = key < e
    perm = torch.where(key[order] < e, order // idx.shape[1], -1).int()
    return offsets, perm, torch.where(there, place, -1).int().reshape(idx.shape)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)
    op, s = case["op"], {"case": case}
    if op in ("rms_fwd", "rms_bwd"):
        n, d, dt = case["n"], case["d"], DT[case["dtype"]]
        # a residual stream: a few channels carry large values
        chan = 1.0 + 15.0 * (torch.rand(d, generator=g, device=DEV) < 0.01)
        s["x"] = (_randn(g, n, d) * chan).to(dt)
        s["r"] = _randn(g, n, d).to(dt) if case["residual"] else None
        s["w"] = 1.0 + 0.1 * _randn(g, d)
        if op == "rms_bwd":  # what the forward kept, and the incoming gradient
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dy"] = _randn(g, n, d).to(dt)
        return s
    if op in ("dispatch", "return"):
        t, k, d = case["tokens"], case["k"], case["d"]
        s["idx"] = _selections(g, case)
        if op == "dispatch":
            if case["dtype"] == "fp8":  # tiles scaled to their largest value
                f = _randn(g, t, _tiles(d, TILE) * TILE)
                f[:, d:] = 0
                f = f.reshape(t, -1, TILE)
                top = f.abs().amax(2, keepdim=True)
                s["scale"] = (top / 448.0).squeeze(2).contiguous()
                s["x"] = (f * (448.0 / top)).to(torch.float8_e4m3fn).reshape(t, -1)[:, :d] \
                    .contiguous().view(torch.uint8)
            else:
                s["x"], s["scale"] = _randn(g, t, d).to(DT[case["dtype"]]), None
            # the program's own buffers: rows behind the last pair stay as they are
            s["rows"] = torch.zeros(t * k, d, dtype=s["x"].dtype, device=DEV)
            s["row_scale"] = None if s["scale"] is None else torch.zeros(
                t * k, s["scale"].shape[1], device=DEV)
            return s
        dt = DT[case["dtype"]]
        s["inv"] = _sorted(s["idx"], case["experts"])[2]
        s["rows"] = _randn(g, t * k, d).to(dt)
        s["weight"] = torch.softmax(_randn(g, t, k), 1) if case["weight"] else None
        s["base"] = _randn(g, t, d).to(dt) if case["base"] else None
        if case["grad"]:
            s["dy"] = _randn(g, t, d).to(dt)
            s["drows"] = torch.zeros(t * k, d, dtype=dt, device=DEV)
        return s
    if op == "mx4_weights":
        m, r, k = case["mats"], case["rows"], case["k"]
        s["w"] = torch.empty(m, r, k, dtype=DT[case["dtype"]], device=DEV)
        for i in range(m):  # rows of different magnitudes, as trained weights have
            s["w"][i] = _randn(g, r, k) * 0.02 * torch.exp(0.5 * _randn(g, r, 1))
        return s
    rows, G, n, k = case["rows"], case["groups"], case["n"], case["k"]
    rs = np.random.RandomState(seed % (1 << 31))
    # loads in a random order of the experts; the host knows them from its own batch plan
    lens = rs.multinomial(rows, rs.permutation(_shares(case)))
    s["lens"] = [int(v) for v in lens]
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    s["offsets"] = torch.from_numpy(off).to(DEV)
    # weights as they are kept: packed codes, scales in groups of four blocks
    kb = _tiles(k, BLOCK)
    s["codes"] = torch.empty(G, n, kb * 16, dtype=torch.uint8, device=DEV)
    s["scales"] = torch.empty(G, _tiles(kb, 4), n, 4, dtype=torch.uint8, device=DEV)
    for e in range(G):
        q, b = _mx4(_randn(g, n, k) * 0.02)
        s["codes"][e], s["scales"][e] = _pack(q), _grouped_scales(b)
    s["x"] = _randn(g, rows, 2 * k if case["act"] else k).bfloat16()
    return s


def run(s):
    return _own(s) if own else _plain(s)


# ---- the package's entry points ------------------------------------------------
def _kept(s, make):
    """The operator object that a program keeps from call to call."""
    if "op" not in s:
        s["op"] = make()
    return s["op"]


def _own(s):
    import sparse_mixture_experts_gate_amd as M
    c = s["case"]
    op = c["op"]
    if op == "rms_fwd":
        norm = _kept(s, lambda: M.RMSNorm(s["w"], EPS))
        o = norm.forward(s["x"], s["r"], rows=c["out"] != "codes", codes=c["out"] != "rows")
        out = {"rstd": o["rstd"]}
        if c["out"] != "codes":
            out["y"] = o["y"]
        if c["out"] != "rows":
            out["codes"], out["scale"] = o["codes"].view(torch.float8_e4m3fn), o["scale"]
        if s["r"] is not None:
            out["sum"] = o["sum"]
        return out
    if op == "rms_bwd":
        norm = _kept(s, lambda: M.RMSNorm(s["w"], EPS))
        return norm.backward(s["dy"], s["x"], s["rstd"], s["r"])
    if op == "dispatch":
        disp = _kept(s, lambda: M.TokenDispatch(c["experts"]))
        o = disp.forward(s["x"], s["idx"], s["scale"], into=s["rows"], scale_into=s["row_scale"])
        return _dispatched(s, o["rows"], o["scale"], o["offsets"], o["perm"], o["inv"])
    if op == "return":
        out = {"y": M.TokenDispatch.combine(s["rows"], s["inv"], s["weight"], s["base"])}
        if c["grad"]:
            o = M.TokenDispatch.combine_grad(s["dy"], s["rows"], s["inv"], s["weight"],
                                             into=s["drows"])
            out["drows"] = o["drows"]
            if c["weight"]:
                out["dweight"] = o["dweight"]
        return out
    if op == "mx4_weights":
        codes, scales = M.mx4_quantize(s["w"])
        return {"w": M.mx4_dequantize(codes, scales, c["k"])}
    lin = _kept(s, lambda: M.MX4Linear(s["codes"], s["scales"], c["k"]))
    return {"y": lin.forward(s["x"], s["offsets"], act="swiglu" if c["act"] else None)}


def _dispatched(s, rows, scale, offsets, perm, inv):
    out = {"offsets": offsets, "perm": perm, "inv": inv}
    out["rows"] = rows if scale is None else rows.view(torch.float8_e4m3fn)
    if scale is not None:
        out["scale"] = scale
    return out


# ---- plain form, 32 bits -------------------------------------------------------
def _power(e):
    """2^e, e = -127 .. 127, from its bits (a power function may be off by some)."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).int().view(torch.float32)


def _mx4(v):
    """Codes (0 .. 15) and scale bytes of the blocks of 32 along the last axis:
    the scale is the power of two below the block's largest value, over 4; halves
    go to the even code, values past 6 to 6."""
    k = v.shape[-1]
    v = torch.nn.functional.pad(v.float(), (0, -k % BLOCK))
    v = v.reshape(*v.shape[:-1], -1, BLOCK)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
    a = v.abs() * _power(-e)
    q = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
         + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    return (q + 8 * torch.signbit(v).int()).flatten(-2), (e + 127).squeeze(-1)


def _pack(q):
    return (q[..., 0::2] + 16 * q[..., 1::2]).to(torch.uint8)


def _grouped_scales(b):
    """[rows, blocks] -> [blocks / 4, rows, 4], zeros past the last block."""
    b = torch.nn.functional.pad(b, (0, -b.shape[-1] % 4))
    return b.reshape(b.shape[0], -1, 4).transpose(0, 1).to(torch.uint8)


def _value(q, b):
    """Values of codes [..., k'] and scale bytes [..., k' / 32]."""
    m = q & 7
    mag = torch.where(m < 2, 0.5 * m, 0.25 * ((2 + (m & 1)) << (m >> 1)))
    v = torch.where(q > 7, -mag, mag).reshape(*b.shape, BLOCK)
    return (v * _power(b - 127).unsqueeze(-1)).flatten(-2)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "rms_fwd":
        v, dt = s["x"].float(), s["x"].dtype
        if s["r"] is not None:
            v = v + s["r"].float()
        rstd = torch.rsqrt(v.square().mean(1) + EPS)
        o = v * rstd[:, None] * s["w"]
        out = {"rstd": rstd}
        if c["out"] != "codes":
            out["y"] = o.to(dt)
        if c["out"] != "rows":
            t = torch.nn.functional.pad(o, (0, -c["d"] % TILE)).reshape(c["n"], -1, TILE)
            top = t.abs().amax(2, keepdim=True)
            out["scale"] = (top / 448.0).squeeze(2)
            out["codes"] = (t * (448.0 / top)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn) \
                .reshape(c["n"], -1)[:, :c["d"]].contiguous()
        if s["r"] is not None:
            out["sum"] = v.to(dt)
        return out
    if op == "rms_bwd":
        dt = s["x"].dtype
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        z = s["x"].float() * rstd
        g = dy * s["w"]
        dx = rstd * (g - z * (g * z).mean(1, keepdim=True))
        if s["r"] is not None:
            dx = dx + s["r"].float()
        return {"dx": dx.to(dt), "dweight": (dy * z).sum(0)}
    if op == "dispatch":
        offsets, perm, inv = _sorted(s["idx"], c["experts"])
        rows, scale = s["rows"], s["row_scale"]
        there = (perm >= 0)[:, None]
        at = perm.clamp(min=0).long()
        rows.copy_(torch.where(there, s["x"][at], rows))
        if scale is not None:
            scale.copy_(torch.where(there, s["scale"][at], scale))
        return _dispatched(s, rows, scale, offsets, perm, inv)
    if op == "return":
        inv, rows, w = s["inv"], s["rows"], s["weight"]
        there = inv >= 0
        at = inv.clamp(min=0).long()
        y = torch.zeros(inv.shape[0], rows.shape[1], device=DEV) if s["base"] is None \
            else s["base"].float()
        wt = there.float() if w is None else torch.where(there, w, 0.0)
        picked = torch.where(there[:, :, None], rows[at], 0)  # in the rows' own type
        out = {"y": (y + torch.bmm(wt[:, None], picked.float()).squeeze(1)).to(rows.dtype)}
        if c["grad"]:
            dy = s["dy"].float()
            d = (wt[:, :, None] * dy[:, None]).to(rows.dtype)
            s["drows"][inv[there].long()] = d[there]
            out["drows"] = s["drows"]
            if w is not None:
                out["dweight"] = (picked.float() * dy[:, None]).sum(2)
        return out
    if op == "mx4_weights":
        w = torch.empty(s["w"].shape, dtype=torch.bfloat16, device=DEV)
        for o, m in zip(w, s["w"]):
            o.copy_(_value(*_mx4(m))[:, :c["k"]])
        return {"w": w}
    # one product for each expert that has rows: no padding to the largest load
    x = s["x"].float()
    if c["act"]:
        gate, up = x.chunk(2, 1)
        x = gate * torch.sigmoid(gate) * up
    x = _value(*_mx4(x))
    out = torch.empty(x.shape[0], c["n"], dtype=torch.bfloat16, device=DEV)
    kb = _tiles(c["k"], BLOCK)
    for e, (a, o) in enumerate(zip(x.split(s["lens"]), out.split(s["lens"]))):
        if s["lens"][e]:
            q = s["codes"][e].int()
            q = torch.stack((q & 15, q >> 4), 2).flatten(1)
            b = s["scales"][e].transpose(0, 1).flatten(1)[:, :kb].int()
            o.copy_(torch.matmul(a, _value(q, b).t()))
    return {"y": out}


# ---- the definitions in 64 bits ------------------------------------------------
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _power64(e):
    return ((e.long() + 1023) * 2 ** 52).view(torch.float64)


def _exact_mx4(v):
    """Values that 4 bits keep of v [rows, k], in 64 bits: even halves of the spacing
    at the value's magnitude, in units of the block's scale."""
    rows, k = v.shape
    p = torch.zeros(rows, _tiles(k, BLOCK) * BLOCK, dtype=torch.float64, device=DEV)
    p[:, :k] = v
    p = p.view(rows, -1, BLOCK)
    top = p.abs().max(2, keepdim=True).values
    _, up = torch.frexp(torch.where(top > 0, top, 1.0))  # top < 2^up <= 2 top
    unit = _power64(up - 3)
    a = p.abs() / unit
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    return (torch.sign(p) * a * unit).view(rows, -1)[:, :k]


def exact(case, seed):
    s = prepare(case, seed)
    op, f8 = case["op"], torch.float64
    if op in ("rms_fwd", "rms_bwd"):
        v, w = s["x"].to(f8), s["w"].to(f8)
        if op == "rms_fwd":
            if case["residual"]:
                v = v + s["r"].to(f8)
            inv = 1.0 / torch.sqrt((v * v).sum(1) / case["d"] + EPS)
            o = v * inv.unsqueeze(1) * w
            out = {"rstd": inv}
            if case["out"] != "codes":
                out["y"] = o
            if case["out"] != "rows":  # the scaled values, before their rounding
                d = case["d"]
                edge = list(range(0, d, TILE))
                top = torch.stack([o[:, i:i + TILE].abs().max(1).values for i in edge], 1)
                out["scale"] = top / 448
                out["codes"] = o / out["scale"].repeat_interleave(TILE, 1)[:, :d]
            if case["residual"]:
                out["sum"] = v
            return out
        # y_i = w_i z_i, z = x rstd(x): the chain rule, term by term
        inv, dy = s["rstd"].to(f8).unsqueeze(1), s["dy"].to(f8)
        dz = dy * w
        dx = inv * dz - v * inv ** 3 * (dz * v).sum(1, keepdim=True) / case["d"]
        if case["residual"]:
            dx = dx + s["r"].to(f8)
        return {"dx": dx, "dweight": torch.einsum("nd,nd->d", dy, v * inv)}
    if op == "dispatch":
        # pair by pair on the host: a place is the number of pairs before it
        idx = s["idx"].cpu().numpy()
        flat, k = idx.reshape(-1), case["k"]
        order = [p for p in np.argsort(flat, kind="stable") if flat[p] >= 0]
        inv = np.full(flat.size, -1, np.int32)
        inv[order] = np.arange(len(order))
        perm = np.full(flat.size, -1, np.int32)
        perm[:len(order)] = np.asarray(order, np.int64) // k
        off = np.searchsorted(flat[order], np.arange(case["experts"] + 1)).astype(np.int32)
        src = torch.from_numpy(perm[:len(order)].astype(np.int64)).to(DEV)
        s["rows"][:len(order)] = s["x"].index_select(0, src)
        if s["scale"] is not None:
            s["row_scale"][:len(order)] = s["scale"].index_select(0, src)
        return _dispatched(s, s["rows"], s["row_scale"], off, perm, inv.reshape(idx.shape))
    if op == "return":
        inv = s["inv"].long()
        t, k = inv.shape
        y = torch.zeros(t, case["d"], dtype=f8, device=DEV)
        if case["base"]:
            y += s["base"].to(f8)
        out, dwt = {}, torch.zeros(t, k, dtype=f8, device=DEV)
        for j in range(k):  # slot by slot, over the tokens that have a row there
            tok = torch.nonzero(inv[:, j] >= 0).squeeze(1)
            src = inv[tok, j]
            r = s["rows"].index_select(0, src).to(f8)
            wj = s["weight"][tok, j].to(f8).unsqueeze(1) if case["weight"] else 1.0
            y.index_add_(0, tok, r * wj)
            if case["grad"]:
                dy = s["dy"].index_select(0, tok).to(f8)
                dwt[tok, j] = (dy * r).sum(1)
                if "drows" not in out:
                    out["drows"] = s["drows"].to(f8)
                out["drows"][src] = dy * wj
        out["y"] = y
        if case["grad"] and case["weight"]:
            out["dweight"] = dwt
        return out
    if op == "mx4_weights":
        return {"w": torch.stack([_exact_mx4(m.to(f8)) for m in s["w"]])}
    x = s["x"].to(f8)
    if case["act"]:
        gate, up = x[:, :case["k"]], x[:, case["k"]:]
        x = gate / (1.0 + torch.exp(-gate)) * up
    x = _exact_mx4(x)
    grid = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=f8, device=DEV)
    kb, n = _tiles(case["k"], BLOCK), case["n"]
    parts, at = [], 0
    for e, m in enumerate(s["lens"]):
        if m:
            two = s["codes"][e].long()
            w = torch.empty(n, kb * BLOCK, dtype=f8, device=DEV)
            w[:, 0::2], w[:, 1::2] = grid[two % 16], grid[two // 16]
            unit = _power64(s["scales"][e].permute(1, 0, 2).reshape(n, -1)[:, :kb].long() - 127)
            w = w * unit.repeat_interleave(BLOCK, 1)
            parts.append(x[at:at + m] @ w[:, :case["k"]].T)
        at += m
    return {"y": torch.cat(parts)}
