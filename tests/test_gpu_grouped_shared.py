"""Long contractions of fewer tiles than workgroups: the idle workgroups share
them. Their partial tiles meet in the workspace, which shows the sharing.

Bound: fp32 sums of k terms in any order are off by at most k u of their
absolute terms (u = 2^-24); a bf16 output adds up to 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import oracle.block_ops as B
from parity_util import host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SLOT = 256 * 256 * 4  # bytes of a partial tile


def _rand(seed, *shape):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda:0").bfloat16()


@pytest.mark.parametrize("op", ["forward", "dgrad"])
@pytest.mark.parametrize("lens,deep", [([1536], 7168), ([500] * 8, 4096)])
def test_tiles_of_one_round_are_shared(op, lens, deep):
    import sparse_mixture_experts_gate_amd as M
    rows, wide = sum(lens), 1408
    n, k = (wide, deep) if op == "forward" else (deep, wide)
    off_h = np.concatenate([[0], np.cumsum(lens)])
    off = torch.tensor(off_h, dtype=torch.int32, device="cuda:0")
    w, a = _rand(1, len(lens), n, k), _rand(2, rows, deep)
    d = M.MoeGroupedDesc(rows=rows, n_groups=len(lens), n=n, k=k, out_dtype=M.MOE_DT_F32)
    which = M.MOE_GROUPED_FORWARD if op == "forward" else M.MOE_GROUPED_DGRAD
    size = M.moe_grouped_gemm_workspace_size(d, which)
    assert size > 256 * SLOT
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda:0")
    out = torch.empty(rows, wide, device="cuda:0")
    call = M.moe_grouped_gemm if op == "forward" else M.moe_grouped_gemm_dgrad
    call(d, a, w, off, out, ws)
    written = ws[:256 * SLOT].view(torch.int32).view(256, -1).ne(-1).any(1)
    used = int(written.sum())
    assert used >= 64 and bool(written[:used].all())
    # no counter is left behind, and a repeat gives the same bits
    assert not ws[256 * SLOT:].any()
    again = torch.empty_like(out)
    call(d, a, w, off, again, ws)
    assert torch.equal(out, again)
    f = B.grouped if op == "forward" else B.grouped_dgrad
    ha, hw = host(a).astype(np.float64), host(w).astype(np.float64)
    ref, mag = f(ha, hw, off_h), f(np.abs(ha), np.abs(hw), off_h)
    bad = ~(np.abs(host(out) - ref) <= (deep + 2) * U * mag)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
