"""Weight gradients of odd widths in buffers whose rows are padded to whole
16-byte chunks: the last column of a group's last row ends inside a dword.

Bound: the sum over K rows in any order is off by at most K u of its absolute
terms (u = 2^-24); the products of bf16 values are exact in fp32.
"""
import numpy as np
import pytest
import torch

import oracle.block_ops as B
from parity_util import host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _rand(seed, *shape):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda:0").bfloat16()


def _padded(t):
    """t inside rows padded to a multiple of eight values with NaN."""
    buf = torch.full((t.shape[0], (t.shape[1] + 7) // 8 * 8), float("nan"), device="cuda:0",
                     dtype=t.dtype)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


@pytest.mark.parametrize("lens", [[1], [1, 1, 1], [1, 64, 0, 65, 7], [200, 129, 1]])
@pytest.mark.parametrize("n,k", [(407, 213), (65, 64), (64, 65), (1, 1), (213, 407), (3, 2049)])
def test_weight_gradient_odd_widths_in_padded_rows(lens, n, k):
    _check(lens, n, k)


@pytest.mark.parametrize("lens,n,k", [
    ([4000, 5000], 133, 71),                  # the contraction is split
    ([8001], 71, 133),
    ([500, 0, 999, 1], 2055, 2049),           # 256 x 256 tiles
])
def test_weight_gradient_odd_widths_in_padded_rows_of_other_tiles(lens, n, k):
    _check(lens, n, k)


def _check(lens, n, k):
    import sparse_mixture_experts_gate_amd as M
    off_h = np.concatenate([[0], np.cumsum(lens)])
    off = torch.tensor(off_h, dtype=torch.int32, device="cuda:0")
    x, dy = _rand(1, sum(lens), k), _rand(2, sum(lens), n)
    dw = host(M.GroupedLinear.weight_grad(_padded(dy), _padded(x), off)).astype(np.float64)
    hx, hdy = host(x).astype(np.float64), host(dy).astype(np.float64)
    ref, mag = B.grouped_wgrad(hdy, hx, off_h), B.grouped_wgrad(np.abs(hdy), np.abs(hx), off_h)
    bad = ~(np.abs(dw - ref) <= U * np.abs(ref) + (max(lens) + 2) * U * mag + 1e-30)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), dw[bad][:4], ref[bad][:4])
