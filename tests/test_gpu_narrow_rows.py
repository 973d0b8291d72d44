"""Rows that fewer lanes hold than a token has slots, and rows that end inside a wave:
every slot's place reaches all lanes of the wave."""
import numpy as np
import pytest
import torch

from test_gpu_dispatch import DEV, _check_return, _idx, _place, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K", [(3, 64), (40, 33), (70, 64), (5, 8)])
@pytest.mark.parametrize("d", [1, 7, 8, 17, 120, 511, 513, 1030, 2080, 4100])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_return(T, K, d, dt):
    _check_return(T, K, d, dt, _idx(T + d, T, K, 30, 0.2), 30, None, True, True)


@pytest.mark.parametrize("T,K", [(3, 64), (40, 33), (70, 64), (5, 8)])
@pytest.mark.parametrize("d", [1, 15, 16, 17, 250, 1030, 2080, 4100])
@pytest.mark.parametrize("dt", ["bf16", "f32", "fp8"])
def test_dispatch(T, K, d, dt):
    import sparse_mixture_experts_gate_amd as M
    idx = _idx(T + d, T, K, 30, 0.2)
    off, perm, inv = _place(idx, 30)
    x = _rows(1, T, d, dt)
    scale = _rows(2, T, -(-d // 128), "f32") if dt == "fp8" else None
    o = M.TokenDispatch(30).forward(x, torch.from_numpy(idx).to(DEV), scale)
    n = int(off[-1])
    src = torch.from_numpy(perm[:n].astype(np.int64)).to(DEV)
    assert torch.equal(o["rows"][:n], x[src])
    assert scale is None or torch.equal(o["scale"][:n], scale[src])
