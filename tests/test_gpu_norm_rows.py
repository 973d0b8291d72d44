"""Layer norm over more rows than one launch may hold work items for (2^32 in
a dimension). The rows checked are bit for bit those of a call on them alone,
which other tests compare with the definition."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,d", [((1 << 26) + 5, 8), ((1 << 24) + 3, 1025)])
def test_rows_past_one_launch(n, d):
    import sparse_mixture_experts_gate_amd as M
    x = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda:0")
    g = torch.Generator(device="cuda:0")
    g.manual_seed(1)
    at = sorted({r for p in (0, n // 3, 1 << 22, 1 << 23, 1 << 24, 1 << 25, 1 << 26, n)
                 for r in (p - 1, p, p + 1) if 0 <= r < n})
    some = torch.tensor(at, device="cuda:0")
    rows = torch.randn(len(at), d, generator=g, device="cuda:0").bfloat16()
    x[some] = rows
    b = torch.randn(d, generator=g, device="cuda:0")
    desc = M.MoeNormDesc(n=n, d=d, dtype=M.MOE_DT_BF16, eps=1e-5)
    mean, rstd = torch.full((n,), 7.0, device="cuda:0"), torch.full((n,), 7.0, device="cuda:0")
    M.moe_layernorm_forward(desc, x, None, None, b, x, None, mean, rstd)  # in place
    want = M.LayerNorm(None, b).forward(rows)
    assert torch.equal(x[some], want["y"])
    assert torch.equal(mean[some], want["mean"]) and torch.equal(rstd[some], want["rstd"])
    # every other row held zeros: its y is the bias
    mean[some] = 0
    assert not mean.any()
    x[some] = b.bfloat16()
    for i in range(0, n, 1 << 24):
        assert bool((x[i:i + (1 << 24)] == b.bfloat16()).all())


def test_rows_of_one_value_far_apart():
    """An [n, 1] view has a row stride only; its mean is the value itself."""
    import sparse_mixture_experts_gate_amd as M
    buf = torch.randn(2, 300, device="cuda:0")
    x, buf = buf.t()[::3, :1], buf[0]
    b = torch.full((1,), 2.5, device="cuda:0")
    f = M.LayerNorm(None, b).forward(x)
    assert torch.equal(f["mean"], buf[::3]) and bool((f["y"] == 2.5).all())
    dx = M.LayerNorm(None, b).backward(x, x, f["mean"], f["rstd"], x)["dx"]
    assert torch.equal(dx, x)


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_vectors_at_any_element(shift):
    """Weights that are views of one flat parameter buffer, statistics of a
    slice of the rows: bit for bit the same as aligned ones."""
    import sparse_mixture_experts_gate_amd as M
    n, d = 9, 200
    x, dy = torch.randn(n, d, device="cuda:0"), torch.randn(n, d, device="cuda:0")
    flat = torch.randn(2 * d + shift, device="cuda:0")
    w, b = flat[shift:shift + d], flat[shift + d:]
    f = M.LayerNorm(w, b).forward(x)
    want = M.LayerNorm(w.clone(), b.clone()).forward(x)
    assert torch.equal(f["y"], want["y"])
    norm = M.LayerNorm(w, b)
    got = norm.backward(dy[shift:], x[shift:], f["mean"][shift:], f["rstd"][shift:])
    ref = M.LayerNorm(w.clone()).backward(dy[shift:], x[shift:], f["mean"][shift:].clone(),
                                          f["rstd"][shift:].clone())
    for k in ref:
        assert torch.equal(got[k], ref[k])
    s = torch.cuda.Stream()  # an aligned copy is made on the stream of the call
    s.wait_stream(torch.cuda.current_stream())
    w.mul_(2)
    s.wait_stream(torch.cuda.current_stream())
    y = norm.forward(x, stream=s)["y"]
    s.synchronize()
    assert torch.equal(y, norm.forward(x)["y"]) and not torch.equal(y, f["y"])
