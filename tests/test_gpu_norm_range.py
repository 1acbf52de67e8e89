"""Layer normalisation of rows with large means, and of equal values, on the GPU against fp64."""
import pytest
import torch

import tiled_newton_schulz_amd as H
from test_gpu_norm import COLS, U, check_grad, close, randn

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("cols", [1, 2, 3, 5, 7, 8, 12, 33, 40, 64, 100, 104])
def test_gradients_of_large_equal_rows(cuda, cols, dt):
    """Rows of equal values so large that mean rstd is infinite: x_hat is 0 in the row, and
    what a thread holds past the row's end reaches no gradient."""
    print(f"layer norm gradients, large equal rows of {cols} {dt}", flush=True)
    x = torch.tensor([2.0, -(2.0 ** 120), 2.0 ** 121, 0.0, -(2.0 ** 121)], device=cuda)[:, None].expand(5, cols).to(TYPES[dt]).contiguous()
    w, dy = randn((cols,), dt, 1), randn((5, cols), dt, 2)
    stats = torch.stack([x[:, 0].float(), torch.full((5,), 1e-5, device=cuda).rsqrt()], dim=1).contiguous()
    g = check_grad(x, w, stats, dy, dt)
    check_grad(x, None, stats, dy, dt)
    assert torch.all(g.dweight == 0)


@pytest.mark.parametrize("cols", COLS)
def test_equal_values(cuda, cols):
    """Rows of equal fp32 values of 24 bits: mean exact, variance 0, so y is the bias.  (The
    mean is first off by m <= 16 units in the last place; the differences are all m units,
    and their sums, up to 32768 m and 32768 m^2 units, are exact for m up to 22.)"""
    print(f"layer norm, equal values, {cols} columns", flush=True)
    values = torch.tensor([1.1, 3.3, 0.1, -1e5 / 3, 7e-5, -2.7e10, 1.9999999, 1.0000001, 1e-12, 123456.789], device=cuda)
    x = values[:, None].expand(len(values), cols).contiguous()
    w, b = randn((cols,), "fp32", 1), randn((cols,), "fp32", 2)
    for eps in (1e-5, 1e-12):
        r = H.himuon_layer_norm(x, w, b, eps=eps)
        assert torch.equal(r.y, b.expand_as(x))
        assert torch.equal(r.stats[:, 0], values)
        rstd = torch.tensor(eps, dtype=torch.float32).double().rsqrt()   # (eps as the call takes it)
        assert torch.all((r.stats[:, 1].double() / rstd.cuda() - 1).abs() <= 4 * U)


@pytest.mark.parametrize("cols", [2, 7, 64, 200, 513, 1409, 4096, 4097, 12000, 32767])
@pytest.mark.parametrize("mean", [1e3, -1e5, 3e6])
def test_large_means(cuda, cols, mean):
    """fp32 rows whose mean is far above their spread: y is as near as the spread allows.
    The first mean is off by at most Em = 92 u mean |x|; differences to it are exact (or off
    by u of themselves), their sum by 92 u mean |d| and their squares' by 96 u mean d^2, with
    d up to |x - mean| + Em.  The variance, mean d^2 - (mean d)^2, is off by at most
    300 u (var + Em^2), as |mean d| mean |d| <= mean d^2; the stored mean is rounded once more."""
    print(f"layer norm, mean {mean}, {cols} columns", flush=True)
    x = randn((9, cols), "fp32", 1, 1.5, mean)
    w, b = randn((cols,), "fp32", 2), randn((cols,), "fp32", 3)
    eps = 1e-5
    r = H.himuon_layer_norm(x, w, b, eps=eps)
    x64, w64, b64 = x.double(), w.double(), b.double()
    m = x64.mean(1, keepdim=True)
    d = x64 - m
    var = d.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    em = 92 * U * x64.abs().mean(1, keepdim=True)
    off_m = 95 * U * (d.abs().mean(1, keepdim=True) + em)
    off_r = 150 * U * (var + em ** 2) / (var + eps) + 4 * U
    y = d * rstd * w64 + b64
    off = w64.abs() * (rstd * (off_m + 2 * U * (d.abs() + em)) + (d * rstd).abs() * off_r) + 2 * U * (y.abs() + b64.abs())
    close(r.y, y, off, "fp32", "y")
    s = r.stats.double()
    assert torch.all((s[:, :1] - m).abs() <= off_m + U * m.abs())
    assert torch.all((s[:, 1:] / rstd - 1).abs() <= off_r)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("cols", [8, 64, 100, 513, 4096, 20000])
def test_squares_past_the_range(cuda, cols, dt):
    """Differences whose squares are infinite in fp32: rstd is 0 and y the bias, also where
    sums of the differences pass the range on their way."""
    print(f"layer norm, squares past fp32's range, {cols} columns {dt}", flush=True)
    x = torch.zeros((4, cols), device=cuda)
    x[0, 0], x[0, 1] = 3e38, -3e38
    x[1] = randn((cols,), "fp32", 1, 1e25)
    x[2, :2], x[2, 4:6] = 1.6e38, -1.6e38        # 3.2e38 in one thread's sum, 0 in all
    x[3, :2], x[3, 2:6] = 1.6e38, -1.6e38        # as far, and a mean below 0
    w, b = randn((cols,), dt, 2), randn((cols,), dt, 3)
    r = H.himuon_layer_norm(x.to(TYPES[dt]), w, b)
    assert torch.all(r.stats[:, 1] == 0) and torch.isfinite(r.stats).all()
    assert torch.equal(r.y, b.expand_as(r.y))


@pytest.mark.parametrize("cols", COLS)
def test_equal_values_in_bf16(cuda, cols):
    """Equal bf16 values have exact sums: up to 2^15 times 8 bits."""
    print(f"layer norm, equal bf16 values, {cols} columns", flush=True)
    x = torch.tensor([1.1, 3.3, -1e5 / 3, 2.7e10, 1e-12], device=cuda).bfloat16()[:, None].expand(5, cols).contiguous()
    w, b = randn((cols,), "bf16", 1), randn((cols,), "bf16", 2)
    r = H.himuon_layer_norm(x, w, b)
    assert torch.equal(r.y, b.expand_as(x)) and torch.equal(r.stats[:, 0], x[:, 0].float())


def test_the_stats_refusal_names_the_rows(cuda):
    x = randn((4, 16), "bf16", 1)
    st = H.himuon_layer_norm(x).stats
    for bad in (st[:3], st.t().contiguous().t(), st.cpu()):
        with pytest.raises(ValueError, match="stats must be contiguous with 2 entries per row, on the rows' GPU|tensors must be on one GPU"):
            H.himuon_layer_norm_grad(x, None, bad, x)
