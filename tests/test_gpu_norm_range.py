"""Layer normalisation of rows with large means, and of equal values, on the GPU against fp64."""
import pytest
import torch

import tiled_newton_schulz_amd as H
from test_gpu_norm import U, check_grad, close, randn

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
