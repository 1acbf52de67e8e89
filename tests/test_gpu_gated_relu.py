"""relu in the gated experts' block at gates of any size.

Every product here is a power of two times one factor, and all other terms of a sum are
0: results are exact in either type.  (du is looked at where it is a normal number.)
"""
import pytest
import torch

import tiled_newton_schulz_amd as H

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
LEAST = 2.0 ** -126   # smallest normal number
SIZES = [LEAST, 1.5 * LEAST, 1e-36, 1e-30, 1e-28, 1.9e-28, 1.95e-28, 2e-28, 2.05e-28, 2.1e-28, 3e-28, 1e-27, 1e-20, 1e-3, 1.0, 300.0]
UP = 2.0 ** 90


def gates(n, dt, more=()):
    """n gates: the sizes above in both signs, zeros of both signs, and `more`."""
    v = torch.tensor([s * x for x in [*SIZES, *more] for s in (1.0, -1.0)] + [0.0, -0.0], dtype=torch.float64)
    return v.repeat(-(-n // len(v)))[:n].to(TYPES[dt]).cuda()


def ends_of(counts):
    return torch.tensor(counts).cumsum(0).to(torch.int32).cuda()


# rows of each expert, K, N: few rows, 256-tiles, tiles of 64 (one or four parts) and of 128 off the 16-byte grid
CASES = [([3, 5], 16, 24), ([20] * 64, 16, 776), ([40, 30], 17, 25), ([40, 30], 600, 25), ([3000], 17, 1501)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_forward(cuda, counts, K, N, dt):
    print(f"relu gates {len(counts)} x {counts[0]} rows, {K} x {N} {dt}", flush=True)
    n, M = len(counts), sum(counts)
    x = torch.zeros((M, K), dtype=TYPES[dt], device=cuda)
    x[:, 0] = 1
    w = torch.ones((n, K, 2 * N), dtype=TYPES[dt], device=cuda)
    g = gates(N, dt)
    w[:, 0, :N], w[:, 0, N:] = g, UP
    r = H.himuon_grouped_gated_mm(x, w, ends_of(counts), act="relu", keep=True)
    assert torch.equal(r.pre[:, :N], g.expand(M, N)) and torch.all(r.pre[:, N:] == UP)
    assert torch.equal(r.h, (g.double().clamp(min=0) * UP).to(TYPES[dt]).expand(M, N))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_gradient(cuda, counts, K, N, dt):
    print(f"relu gates, gradient {len(counts)} x {counts[0]} rows, {K} x {N} {dt}", flush=True)
    n, M = len(counts), sum(counts)
    dy = torch.zeros((M, K), dtype=TYPES[dt], device=cuda)
    dy[:, 0] = 1
    w = torch.ones((n, N, K), dtype=TYPES[dt], device=cuda)
    w[:, :, 0] = 2
    g = gates(N, dt, more=(1e-39, 1e-40))
    pre = torch.cat([g.expand(M, N), torch.full((M, N), UP, dtype=TYPES[dt], device=cuda)], dim=1)
    r = H.himuon_grouped_gated_mm_grad(dy, w, ends_of(counts), pre, act="relu", hidden=True)
    slope, act = (g > 0).double(), g.double().clamp(min=0)
    assert torch.equal(r.grad[:, :N], (2 * UP * slope).to(TYPES[dt]).expand(M, N)), "slope"
    assert torch.equal(r.h, (act * UP).to(TYPES[dt]).expand(M, N)), "h"
    normal = (g.abs() >= LEAST) | (g == 0)
    assert torch.equal(r.grad[:, N:][:, normal], (2 * act).to(TYPES[dt])[normal].expand(M, int(normal.sum()))), "du"
