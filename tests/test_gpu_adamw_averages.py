"""8-bit states of many steps on the GPU against the averages in fp64.

A step's codes are rounded up or down so that their mean is right, with a variance of
f (1 - f) gap^2, f the place between the two codes: at most |d| gap, d what the step
moves sqrt(v) by, and at most gap^2 / 4; a gap is at most an eighth of the value.  The
variances of sqrt(v) add to v; later steps shrink them with v.
"""
import pytest
import torch

import tiled_newton_schulz_amd as H
from test_gpu_adamw_range import F8, held

pytestmark = pytest.mark.gpu

N, STEPS, B2 = 65536, 300, 0.999


def started(seed):
    w = torch.zeros(N, device="cuda")
    state = H.adamw_state([w], bits=8)
    g = torch.Generator().manual_seed(seed)
    state.v.copy_((torch.rand(N, generator=g) * 200 + 40).cuda().to(F8))
    state.v_scale.fill_(1 / 448)
    return w, state


@pytest.mark.parametrize("target,most", [
    # all r = sqrt(v) move alike, and so do the scales: no rounding but at r's own last bits, 2^-22 gap a step
    (0.0, 1.0 + 300 * 2.0 ** -20),
    # a step moves r by at most 0.001 4 / (2 r) = 0.002 / r, so its variance is at most 0.00025 (0.0003 in
    # the first, that move r by up to a quarter): 0.09 in 300 steps, of an exact average of 1.12
    (2.0, 1.0 + 0.09 / 1.12),
])
def test_second_moments(cuda, target, most):
    """Equal gradients: the mean of v over 65536 elements stays within what the variances
    make of it.  (The mean's own spread: twice the root of the relative variance, 0.53 at
    most, over 256: five times that is 0.01.)"""
    print(f"adamw averages, gradients of {target}", flush=True)
    w, state = started(3)
    v0 = held(state)[1] ** 2
    g = torch.full((N,), target, device=cuda)
    for t in range(STEPS):
        H.himuon_adamw_step([w], [g], state, lr=0.0, step=1000 + t)
    want = v0 * B2 ** STEPS + (1 - B2 ** STEPS) * target ** 2
    ratio = float((held(state)[1] ** 2).mean() / want.mean())
    print(f"mean v: {ratio:.4f} of the exact average's, at most {most + 0.01:.3f}", flush=True)
    assert 0.99 <= ratio <= most + 0.01


def test_both_averages_of_noise(cuda):
    """Normal gradients.  A step moves r by 0.0005 |g^2 / v - 1| r, in the mean by at most
    0.001 r where v is around g's variance: a relative variance of 0.001 / 8 a step, 0.0375
    in 300 of them, by which v's mean may be above the exact average's; their spread over
    256 is 0.0015.  m's mean is right: a step's rounding is off by at most a gap, 1 / 14 of the
    block's largest, with a deviation of half of that; steps that fade by 0.9 add to
    sqrt(1 / (1 - 0.81)) = 2.3 of it, over 256 elements' root; five times that."""
    print("adamw averages, normal gradients", flush=True)
    w, state = started(4)
    state.v_scale.fill_(1 / 150)   # (v around 1)
    v = held(state)[1] ** 2
    m = torch.zeros(N, dtype=torch.float64, device=cuda)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for t in range(STEPS):
        g = torch.empty(N, device=cuda).normal_(generator=gen)
        H.himuon_adamw_step([w], [g], state, lr=0.0, step=2000 + t)
        m, v = 0.9 * m + 0.1 * g.double(), B2 * v + (1 - B2) * g.double() ** 2
    got_m, got_r = held(state)
    ratio = float((got_r ** 2).mean() / v.mean())
    far = float((got_m - m).mean().abs())
    bound = 5 / 256 * 2.3 * float(m.abs().max()) / 28
    print(f"mean v: {ratio:.4f} of the exact average's; mean m off by {far:.2e}, at most {bound:.2e}", flush=True)
    assert 0.99 <= ratio <= 1.0375 + 0.01
    assert far <= bound
    # element by element: a deviation of 2.3 / 28 of the largest m, below five of m's deviations: 0.41 of one
    assert float(torch.corrcoef(torch.stack([got_m, m]))[0, 1]) > (1 + 0.41 ** 2) ** -0.5
