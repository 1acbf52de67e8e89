"""AdamW steps on the GPU at the ends of fp32's range, against fp64.

g^2 and v lose bits below 2^-126 (fp32 is then 2^-149 apart).  v is a sum of two
products: its roundings are at most 6 2^-24 of v, and where they leave subnormal
numbers at most 2^-150 each: of g^2 (times 1 - beta2), of the square that 8-bit states
stand for (times beta2), of the two products and of the sum, less than 5 2^-150 in all.
So v is known to an interval and sqrt(v) to that interval's roots, widened by 4 2^-24.
A code is the value at or below sqrt(v) / scale + bits / 65536 of the gap there: within
one gap of either end.
"""
import math

import pytest
import torch

import tiled_newton_schulz_amd as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B = H.ADAMW_BLOCK
F8 = torch.float8_e4m3fn


def held(state):
    """(m, sqrt(v)) that the 8-bit states of one tensor stand for, in fp64; in 32 bits (m, v)."""
    if state.bits == 32:
        return state.m.double(), state.v.double()
    wide = lambda c, s: (c.float().double().view(-1, B) * s.double()[:, None]).view(-1)
    return wide(state.m, state.m_scale), wide(state.v, state.v_scale)


def spread(n, lo, hi, seed):
    """n fp32 numbers of either sign, sizes even over their logarithm, shuffled."""
    g = torch.Generator().manual_seed(seed)
    x = 10.0 ** torch.linspace(math.log10(lo), math.log10(hi), n, dtype=torch.float64)
    sign = torch.where(torch.rand(n, generator=g) < 0.5, -1.0, 1.0)
    return (x * sign)[torch.randperm(n, generator=g)].float().cuda()


def gap_of(x, unit):
    """The step between codes at x, of blocks' scales `unit`."""
    y = (x / unit).clamp(min=2.0 ** -6, max=448)
    return torch.exp2(torch.floor(torch.log2(y)) - 3) * unit


def tiny_step(w, g, state, step, eps):
    """One step in 8 or 32 bits against fp64."""
    n = w.numel()
    b1, b2, lr = 0.9, 0.999, 3e-3
    m0, r0 = (t[:n] for t in held(state))
    v0 = r0 if state.bits == 32 else r0 ** 2
    w0, g64 = w.double(), g.double()
    H.himuon_adamw_step([w], [g], state, lr=lr, step=step, betas=(b1, b2), eps=eps)
    torch.cuda.synchronize()
    m, v = b1 * m0 + (1 - b1) * g64, b2 * v0 + (1 - b2) * g64 ** 2
    far = 6 * U * v + 5 * 2.0 ** -150
    lo, hi = (v - far).clamp(min=0).sqrt() * (1 - 4 * U), (v + far).sqrt() * (1 + 4 * U)
    # the update, from either end
    root, rate = 1 / math.sqrt(1 - b2 ** step), lr / (1 - b1 ** step)
    dm = 5 * U * ((b1 * m0).abs() + ((1 - b1) * g64).abs()) + 2.0 ** -149
    most, least = rate * (m.abs() + dm) / (lo * root + eps), rate * (m.abs() - dm).clamp(min=0) / (hi * root + eps)
    up = (w0 - w.double()) * torch.sign(m)
    slack = 14 * U * most + 4 * U * (w0.abs() + most)
    assert torch.all(up <= most + slack), float((up - most - slack).max())
    assert torch.all(up >= least - slack), float((least - up - slack).max())
    m1, r1 = (t[:n] for t in held(state))
    if state.bits == 32:
        assert torch.all((m1 - m).abs() <= dm) and torch.all((r1 - v).abs() <= far)
        return
    blocks = -(-n // B)
    vs = state.v_scale[:blocks].double().repeat_interleave(B)[:n]
    top = lambda x: torch.cat([x, x.new_zeros(blocks * B - n)]).view(-1, B).amax(1).clamp(min=1e-30)
    got = state.v_scale[:blocks].double() * 448
    assert torch.all(got >= top(lo) * (1 - 4 * U)) and torch.all(got <= top(hi) * (1 + 4 * U))
    assert torch.all(r1 >= lo - gap_of(lo, vs) * 1.001) and torch.all(r1 <= torch.maximum(hi + gap_of(hi, vs) * 1.001, 2.0 ** -9 * vs))
    assert torch.all(r1[lo > 0] > 0), "sqrt(v) above 0 keeps a code above 0"
    assert torch.all(r1[(r0 == 0) & (g64 == 0)] == 0)
    ms = state.m_scale[:blocks].double().repeat_interleave(B)[:n]
    got = state.m_scale[:blocks].double() * 448
    assert torch.all((got - top(m.abs())).abs() <= 4 * U * top(m.abs()) + top(dm))
    assert torch.all((m1 - m).abs() <= gap_of(m.abs(), ms) * 1.001 + dm)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-8, 1e-30])
def test_tiny_gradients_from_zero(cuda, bits, eps):
    """Gradients from 1e-25 to 1 side by side, from zero states: second moments that are
    subnormal, or 0, beside ordinary ones; then blocks that hold tiny ones alone, odd
    lengths and zeros among them.  No element reaches its neighbours."""
    print(f"adamw, tiny gradients, {bits} bits, eps {eps}", flush=True)
    for lo, hi, n in ((1e-25, 1.0, 256), (1e-25, 1.0, 5003), (1e-22, 1e-17, 4096), (1e-21, 4e-18, 777)):
        w, g = spread(n, 1e-3, 1.0, 1), spread(n, lo, hi, 2)
        g[::7] = 0
        state = H.adamw_state([w], bits=bits)
        for step in (1, 2, 3):
            tiny_step(w, g, state, step, eps)
            g = g.roll(1)


@pytest.mark.parametrize("gdt", [torch.bfloat16, torch.float32])
def test_tiny_states(cuda, gdt):
    """8 bits: states that have decayed to where their squares are subnormal, with and
    without gradients."""
    n = 64 * B
    print("adamw, tiny 8-bit states", flush=True)
    for size in (0.0, 1e-19):
        w = spread(n, 1e-3, 1.0, 3)
        g = (spread(n, 1e-3, 1.0, 4) * size).to(gdt)
        state = H.adamw_state([w], bits=8)
        gen = torch.Generator().manual_seed(5)
        state.m.copy_((torch.randn(n, generator=gen) * 100).clamp(-448, 448).cuda().to(F8))
        state.v.copy_((torch.rand(n, generator=gen) * 447 + 1).cuda().to(F8))
        state.v_scale.copy_(torch.logspace(-25, -17, n // B))
        state.m_scale.copy_(torch.logspace(-25, -17, n // B))
        for step in (1000, 1001):
            tiny_step(w, g, state, step, 1e-8)


@pytest.mark.parametrize("bits", [32, 8])
def test_one_tiny_gradient_leaves_its_block(cuda, bits):
    """A block of ordinary gradients with one whose second moment is subnormal: all
    other elements end with the bits that they have beside a 0 there."""
    print(f"adamw, one tiny gradient, {bits} bits", flush=True)
    w, g = spread(B, 1e-2, 1.0, 6), spread(B, 1e-4, 1.0, 7)
    ends = []
    for value in (0.0, 1e-18):
        g[100] = value
        one, state = w.clone(), H.adamw_state([w], bits=bits)
        for step in (1, 2):
            H.himuon_adamw_step([one], [g], state, lr=1e-2, step=step)
        ends.append([one, state.m.float(), state.v.float()] + ([state.m_scale, state.v_scale] if bits == 8 else []))
    keep = torch.arange(B, device=cuda) != 100
    for a, b in zip(*ends):
        assert torch.equal(a, b) if a.numel() == 1 else torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("wdt,gdt", [("float32", "float32"), ("bfloat16", "bfloat16")])
def test_squares_past_the_range(cuda, wdt, gdt, bits):
    """Finite gradients whose squares are infinite in fp32: their elements are updated no
    more, neither then nor later, and stay finite; sqrt(v) and the weights of the
    elements beside them are what they are beside zeros."""
    print(f"adamw, squares past fp32's range, {bits} bits {gdt}", flush=True)
    n, at = 2 * B + 40, torch.tensor([3, 8, 200, 300, 2 * B + 39], device=cuda)
    w, g = spread(n, 1e-2, 1.0, 8).to(getattr(torch, wdt)), spread(n, 1e-4, 1e-2, 9).to(getattr(torch, gdt))
    rest = torch.ones(n, dtype=torch.bool, device=cuda)
    rest[at] = False
    ends = []
    for values in (0.0, torch.tensor([1e20, -1e30, 1e25, 3e38, -2e19], device=cuda).to(g.dtype)):
        one, state = w.clone(), H.adamw_state([w], bits=bits)
        first = g.clone()
        first[at] = values
        H.himuon_adamw_step([one], [first], state, lr=1e-2, step=1)
        ends.append((one.clone(), held(state)[1][:n].clone()))
        if isinstance(values, float):
            continue
        assert torch.equal(one[at], w[at])
        r = held(state)[1][at]
        assert torch.all(torch.isinf(r) if bits == 32 else torch.isnan(r))
        for step in (2, 3, 4):
            H.himuon_adamw_step([one], [g], state, lr=1e-2, step=step)
            assert torch.equal(one[at], w[at]) and torch.isfinite(one).all(), step
    for a, b in zip(*ends):
        assert torch.equal(a[rest], b[rest])


@pytest.mark.parametrize("size", [7e37, 9e37, 1.2e38, 3.3e38])
def test_largest_averages(cuda, size):
    """8 bits: averages m up to the end of fp32's range, where 1 / m is subnormal: codes and
    scale stand for them, within a gap."""
    print(f"adamw, m of {size}", flush=True)
    w, g = torch.zeros(B, device=cuda), spread(B, size * 1e-2, size, 10)
    state = H.adamw_state([w], bits=8)
    H.himuon_adamw_step([w], [g], state, lr=1e-2, step=1, betas=(0.0, 0.5))
    m, unit = held(state)[0], state.m_scale[0].double()
    most = g.double().abs().max()
    assert torch.all((unit * 448 - most).abs() <= 4 * U * most)
    assert torch.all((m - g.double()).abs() <= gap_of(g.double().abs(), unit) * 1.001 + 4 * U * most)
    assert torch.all(w == 0)
