"""AdamW steps on the GPU against fp64.

Tolerances, elementwise, with u = 2^-24: m is two products and a sum of rounded
coefficients, off by at most 4 u of both terms' sizes; v by 6 u v; sqrt(v) by 4 u; the
update by what m's error makes of it and 12 u; w by 3 u (|w| + |update|) and its one
rounding.  States in 8 bits are compared as code times scale: within one step between
codes of the value that the code stands for, and with no bias over many elements.
"""
import math

import pytest
import torch

import tiled_newton_schulz_amd as H

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
U = 2.0 ** -24
B = H.ADAMW_BLOCK
SETUP = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)


def randn(shape, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(TYPES[dt]).cuda()


def parts(state, flat):
    """Each tensor's part of a flat state, in its shape."""
    return [flat[s:s + math.prod(n)].view(n) for s, n in zip(state.starts, state.shapes)]


def held(state):
    """(m, sqrt(v)) or (m, v) of every tensor in fp64: what the states stand for."""
    if state.bits == 32:
        return [t.double() for t in parts(state, state.m)], [t.double() for t in parts(state, state.v)]
    wide = lambda c, s: (c.float().double().view(-1, B) * s.double()[:, None]).view(-1)
    return parts(state, wide(state.m, state.m_scale)), parts(state, wide(state.v, state.v_scale))


def fill(state, seed):
    """Random states, as after some steps."""
    g = torch.Generator().manual_seed(seed)
    n = state.m.numel()
    m, v = torch.randn(n, generator=g), torch.randn(n, generator=g).abs()
    if state.bits == 32:
        state.m.copy_(m * 0.01)
        state.v.copy_((v * 0.02) ** 2)
    else:
        state.m.copy_((m * 100).clamp(-448, 448).cuda().to(torch.float8_e4m3fn))
        state.v.copy_((v * 120).clamp(1, 448).cuda().to(torch.float8_e4m3fn))
        state.m_scale.copy_(torch.rand(n // B, generator=g) * 1e-4 + 1e-5)
        state.v_scale.copy_(torch.rand(n // B, generator=g) * 1e-4 + 1e-4)


def random_bits(n, step):
    """The 16 bits of each of n elements for sqrt(v), and for m."""
    low = 0xFFFFFFFF
    k = (step * 0x9AD24435 + 0xB3B07CC5) & low
    k = ((k ^ (k >> 16)) * 0xB06A350D) & low
    i = torch.arange(n, dtype=torch.int64)
    h = ((i >> 1) * 0xB890E049 + k) & low
    h = ((h ^ (h >> 15)) * 0xB4A1B41D) & low
    h = ((h ^ (h >> 13)) * 0xF5BBB081) & low
    u = torch.where((i & 1) == 0, h & 0xFFFF, h >> 16)
    return u.cuda(), (((u << 8) | (u >> 8)) & 0xFFFF).cuda()


def check_codes(code, scale, x, off, step, which):
    """Flat codes and scales of a tensor whose state should be x, known to `off`."""
    n = x.numel()
    full = -(-n // B) * B
    pad = lambda t: torch.cat([t.reshape(-1), torch.zeros(full - n, dtype=t.dtype, device=t.device)]).view(-1, B)
    most = pad(x.abs()).amax(1).clamp(min=1e-30)
    slack = pad(off).amax(1) + 4 * U * most
    assert torch.all((scale.double() * 448 - most).abs() <= slack)
    got = (pad(code.float().double()) * scale.double()[:, None]).reshape(-1)[:n].view(x.shape)
    unit = scale.double().repeat_interleave(B)[:n].view(x.shape)
    y = (x.abs() / unit).clamp(max=448)
    gap = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3) * unit
    far = (got - x).abs()
    assert torch.all(far <= gap * 1.001 + off)
    assert torch.all((got == 0) | (torch.sign(got) == torch.sign(x)))
    # the code is the one at or below y + bits / 65536 of the gap, but where y is as near to a
    # border as its own error
    q = torch.floor(y / (gap / unit) + random_bits(n, step)[which].view(x.shape) / 65536) * gap
    if which == 0:
        q = torch.where((x > 0) & (q == 0), 2.0 ** -9 * unit, q)
        assert torch.all((got > 0) == (x > 0))
    odd = (got.abs() - q).abs() > 1e-3 * gap
    assert odd.sum() <= 2 + 1e-3 * n, float(odd.double().mean())


def check_step(ws, gs, state, step, scale=None, **more):
    setup = {**SETUP, **more}
    w0, (m0, r0) = [w.double() for w in ws], held(state)
    gdt = [g.double() for g in gs]
    H.himuon_adamw_step(ws, gs, state, step=step, grad_scale=scale, **setup)
    torch.cuda.synchronize()
    (b1, b2), lr = setup["betas"], setup["lr"]
    m1, r1 = held(state)
    gmul = 1.0 if scale is None else float(scale)
    for i, w in enumerate(ws):
        g = gdt[i] * gmul
        v0 = r0[i] if state.bits == 32 else r0[i] ** 2
        m, v = b1 * m0[i] + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
        dm = 5 * U * ((b1 * m0[i]).abs() + ((1 - b1) * g).abs())
        root = (v / (1 - b2 ** step)).sqrt() + setup["eps"]
        rate = lr / (1 - b1 ** step)
        up = rate * m / root
        want = w0[i] * (1 - lr * setup["weight_decay"]) - up
        dt = "bf16" if w.dtype == torch.bfloat16 else "fp32"
        off = rate * dm / root + 14 * U * up.abs() + 4 * U * (w0[i].abs() + up.abs())
        d = (w.double() - want).abs()
        assert torch.all(d <= off + HALF[dt] * (want.abs() + off) + 1e-37), float(d.max())
        if state.bits == 32:
            assert torch.all((m1[i] - m).abs() <= dm + 1e-37) and torch.all((r1[i] - v).abs() <= 8 * U * v + 1e-37)
            continue
        n, s = w.numel(), state.starts[i]
        blocks = slice(s // B, s // B + -(-n // B))
        check_codes(state.m[s:s + n], state.m_scale[blocks], m.reshape(-1), dm.reshape(-1), step, 1)
        check_codes(state.v[s:s + n], state.v_scale[blocks], v.sqrt().reshape(-1), 6 * U * v.sqrt().reshape(-1), step, 0)


SHAPES = [(1,), (7,), (8,), (255,), (256,), (257,), (4095,), (4096,), (4097,), (3, 5, 7), (64, 65), (), (20000,), (1, 1)]
KINDS = [("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "fp32")]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("wdt,gdt", KINDS)
def test_shapes(cuda, wdt, gdt, bits):
    print(f"adamw {wdt} weights, {gdt} gradients, {bits} bits", flush=True)
    ws = [randn(s, wdt, i, 0.1) for i, s in enumerate(SHAPES)]
    gs = [randn(s, gdt, 100 + i, 0.02) for i, s in enumerate(SHAPES)]
    state = H.adamw_state(ws, bits=bits)
    check_step(ws, gs, state, 1)          # from zero states
    check_step(ws, gs, state, 2, scale=torch.full((1,), 0.37, device=cuda))
    fill(state, 7)
    check_step(ws, gs, state, 1000, weight_decay=0.0, eps=1e-3, betas=(0.0, 0.95))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("wdt,gdt", KINDS)
def test_rows_with_gaps(cuda, wdt, gdt, bits):
    """Column blocks of wider tensors: their other columns stay; widths of whole
    chunks and odd ones, weights or gradients without gaps beside the others."""
    print(f"adamw rows with gaps {wdt} {gdt} {bits}", flush=True)
    shapes, ws, gs, rooms = [(40, 24), (33, 7), (5, 1), (1, 300), (70, 129), (9, 4096)], [], [], []
    for i, (r, c) in enumerate(shapes):
        t = torch.full((r, c + 9), 7.0, dtype=TYPES[wdt], device=cuda)
        w = t[:, 3:3 + c]
        w.copy_(randn((r, c), wdt, i, 0.1))
        rooms.append((t, w))
        ws.append(w if i % 3 else w.contiguous())
        g = torch.full((r, c + 4), float("nan"), dtype=TYPES[gdt], device=cuda)
        g[:, 1:1 + c] = randn((r, c), gdt, 50 + i, 0.02)
        gs.append(g[:, 1:1 + c] if i % 2 else g[:, 1:1 + c].contiguous())
    state = H.adamw_state(ws, bits=bits)
    fill(state, 8)
    check_step(ws, gs, state, 10)
    for (t, w) in rooms:
        assert torch.all(t[:, :3] == 7.0) and torch.all(t[:, 3 + w.shape[1]:] == 7.0)


@pytest.mark.parametrize("bits", [32, 8])
def test_places_off_any_grid(cuda, bits):
    """Tensors packed one after the other, beginning anywhere; what lies before and
    behind them stays, states included."""
    print(f"adamw packed tensors {bits}", flush=True)
    sizes, at, ws, gs = [3, 700, 1, 5001, 256], 1, [], []
    flat, grads = torch.full((6001,), 7.0, dtype=torch.bfloat16, device=cuda), randn((6001,), "bf16", 2, 0.02)
    for n in sizes:
        ws.append(flat[at:at + n])
        gs.append(grads[at:at + n])
        at += n
    for i, w in enumerate(ws):
        w.copy_(randn(w.shape, "bf16", i, 0.1))
    state = H.adamw_state(ws, bits=bits)
    fill(state, 9)
    behind = [torch.cat([f[s + n:s + -(-n // B) * B].float() for s, n in zip(state.starts, sizes)]) for f in (state.m, state.v)]
    check_step(ws, gs, state, 3)
    assert flat[0] == 7.0 and torch.all(flat[at:] == 7.0)
    after = [torch.cat([f[s + n:s + -(-n // B) * B].float() for s, n in zip(state.starts, sizes)]) for f in (state.m, state.v)]
    assert all(torch.equal(a, b) for a, b in zip(behind, after))


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(cuda, bits):
    """More than one launch's tensors; described once; the same bits again."""
    print(f"adamw 600 tensors {bits}", flush=True)
    shapes = [((i * 37) % 500 + 1,) if i % 50 else (9001,) for i in range(600)]
    ws = [randn(s, "fp32", i, 0.1) for i, s in enumerate(shapes)]
    gs = [randn(s, "fp32", 1000 + i, 0.02) for i, s in enumerate(shapes)]
    copies = [w.clone() for w in ws]
    one, two = H.adamw_state(ws, bits=bits), H.adamw_state(ws, bits=bits)
    check_step(ws, gs, one, 5)
    W, G = H.tensors(copies), H.tensors(gs)
    H.himuon_adamw_step(W, G, two, step=5, **SETUP)
    assert all(torch.equal(a, b) for a, b in zip(ws, copies))
    assert torch.equal(one.m.view(torch.uint8), two.m.view(torch.uint8)) and torch.equal(one.v.view(torch.uint8), two.v.view(torch.uint8))
    copies[3].data = copies[3].clone()
    with pytest.raises(ValueError):
        H.himuon_adamw_step(W, G, two, step=6, **SETUP)


def test_large_tensor(cuda):
    """More than 2^31 bytes of weights and more units than workgroups; the last
    elements too."""
    n = (1 << 30) + 12345
    print(f"adamw {n} elements", flush=True)
    w, g = torch.full((n,), 0.5, dtype=torch.bfloat16, device=cuda), torch.full((n,), 0.25, dtype=torch.bfloat16, device=cuda)
    state = H.adamw_state([w], bits=8)
    H.himuon_adamw_step([w], [g], state, lr=0.125, step=1, betas=(0.5, 0.5), eps=1e-6)
    # m / (1 - beta) = g and v / (1 - beta) = g^2 : w - lr g / (g + eps)
    assert torch.all(w == 0.375)
    assert torch.all(state.m_scale == state.m_scale[0]) and torch.all(state.m.view(torch.uint8)[:n] == 126)


@pytest.mark.parametrize("bits", [32, 8])
def test_not_finite(cuda, bits):
    """NaN and infinity stay in their elements; a block of zeros stays zero."""
    print(f"adamw not finite {bits}", flush=True)
    w, g = randn((3, 256), "fp32", 1), randn((3, 256), "fp32", 2, 0.01)
    g[0, 5], g[0, 6], g[0, 7] = float("nan"), float("inf"), float("-inf")
    g[2] = 0
    state = H.adamw_state([w], bits=bits)
    before = w.clone()
    H.himuon_adamw_step([w], [g], state, step=1, **{**SETUP, "weight_decay": 0.0})
    bad = torch.zeros((3, 256), dtype=torch.bool, device=cuda)
    bad[0, 5] = bad[0, 6] = bad[0, 7] = True
    assert torch.equal(torch.isfinite(w), ~bad) and torch.equal(w[2], before[2])
    m, v = (t[0] for t in held(state))
    assert torch.equal(torch.isfinite(m), ~bad) and torch.equal(torch.isfinite(v), ~bad)
    assert torch.all(m[2] == 0) and torch.all(v[2] == 0)
    good = w.clone()
    H.himuon_adamw_step([w], [g.nan_to_num(0, 0, 0)], state, step=2, **SETUP)
    assert torch.equal(torch.isfinite(w), ~bad) and torch.equal(torch.isfinite(good), ~bad)


def test_slow_averages_move(cuda):
    """8 bits: 300 steps without a gradient at beta2 = 0.999 take sqrt(v) down by
    0.999^150, though each step is far below half a step between codes, and steps
    towards a larger second moment take it up.  Bounds: a step adds an error of at
    most one gap (2^-3 of the value) whose mean is 0, 300 of them sqrt(300) / 8 of an
    element at most and 1 / sqrt(65536) of that in the mean over the elements."""
    n = 65536
    print("adamw 8 bits, slow averages", flush=True)
    w, g = torch.zeros(n, device=cuda), torch.zeros(n, device=cuda)
    for target, start in ((0.0, 1.0), (2.0, 1.0)):
        state = H.adamw_state([w], bits=8)
        gen = torch.Generator().manual_seed(3)
        state.v.copy_((torch.rand(n, generator=gen) * 200 + 40).cuda().to(torch.float8_e4m3fn))
        state.v_scale.fill_(start / 448)
        v0 = held(state)[1][0] ** 2
        g.fill_(target)
        for t in range(300):
            H.himuon_adamw_step([w], [g], state, lr=0.0, step=1000 + t)
        v = held(state)[1][0] ** 2
        k = 0.999 ** 300
        want = v0 * k + (1 - k) * target ** 2
        # (the squares of the errors add to v: each step's error has at most a quarter gap^2 of variance,
        # (2^-3)^2 / 4 of r^2, which fades with v: at most 300 (2^-8) of v)
        mean, most = float(v.mean() / want.mean()), 1 + 300 * 2.0 ** -8
        assert 0.95 <= mean <= most, mean
        r, rw = held(state)[1][0].mean(), want.sqrt().mean()
        print(f"target {target}: mean v {mean:.3f}, mean sqrt(v) {float(r / rw):.3f} of the exact average's", flush=True)


@pytest.mark.parametrize("bits", [32, 8])
def test_streams_and_graphs(cuda, bits):
    print(f"adamw captured {bits}", flush=True)
    shapes = [(300, 40), (17,), (5000,)]
    ws, gs = [randn(s, "bf16", i, 0.1) for i, s in enumerate(shapes)], [randn(s, "bf16", 9 + i, 0.02) for i, s in enumerate(shapes)]
    scale = torch.ones(1, device=cuda)
    copies = [w.clone() for w in ws]
    a, b = H.adamw_state(ws, bits=bits), H.adamw_state(ws, bits=bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    H.himuon_adamw_step(copies, gs, b, step=3, grad_scale=scale, **SETUP)
    H.himuon_adamw_step(ws, gs, a, step=3, grad_scale=scale, stream=side, **SETUP)
    torch.cuda.current_stream().wait_stream(side)
    same = lambda: (all(torch.equal(p, q) for p, q in zip(ws, copies)) and torch.equal(a.m.view(torch.uint8), b.m.view(torch.uint8))
                    and torch.equal(a.v.view(torch.uint8), b.v.view(torch.uint8)))
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H.himuon_adamw_step(ws, gs, a, step=4, grad_scale=scale, **SETUP)
    for k in range(3):
        for i, g in enumerate(gs):
            g.copy_(randn(g.shape, "bf16", 50 + 10 * k + i, 0.02))
        scale.fill_(1.0 / (k + 1))
        H.himuon_adamw_step(copies, gs, b, step=4, grad_scale=scale, **SETUP)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(), k


def test_refusals_in_python(cuda):
    w, g = [torch.zeros(8, 8, device=cuda)], [torch.zeros(8, 8, device=cuda)]
    state = H.adamw_state(w)
    step = lambda *a, **k: H.himuon_adamw_step(*a, lr=0.1, **{"step": 1, **k})
    for bad in ([torch.zeros(64, device=cuda)], [torch.zeros(8, 8)], [torch.zeros(8, 8, device=cuda).t()[:, :4]], []):
        with pytest.raises((ValueError, TypeError)):
            step(w, bad, state)
    with pytest.raises(ValueError):
        step([torch.zeros(8, 9, device=cuda)], [torch.zeros(8, 9, device=cuda)], state)
    with pytest.raises(ValueError):   # a transposed view: its rows have no unit stride
        step([torch.zeros(8, 8, device=cuda)[:, :7].t()], [torch.zeros(7, 8, device=cuda)], H.adamw_state([torch.zeros(7, 8, device=cuda)]))
    with pytest.raises(TypeError):
        step([torch.zeros(8, 8, device=cuda).half()], g, state)
    with pytest.raises(TypeError):
        step(w, g, state, grad_scale=torch.ones(1, device=cuda).double())
    with pytest.raises(ValueError):
        step(w, g, state, grad_scale=torch.ones(1))
    with pytest.raises(H.HimuonError):
        step(w, w, state)   # gradients in place of the weights
    with pytest.raises(H.HimuonError):
        step(w, g, state, step=0)
    with pytest.raises(ValueError):
        H.adamw_state(w, bits=16)
    step([], [], H.adamw_state([]))
