"""The gated experts' block on the GPU against fp64.

Tolerances, elementwise.  The projections and the down product's gradient are
accumulated in fp32 over K terms in some order: off by at most E = 2 K 2^-24
sum |a b| (as for the experts' products).  The activations' slopes are below 1.2, so
that much of E reaches act(g) at most.  act(g) = g s(g) itself is off by

    rel(g) = (16 + 2 |g| + g^2 + 0.1 |g|^3) 2^-22

of its size: a dozen operations of at most 2^-23 each (the hardware's exponential and
reciprocal, or the library's erfc with at most 16 units), and an exponent z with
|z| <= 1.6 |g| + 0.08 |g|^3 (erfc: g^2 / 2), whose own roundings, 4 2^-24 of it,
multiply the result by as much.  The slope s + act (1 - s) p' has the same relative
error in both terms, and 1 - s another 2^-24.  Each result is rounded once, by at most
half a step: eps / 2 of its size.
"""
import math

import pytest
import torch

import tiled_newton_schulz_amd as H

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
ACTS = list(H.ACTIVATIONS)


def randn(shape, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(TYPES[dt]).cuda()


def ends_of(counts):
    return torch.tensor(counts).cumsum(0).to(torch.int32).cuda()


def share(act, g):
    """s(g), act(g), act'(g) and |p'| in fp64, p the argument of a sigmoid."""
    one = torch.ones_like(g)
    if act == "relu":
        s = (g > 0).double()
        return s, torch.relu(g), s, 0 * g
    if act == "gelu":
        s = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return s, g * s, s + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi), one
    k0, k1 = (1.0, 0.0) if act == "silu" else (2 * math.sqrt(2 / math.pi), 2 * math.sqrt(2 / math.pi) * 0.044715)
    s, p = torch.sigmoid(k0 * g + k1 * g ** 3), k0 + 3 * k1 * g * g
    return s, g * s, s + g * s * (1 - s) * p, p


def rel(g):
    a = g.abs()
    return (16 + 2 * a + a * a + 0.1 * a ** 3) * 2.0 ** -22


def accumulated(a, b):
    a, b = a.double(), b.double().contiguous()
    return a @ b, 2 * a.shape[1] * 2.0 ** -24 * (a.abs() @ b.abs())


def close(got, want, off, dt, what):
    bound = off + HALF[dt] * (want.abs() + off) + 1e-30
    d = (got.double() - want).abs()
    assert torch.all(d <= bound), f"{what}: {float((d - bound).max())} over, of {float(want.abs().max())}"


def check_forward(x, w, counts, act, dt, keep=True, **more):
    r = H.himuon_grouped_gated_mm(x, w, ends_of(counts), act=act, keep=keep, **more)
    torch.cuda.synchronize()
    N, at = w[0].shape[1] // 2, 0
    for e, c in enumerate(counts):
        if c:
            pre, off = accumulated(x[at:at + c], w[e])
            g, u, eg, eu = pre[:, :N], pre[:, N:], off[:, :N], off[:, N:]
            _, a, _, _ = share(act, g)
            da = 1.2 * eg + (a.abs() + 1.2 * eg) * rel(g)
            close(r.h[at:at + c], a * u, u.abs() * da + a.abs() * eu + da * eu + 2.0 ** -23 * (a * u).abs(), dt, "h")
            if keep is not False:
                close(r.pre[at:at + c], pre, off, dt, "pre")
        at += c
    assert torch.all(r.h[at:] == 0) and (keep is False or torch.all(r.pre[at:] == 0))
    return r


def check_grad(dy, w, counts, pre, act, dt, hidden=True, **more):
    kept = pre.double()   # (out may be pre)
    r = H.himuon_grouped_gated_mm_grad(dy, w, ends_of(counts), pre, act=act, hidden=hidden, **more)
    torch.cuda.synchronize()
    N, at = w[0].shape[0], 0
    for e, c in enumerate(counts):
        if c:
            dh, off = accumulated(dy[at:at + c], w[e].t())
            g, u = kept[at:at + c, :N], kept[at:at + c, N:]
            s, a, slope, p = share(act, g)
            ds = rel(g) * (s + (a * (1 - s) * p).abs() + (slope - s).abs()) + 2.0 ** -23 * (a * p).abs()
            k = 2.0 ** -22
            close(r.grad[at:at + c, :N], dh * u * slope,
                  (u * slope).abs() * off + (dh.abs() + off) * u.abs() * ds + k * (dh * u * slope).abs(), dt, "gate")
            close(r.grad[at:at + c, N:], dh * a, a.abs() * off + (dh.abs() + off) * a.abs() * rel(g) + k * (dh * a).abs(),
                  dt, "up")
            if hidden is not False:
                close(r.h[at:at + c], a * u, (a * u).abs() * (rel(g) + k), dt, "h")
        at += c
    assert torch.all(r.grad[at:] == 0) and (hidden is False or torch.all(r.h[at:] == 0))
    return r


# rows of each expert, K, N
CASES = [
    ([1], 1, 1),
    ([5], 8, 8),
    ([0, 3, 0], 16, 40),
    ([7, 0, 1, 64, 65], 24, 136),
    ([130, 1, 0, 63], 100, 96),
    ([256, 257, 31], 192, 264),
    ([3, 300, 0, 17], 515, 261),
    ([1, 2, 0, 1, 1, 0, 3, 1], 512, 256),
    ([600, 20], 1031, 72),
    ([33, 90, 200], 320, 704),
    ([2, 0, 5, 16], 40, 7),
]


def weights(n, K, N2, stored, dt, seed):
    if stored == "kn":
        return randn((n, K, N2), dt, seed, 1.5 / math.sqrt(K))
    return randn((n, N2, K), dt, seed, 1.5 / math.sqrt(K)).transpose(1, 2)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("stored", ["kn", "nk"])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_forward(cuda, counts, K, N, stored, dt):
    act = ACTS[(K + N) % 4]
    print(f"gated {counts} {K}x{N} {stored} {dt} {act}", flush=True)
    x = randn((sum(counts) + 3, K), dt, 1)
    check_forward(x, weights(len(counts), K, 2 * N, stored, dt, 2), counts, act, dt, keep=N % 3 != 0)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("stored", ["kn", "nk"])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_backward(cuda, counts, K, N, stored, dt):
    act = ACTS[(K + N + 1) % 4]
    print(f"gated gradient {counts} {K}x{N} {stored} {dt} {act}", flush=True)
    M = sum(counts) + 3
    pre = randn((M, 2 * N), dt, 4, 1.5)
    pre[-3:] = float("nan")   # rows of no expert: zeros whatever is there
    check_grad(randn((M, K), dt, 3), weights(len(counts), N, K, stored, dt, 5), counts, pre, act, dt, hidden=N % 3 != 0)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("act", ACTS)
def test_activations(cuda, act, dt):
    """Gates from far below to far above 0, exact zeros among them."""
    counts, K, N = [40, 90], 64, 96
    print(f"gated {act} {dt}", flush=True)
    x, w = randn((130, K), dt, 6), weights(2, K, 2 * N, "kn", dt, 7)
    x[::7] *= 8
    x[5] = 0
    r = check_forward(x, w, counts, act, dt)
    check_grad(randn((130, K), dt, 8), weights(2, N, K, "kn", dt, 9), counts, r.pre, act, dt)


@pytest.mark.parametrize("act", ACTS)
def test_infinite_gates(cuda, act):
    """A gate of -inf gives 0 (its slope too), one of +inf passes the gradient on;
    NaN stays in its element."""
    N = 8
    pre = torch.ones((4, 2 * N), device=cuda)
    pre[0, :N], pre[1, :N], pre[2, 3] = float("-inf"), float("inf"), float("nan")
    dy, w = torch.ones((4, 2), device=cuda), torch.ones((1, N, 2), device=cuda)
    print(f"gated gradient at infinite gates {act}", flush=True)
    r = H.himuon_grouped_gated_mm_grad(dy, w, ends_of([4]), pre, act=act, hidden=True)
    assert torch.all(r.grad[0] == 0) and torch.all(r.h[0] == 0)
    assert torch.all(torch.isinf(r.h[1])) and torch.all(torch.isinf(r.grad[1, N:])) and torch.all(r.grad[1, :N] == 2)
    assert torch.isnan(r.h[2]).sum() == 1 and torch.isnan(r.grad[2]).sum() in (1, 2)
    assert not torch.any(torch.isnan(r.grad[3]))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 1), (24, 8)])
def test_strides_and_padding(cuda, dt, pad, shift):
    """Column blocks of wider tensors whose other columns hold NaN, results into the
    middle of wider tensors whose other columns stay; weights as lists."""
    counts, K, N = [70, 0, 130, 9], 144, 88
    M, n = sum(counts), len(counts)

    def wide(rows, cols, seed, scale=1.0):
        t = torch.full((rows, cols + pad + shift), float("nan"), dtype=TYPES[dt], device=cuda)
        v = t[:, shift:shift + cols]
        v.copy_(randn((rows, cols), dt, seed, scale))
        return v

    def room(cols):
        t = torch.full((M, cols + pad + shift), 7.0, dtype=TYPES[dt], device=cuda)
        return t, t[:, shift:shift + cols]

    print(f"gated strides pad {pad} shift {shift} {dt}", flush=True)
    for tr in (False, True):
        w_in = [wide(2 * N, K, 10 + e, 0.1).t() if tr else wide(K, 2 * N, 10 + e, 0.1) for e in range(n)]
        w_out = [wide(K, N, 20 + e, 0.1).t() if tr else wide(N, K, 20 + e, 0.1) for e in range(n)]
        rooms = [room(N), room(2 * N), room(2 * N), room(N)]
        r = check_forward(wide(M, K, 5), w_in, counts, "silu", dt, keep=rooms[1][1], out=rooms[0][1])
        check_grad(wide(M, K, 6), w_out, counts, r.pre, "silu", dt, hidden=rooms[3][1], out=rooms[2][1])
        for t, v in rooms:
            end = shift + v.shape[1]
            assert torch.all(t[:, :shift] == 7.0) and torch.all(t[:, end:] == 7.0)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("counts,K,N", [([300, 0, 40], 136, 200), ([9, 30], 77, 33)])
def test_gradient_in_place(cuda, counts, K, N, dt):
    M = sum(counts)
    print(f"gated gradient in place {counts} {K}x{N} {dt}", flush=True)
    dy, w, pre = randn((M, K), dt, 1), weights(len(counts), N, K, "kn", dt, 2), randn((M, 2 * N), dt, 3)
    want = check_grad(dy, w, counts, pre, "silu", dt)
    got = check_grad(dy, w, counts, pre, "silu", dt, out=pre)
    assert got.grad.data_ptr() == pre.data_ptr() and torch.equal(got.grad, want.grad) and torch.equal(got.h, want.h)


def test_many_experts_and_no_rows(cuda):
    n, K, N = 300, 24, 40   # two launches
    counts = [(i * 7) % 4 for i in range(n)]
    print("gated, 300 experts", flush=True)
    x, w = randn((sum(counts) + 5, K), "bf16", 1), weights(n, K, 2 * N, "kn", "bf16", 2)
    r = check_forward(x, w, counts, "silu", "bf16")
    check_grad(randn((sum(counts) + 5, 16), "bf16", 3), weights(n, N, 16, "nk", "bf16", 4), counts, r.pre, "silu", "bf16")
    r = H.himuon_grouped_gated_mm(x[:0], w, torch.zeros(n, dtype=torch.int32, device=cuda), keep=True)
    assert r.h.shape == (0, N) and r.pre.shape == (0, 2 * N)
    r = check_forward(x, w, [0] * n, "silu", "bf16")


def ragged(n, most, seed, none=0.1):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(1, most + 1, (n,), generator=g)
    return c.masked_fill(torch.rand(n, generator=g) < none, 0).tolist()


# tiles enough for every kernel: experts, most rows of one, K, N
TILED = [(64, 300, 200, 264), (20, 700, 1032, 392), (300, 40, 264, 72), (64, 130, 264, 320), (40, 16, 520, 200), (9, 2100, 72, 520),
         (64, 3, 1096, 136), (64, 4, 200, 328), (5, 30, 456, 4104), (70, 20, 40, 264)]


@pytest.mark.parametrize("stored", ["kn", "nk"])
@pytest.mark.parametrize("n,most,K,N", TILED)
def test_many_tiles(cuda, n, most, K, N, stored):
    counts = ragged(n, most, n + most)
    print(f"gated {n} experts of {K}x{N}, up to {most} rows, {stored}", flush=True)
    M = sum(counts) + 7
    x = randn((M, K), "bf16", 1)
    r = check_forward(x, weights(n, K, 2 * N, stored, "bf16", 2), counts, "silu", "bf16")
    h = H.himuon_grouped_gated_mm(x, weights(n, K, 2 * N, stored, "bf16", 2), ends_of(counts)).h
    assert torch.equal(h, r.h)   # without [g | u]
    r.pre[-7:] = float("nan")
    check_grad(randn((M, K), "bf16", 3), weights(n, N, K, stored, "bf16", 4), counts, r.pre, "gelu", "bf16")


def test_streams_graphs_and_bits(cuda):
    """The same bits on another stream and from every replay of a captured call,
    with eager work and changed inputs in between."""
    for counts, K, N in (([200, 0, 300, 60], 264, 136), ([2, 1, 0, 3], 264, 136), ([40, 30], 65, 33)):
        print(f"gated block captured {counts}", flush=True)
        M, n = sum(counts), len(counts)
        x, w_in, w_out = randn((M, K), "bf16", 1), weights(n, K, 2 * N, "kn", "bf16", 2), weights(n, N, K, "kn", "bf16", 3)
        dy, ends = randn((M, K), "bf16", 4), ends_of(counts)

        def block():
            r = H.himuon_grouped_gated_mm(x, w_in, ends, keep=True)
            g = H.himuon_grouped_gated_mm_grad(dy, w_out, ends, r.pre, hidden=True)
            return r.h, r.pre, g.grad, g.h

        want = block()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = block()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = block()
        for k in range(3):
            x.copy_(randn((M, K), "bf16", 10 + k))
            want = block()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_block_gradients_against_differences(cuda):
    """fp32: the whole block's gradients (through the experts' products too) against
    central differences of sum(y c) in fp64."""
    counts, K, N = [5, 0, 9], 12, 10
    n, M = len(counts), sum(counts)
    print("gated block against differences", flush=True)
    for act in ("silu", "gelu", "gelu_tanh"):
        x, w_in, w_out = randn((M, K), "fp32", 1), randn((n, K, 2 * N), "fp32", 2, 0.3), randn((n, N, K), "fp32", 3, 0.3)
        c, ends = randn((M, K), "fp32", 4), ends_of(counts)
        r = H.himuon_grouped_gated_mm(x, w_in, ends, act=act, keep=True)
        g = H.himuon_grouped_gated_mm_grad(c, w_out, ends, r.pre, act=act, hidden=True)
        got = [H.himuon_grouped_mm(g.grad, w_in.transpose(1, 2), ends), H.himuon_grouped_wgrad(x, g.grad, ends),
               H.himuon_grouped_wgrad(g.h, c, ends)]

        def value(x, w_in, w_out):
            total, at = 0.0, 0
            for e, k in enumerate(counts):
                pre = x[at:at + k] @ w_in[e]
                total = total + (((share(act, pre[:, :N])[1] * pre[:, N:]) @ w_out[e]) * c64[at:at + k]).sum()
                at += k
            return total

        c64, args = c.double(), [x.double(), w_in.double(), w_out.double()]
        gen = torch.Generator().manual_seed(5)
        for i, t in enumerate(args):
            for _ in range(6):
                v = torch.randn(t.shape, generator=gen).double().cuda()
                h = 1e-5
                up, down = ([a + s * h * v if j == i else a for j, a in enumerate(args)] for s in (1, -1))
                slope = (value(*up) - value(*down)) / (2 * h)
                # differences: h^2 / 6 of a third derivative below 10^4 here; the gradient: each of a
                # chain of three fp32 products of at most 20 terms is off by 2^-18 of its terms' sum
                size = (got[i].double().abs() * v.abs()).sum()
                assert abs((got[i].double() * v).sum() - slope) <= 1e-6 + 2.0 ** -14 * size, (act, i)


@pytest.mark.parametrize("dt,K,N", [("bf16", 512, 4096), ("bf16", 511, 4097), ("fp32", 256, 2049)])
def test_operands_past_2_to_the_31_elements(cuda, dt, K, N):
    """[G | U] of more than 2^31 elements, and weights of as many bytes: the first and
    the last rows of the first and the last experts."""
    M = (1 << 31) // (2 * N) + 700
    n = max(3, (1 << 31) // (2 * K * N) // (2 if dt == "fp32" else 1))
    print(f"gated {M} rows, {n} experts of {K} x {2 * N} {dt}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((M, K), device=cuda, generator=gen).to(TYPES[dt])
    w = torch.empty((n, K, 2 * N), dtype=TYPES[dt], device=cuda).normal_(generator=gen).mul_(K ** -0.5)
    counts = [M // n] * (n - 1) + [M - (n - 1) * (M // n)]
    r = H.himuon_grouped_gated_mm(x, w, ends_of(counts), keep=True)
    starts = [sum(counts[:e]) for e in range(n)]
    picks = [(0, 0), (0, counts[0] - 1), (n - 1, starts[-1]), (n - 1, M - 1)]
    for e, row in picks:
        pre, off = accumulated(x[row:row + 1], w[e])
        g, u, eg, eu = pre[:, :N], pre[:, N:], off[:, :N], off[:, N:]
        _, a, _, _ = share("silu", g)
        da = 1.2 * eg + (a.abs() + 1.2 * eg) * rel(g)
        close(r.h[row:row + 1], a * u, u.abs() * da + a.abs() * eu + da * eu + 2.0 ** -23 * (a * u).abs(), dt, "h")
        close(r.pre[row:row + 1], pre, off, dt, "pre")
    del w, r
    torch.cuda.empty_cache()
    pre = torch.empty((M, 2 * N), dtype=TYPES[dt], device=cuda).normal_(generator=gen)
    keep = {row: pre[row:row + 1].double() for _, row in picks}
    w = torch.empty((n, N, K), dtype=TYPES[dt], device=cuda).normal_(generator=gen).mul_(N ** -0.5)
    r = H.himuon_grouped_gated_mm_grad(x, w, ends_of(counts), pre, out=pre)
    for e, row in picks:
        dh, off = accumulated(x[row:row + 1], w[e].t())
        g, u = keep[row][:, :N], keep[row][:, N:]
        s, a, slope, p = share("silu", g)
        ds = rel(g) * (s + (a * (1 - s) * p).abs() + (slope - s).abs()) + 2.0 ** -23 * (a * p).abs()
        close(r.grad[row:row + 1, :N], dh * u * slope,
              (u * slope).abs() * off + (dh.abs() + off) * u.abs() * ds + 2.0 ** -22 * (dh * u * slope).abs(), dt, "gate")
        close(r.grad[row:row + 1, N:], dh * a,
              a.abs() * off + (dh.abs() + off) * a.abs() * rel(g) + 2.0 ** -22 * (dh * a).abs(), dt, "up")


def test_two_streams_at_once(cuda):
    """Two blocks on two streams, each filling the chip, and their gradients."""
    print("gated blocks on two streams", flush=True)
    counts, K, N = ragged(40, 500, 5), 520, 328
    M, n = sum(counts), len(counts)
    ends, sides, sets = ends_of(counts), [torch.cuda.Stream(), torch.cuda.Stream()], []
    for k in range(2):
        x, dy = randn((M, K), "bf16", 10 * k), randn((M, K), "bf16", 10 * k + 1)
        sets.append((x, weights(n, K, 2 * N, "kn", "bf16", 10 * k + 2), dy, weights(n, N, K, "kn", "bf16", 10 * k + 3)))

    def block(x, w, dy, wd):
        r = H.himuon_grouped_gated_mm(x, w, ends, keep=True)
        return (*r, *H.himuon_grouped_gated_mm_grad(dy, wd, ends, r.pre, hidden=True))

    want = [block(*s) for s in sets]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for k in range(2):
            with torch.cuda.stream(sides[k]):
                got[k] = block(*sets[k])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals_in_python(cuda):
    x, w, ends = randn((10, 16), "bf16", 1), randn((2, 16, 24), "bf16", 2), ends_of([4, 6])
    r = H.himuon_grouped_gated_mm(x, w, ends, keep=True)
    wd, dy = randn((2, 12, 16), "bf16", 3), randn((10, 16), "bf16", 4)
    for bad in (dict(act="tanh"), dict(out=r.pre), dict(keep=r.h), dict(out=r.h.cpu())):
        with pytest.raises(ValueError):
            H.himuon_grouped_gated_mm(x, w, ends, **bad)
    for bad in (dict(out=r.h.float()), dict(keep=r.pre.float())):
        with pytest.raises(TypeError):
            H.himuon_grouped_gated_mm(x, w, ends, **bad)
    with pytest.raises(ValueError):
        H.himuon_grouped_gated_mm(x, w[:, :, :23], ends)
    with pytest.raises(TypeError):
        H.himuon_grouped_gated_mm(x.float(), w, ends)
    with pytest.raises(TypeError):
        H.himuon_grouped_gated_mm(x, w, ends.long())
    with pytest.raises(ValueError):
        H.himuon_grouped_gated_mm(x, w, ends.cpu())
    with pytest.raises(H.HimuonError):
        H.himuon_grouped_gated_mm(x[:, :8], w, ends)
    with pytest.raises(H.HimuonError):   # [g | u] over x
        both = randn((10, 24), "bf16", 5)
        H.himuon_grouped_gated_mm(both[:, :16], w, ends, keep=both)
    for bad in (r.pre[:, :22], r.pre[:9], r.h):
        with pytest.raises(H.HimuonError):
            H.himuon_grouped_gated_mm_grad(dy, wd, ends, bad)
    with pytest.raises(TypeError):
        H.himuon_grouped_gated_mm_grad(dy, wd, ends, r.pre.float())
    with pytest.raises(ValueError):
        H.himuon_grouped_gated_mm_grad(dy, wd, ends, r.pre.cpu())
