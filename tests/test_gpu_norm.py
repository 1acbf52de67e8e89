"""Layer normalisation on the GPU against fp64.

Tolerances, elementwise, with u = 2^-24.  A row's sum goes through chains of at most 64
additions in a thread and 16 more over the threads: off by at most 90 u sum |terms|
with the rounding of the terms.  So mean is off by Em = 92 u mean |x|; the variance by
96 u var + Em^2 (differences to a mean that is off by Em); rstd by half its relative
error and 4 u; and y by |w| (rstd Em + |x_hat| (rel(rstd) + 4 u)) + 2 u (|y| + |b|).  A
gradient takes the stats it is given: its two means are off by 92 u of the mean of
their terms' sizes, each term by 4 u.  The sums over N rows go through chains of at
most N / 256 + 128 additions.  Results are rounded once: eps / 2.
"""
import pytest
import torch

import tiled_newton_schulz_amd as H

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
U = 2.0 ** -24


def randn(shape, dt, seed, scale=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + mean).to(TYPES[dt]).cuda()


def close(got, want, off, dt, what):
    bound = off + HALF[dt] * (want.abs() + off) + 1e-37
    d = (got.double() - want).abs()
    assert torch.all(d <= bound), f"{what}: {float((d - bound).max())} over, of {float(want.abs().max())}"


def check_forward(x, w, b, eps, dt, **more):
    r = H.himuon_layer_norm(x, w, b, eps=eps, **more)
    torch.cuda.synchronize()
    check_rows(x, w, b, eps, dt, r.y, r.stats)
    return r


def check_rows(x, w, b, eps, dt, got, stats):
    x64 = x.double()
    mean = x64.mean(1, keepdim=True)
    d = x64 - mean
    var = d.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    em = 92 * U * x64.abs().mean(1, keepdim=True)
    rr = 0.5 * (96 * U * var + em ** 2) / (var + eps) + 4 * U
    w64 = 1.0 if w is None else w.double()
    b64 = torch.zeros((), device=x.device).double() if b is None else b.double()
    y = d * rstd * w64 + b64
    off = abs(w64) * (rstd * em + (d * rstd).abs() * (rr + 4 * U)) + 2 * U * (y.abs() + b64.abs())
    close(got, y, off, dt, "y")
    if stats is not None:
        s = stats.double()
        assert torch.all((s[:, :1] - mean).abs() <= em + 1e-37) and torch.all((s[:, 1:] / rstd - 1).abs() <= rr)


def check_grad(x, w, stats, dy, dt, **more):
    r = H.himuon_layer_norm_grad(x, w, stats, dy, **more)
    torch.cuda.synchronize()
    check_grads(x, w, stats, dy, dt, r)
    return r


def check_grads(x, w, stats, dy, dt, r):
    x64, g = x.double(), dy.double()
    N, s = x.shape[0], stats.double()
    xh = (x64 - s[:, :1]) * s[:, 1:]
    gw = g if w is None else g * w.double()
    s1, s2 = gw.mean(1, keepdim=True), (gw * xh).mean(1, keepdim=True)
    dx = s[:, 1:] * (gw - s1 - xh * s2)
    off = s[:, 1:].abs() * (4 * U * (gw.abs() + s1.abs() + (xh * s2).abs()) + 96 * U * gw.abs().mean(1, keepdim=True) +
                            100 * U * xh.abs() * (gw * xh).abs().mean(1, keepdim=True))
    if r.dx is not None:
        close(r.dx, dx, off, dt, "dx")
    chain = (N / 256 + 128) * U
    if r.dweight is not None:
        close(r.dweight, (g * xh).sum(0), (chain + 4 * U) * (g * xh).abs().sum(0), dt, "dweight")
    if r.dbias is not None:
        close(r.dbias, g.sum(0), chain * g.abs().sum(0), dt, "dbias")


# around every size at which rows are held in another way, and odd ones
COLS = [1, 2, 7, 8, 15, 16, 17, 32, 33, 63, 64, 65, 128, 129, 255, 257, 512, 513, 1000, 1024, 1025, 1409, 2048, 2049, 4095, 4096, 4097,
        8192, 8200, 16384, 16385, 32767, 32768]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("cols", COLS)
def test_widths(cuda, cols, dt):
    for rows in (1, 5, 67) if cols < 9000 else (1, 6):
        print(f"layer norm {rows} x {cols} {dt}", flush=True)
        x = randn((rows, cols), dt, 1, 2.0, 0.5)
        w, b = randn((cols,), dt, 2, 0.3, 1.0), randn((cols,), dt, 3, 0.2)
        r = check_forward(x, w, b, 1e-5, dt)
        check_grad(x, w, r.stats, randn((rows, cols), dt, 4), dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(3000, 24), (5000, 100), (2500, 777), (1300, 2048), (700, 4096), (1100, 5000), (9000, 512)])
def test_many_rows(cuda, rows, cols, dt):
    print(f"layer norm {rows} x {cols} {dt}", flush=True)
    x, w = randn((rows, cols), dt, 1), randn((cols,), dt, 2, 0.3, 1.0)
    r = check_forward(x, w, None, 1e-6, dt)
    a = check_grad(x, w, r.stats, randn((rows, cols), dt, 4), dt)
    b = check_grad(x, w, r.stats, randn((rows, cols), dt, 4), dt)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_optional_parts(cuda, dt):
    """No weight, no bias, no stats; each gradient alone."""
    x, w, b = randn((50, 300), dt, 1), randn((300,), dt, 2), randn((300,), dt, 3)
    print(f"layer norm, parts left out {dt}", flush=True)
    check_forward(x, None, None, 1e-5, dt)
    check_forward(x, None, b, 1e-5, dt)
    assert check_forward(x, w, b, 1e-5, dt, stats=False).stats is None
    st = check_forward(x, w, None, 1e-5, dt).stats
    dy = randn((50, 300), dt, 4)
    full = check_grad(x, w, st, dy, dt)
    check_grad(x, None, st, dy, dt)
    for k in range(3):
        some = check_grad(x, w, st, dy, dt, dx=k == 0, dweight=k == 1, dbias=k == 2)
        assert [p is not None for p in some] == [k == 0, k == 1, k == 2] and torch.equal(some[k], full[k])


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("cols,pad,shift", [(96, 8, 0), (96, 3, 1), (301, 5, 3), (5000, 24, 8)])
def test_strides_and_in_place(cuda, dt, cols, pad, shift):
    """Rows inside wider ones whose other columns hold NaN (read) or 7 (written and
    left); results in place of an operand."""
    def wide(fill, seed=None):
        t = torch.full((40, cols + pad + shift), fill, dtype=TYPES[dt], device=cuda)
        v = t[:, shift:shift + cols]
        if seed is not None:
            v.copy_(randn((40, cols), dt, seed))
        return t, v

    print(f"layer norm strides {cols} pad {pad} shift {shift} {dt}", flush=True)
    w, b = (torch.cat([t[:1], t])[1:] for t in (randn((cols,), dt, 2), randn((cols,), dt, 3)))
    (_, x), (_, dy) = wide(float("nan"), 1), wide(float("nan"), 4)
    (ty, y), (tdx, dx) = wide(7.0), wide(7.0)
    r = check_forward(x, w, b, 1e-5, dt, out=y)
    g = check_grad(x, w, r.stats, dy, dt, dx=dx)
    for t in (ty, tdx):
        assert torch.all(t[:, :shift] == 7.0) and torch.all(t[:, shift + cols:] == 7.0)
    for k in (x, dy):
        t = k.clone()
        h = H.himuon_layer_norm_grad(t if k is x else x, w, r.stats, t if k is dy else dy, dx=t)
        assert all(torch.equal(p, q) for p, q in zip(h, g))
    t = x.clone()
    assert torch.equal(H.himuon_layer_norm(t, w, b, out=t).y, r.y)


def test_no_rows(cuda):
    print("layer norm without rows", flush=True)
    x, w = torch.empty((0, 48), device=cuda), torch.ones(48, device=cuda)
    r = H.himuon_layer_norm(x, w, w)
    g = H.himuon_layer_norm_grad(x, w, r.stats, x)
    assert r.y.shape == g.dx.shape == (0, 48) and torch.all(g.dweight == 0) and torch.all(g.dbias == 0)


def test_hard_rows(cuda):
    """A mean far above the spread, equal values, values near the types' ends, a row
    with NaN and one with infinity, which reach no other row."""
    print("layer norm, hard rows", flush=True)
    x = randn((8, 200), "fp32", 1)
    x[1] += 1e5
    x[2] = 3.25
    x[3] *= 1e-18
    x[4] *= 1e17
    w = randn((200,), "fp32", 2)
    check_forward(x, w, None, 1e-5, "fp32")
    assert torch.all(H.himuon_layer_norm(x, w).y[2] == 0)
    x[5, 7], x[6, 9] = float("nan"), float("inf")
    y = H.himuon_layer_norm(x, w).y
    bad = torch.isnan(y).all(1)
    assert bad.tolist() == [False] * 5 + [True, True, False] and not torch.isnan(y[~bad]).any()


def test_streams_and_graphs(cuda):
    print("layer norm captured", flush=True)
    for rows, cols in ((300, 520), (40, 9000)):
        x, w, b, dy = randn((rows, cols), "bf16", 1), randn((cols,), "bf16", 2), randn((cols,), "bf16", 3), randn((rows, cols), "bf16", 4)

        def both():
            r = H.himuon_layer_norm(x, w, b)
            return (*r, *H.himuon_layer_norm_grad(x, w, r.stats, dy))

        want = both()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = []
        with torch.cuda.stream(side):
            got = both()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = both()
        for k in range(3):
            x.copy_(randn((rows, cols), "bf16", 10 + k))
            want = both()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want)), k


def test_gradients_against_differences(cuda):
    """fp32: central differences of sum(y c) in fp64."""
    print("layer norm against differences", flush=True)
    x, w, b, c = randn((6, 40), "fp32", 1), randn((40,), "fp32", 2), randn((40,), "fp32", 3), randn((6, 40), "fp32", 4)
    g = H.himuon_layer_norm_grad(x, w, H.himuon_layer_norm(x, w, b).stats, c)

    def value(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return ((d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b) * c.double()).sum()

    args, gen = [t.double() for t in (x, w, b)], torch.Generator().manual_seed(5)
    for i, t in enumerate(args):
        for _ in range(6):
            v = torch.randn(t.shape, generator=gen).double().cuda()
            up, down = ([a + s * 1e-5 * v if j == i else a for j, a in enumerate(args)] for s in (1, -1))
            slope = (value(*up) - value(*down)) / 2e-5
            # h^2 / 6 = 2e-11 of the third derivative; the gradients within 100 u of their terms
            assert abs((g[i].double() * v).sum() - slope) <= 1e-7 + 400 * U * (g[i].double().abs() * v.abs()).sum() + 400 * U * c.abs().sum()


@pytest.mark.parametrize("dt,cols", [("bf16", 4096), ("fp32", 2047), ("bf16", 32760)])
def test_rows_past_2_to_the_31_elements(cuda, dt, cols):
    rows = (1 << 31) // cols + 301
    print(f"layer norm {rows} x {cols} {dt}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((rows, cols), dtype=TYPES[dt], device=cuda).normal_(generator=gen)
    w = randn((cols,), dt, 2)
    r = H.himuon_layer_norm(x, w)
    ends = (slice(0, 40), slice(rows - 40, rows))
    for part in ends:
        check_rows(x[part], w, None, 1e-5, dt, r.y[part], r.stats[part])
    dy = r.y   # (any gradient)
    kept = [dy[part].clone() for part in ends]
    g = H.himuon_layer_norm_grad(x, w, r.stats, dy, dx=dy)
    for part, k in zip(ends, kept):
        check_grads(x[part], w, r.stats[part], k, dt, H.NormGrad(g.dx[part]))
    # the sums over all rows, from sums over blocks of them in fp64
    sums, size = torch.zeros(cols, dtype=torch.float64, device=cuda), torch.zeros(cols, dtype=torch.float64, device=cuda)
    again = H.himuon_layer_norm(x, w).y
    for block in again.split(4096):
        sums += block.double().sum(0)
        size += block.double().abs().sum(0)
    close(g.dbias, sums, (rows / 256 + 128) * U * size, dt, "dbias")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 20000), (3, 17000), (37, 30001), (0, 32768), (130, 24576)])
def test_wide_rows(cuda, rows, cols, dt):
    """Rows whose sums are a launch of their own; dx over dy and over x."""
    print(f"layer norm {rows} x {cols} {dt}", flush=True)
    x, w, dy = randn((rows, cols), dt, 1), randn((cols,), dt, 2), randn((rows, cols), dt, 3)
    r = check_forward(x, w, None, 1e-5, dt)
    g = check_grad(x, w, r.stats, dy, dt) if rows else H.himuon_layer_norm_grad(x, w, r.stats, dy)
    if rows == 0:
        assert torch.all(g.dweight == 0) and torch.all(g.dbias == 0)
    for over in (x.clone(), dy.clone()):
        args = (over, dy) if torch.equal(over, x) else (x, over)
        h = H.himuon_layer_norm_grad(args[0], w, r.stats, args[1], dx=over)
        assert all(torch.equal(p, q) for p, q in zip(h, g))


def test_refusals_in_python(cuda):
    x, w = randn((4, 16), "bf16", 1), randn((16,), "bf16", 2)
    r = H.himuon_layer_norm(x, w)
    for bad in (dict(weight=w[:8]), dict(weight=w.cpu()), dict(bias=torch.cat([w, w])[::2]), dict(out=r.y[:3]), dict(out=r.y.cpu())):
        with pytest.raises(ValueError):
            H.himuon_layer_norm(x, **bad)
    for bad in (dict(weight=w.float()), dict(out=r.y.float())):
        with pytest.raises(TypeError):
            H.himuon_layer_norm(x, **bad)
    with pytest.raises(ValueError):
        H.himuon_layer_norm(x.cpu(), w.cpu())
    with pytest.raises(ValueError):
        H.himuon_layer_norm(x.t())
    with pytest.raises(H.HimuonError):
        H.himuon_layer_norm(x, w, eps=-1.0)
    with pytest.raises(H.HimuonError):
        H.himuon_layer_norm(randn((2, H.MAX_NORM_COLS + 1), "bf16", 3))
    with pytest.raises(TypeError):
        H.himuon_layer_norm_grad(x, w, r.stats.double(), x)
    with pytest.raises(ValueError):
        H.himuon_layer_norm_grad(x, w, r.stats[:3], x)
    with pytest.raises(TypeError):
        H.himuon_layer_norm_grad(x, w, r.stats, x.float())
    with pytest.raises(H.HimuonError):
        H.himuon_layer_norm_grad(x, w, r.stats, x[:3])
    with pytest.raises(H.HimuonError):   # one vector for both sums
        v = w.clone()
        H.himuon_layer_norm_grad(x, w, r.stats, r.y, dweight=v, dbias=v)
    with pytest.raises(H.HimuonError):   # a workspace that is too small
        H.himuon_layer_norm_grad(x, w, r.stats, r.y, workspace=torch.empty(16, device=cuda))
