"""The experts' products on the GPU against fp64.

Tolerance, elementwise: the products of bf16 or fp32 inputs are accumulated in
fp32 over L terms in some order, so the error is at most 2 L 2^-24 sum |a b|
(one rounding of up to 2^-23 for each addition of a partial sum that stays
below sum |a b|), and the result is rounded once: 2^-8 |y| bounds half a unit
in bf16, 2^-23 |y| in fp32.
"""
import pytest
import torch

import tiled_newton_schulz_amd as H

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -23}


def randn(shape, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(TYPES[dt]).cuda()


def ends_of(counts):
    return torch.tensor(counts).cumsum(0).to(torch.int32).cuda()


def product(a, b, dt):
    """(a @ b, its bound) in fp64 on the host."""
    a, b = a.double().cpu(), b.double().cpu()
    y = a @ b
    return y, 2 * a.shape[1] * 2.0 ** -24 * (a.abs() @ b.abs()) + ROUND[dt] * y.abs()


def close(got, want, bound):
    d = (got.double().cpu() - want).abs()
    assert torch.all(d <= bound), float((d - bound).max())


def check_mm(x, w, counts, dt, out=None):
    y = H.himuon_grouped_mm(x, w, ends_of(counts), out=out)
    torch.cuda.synchronize()
    r = 0
    for e, c in enumerate(counts):
        if c:
            close(y[r:r + c], *product(x[r:r + c], w[e], dt))
        r += c
    assert torch.all(y[r:] == 0)
    return y


def check_wgrad(x, d, counts, dt, out=None):
    g = H.himuon_grouped_wgrad(x, d, ends_of(counts), out=out)
    torch.cuda.synchronize()
    r = 0
    for e, c in enumerate(counts):
        if c:
            close(g[e], *product(x[r:r + c].t(), d[r:r + c], dt))
        else:
            assert torch.all(g[e] == 0)
        r += c
    return g


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
]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("stored", ["kn", "nk"])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_product(cuda, counts, K, N, stored, dt):
    print(f"product {counts} {K}x{N} {stored} {dt}", flush=True)
    M, n = sum(counts), len(counts)
    x = randn((M, K), dt, 1)
    w = randn((n, K, N), dt, 2) if stored == "kn" else randn((n, N, K), dt, 2).transpose(1, 2)
    check_mm(x, w, counts, dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_weight_gradient(cuda, counts, K, N, dt):
    print(f"weight gradient {counts} {K}x{N} {dt}", flush=True)
    M = sum(counts)
    check_wgrad(randn((M, K), dt, 3), randn((M, N), dt, 4), counts, dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 1), (24, 8)])
def test_strides_and_padding(cuda, dt, pad, shift):
    """Column blocks of wider tensors whose other columns hold NaN, outputs
    into the middle of a wider tensor whose other columns stay as they were,
    a list of separate weights and of transposed ones."""
    counts, K, N = [70, 0, 130, 9], 144, 168
    M, n = sum(counts), len(counts)

    def wide(rows, cols, seed):
        t = torch.full((rows, cols + pad + shift), float("nan"), dtype=TYPES[dt], device=cuda)
        v = t[:, shift:shift + cols]
        v.copy_(randn((rows, cols), dt, seed))
        return v

    print(f"strides pad {pad} shift {shift} {dt}", flush=True)
    x, d = wide(M, K, 5), wide(M, N, 6)
    w = [wide(K, N, 10 + e) for e in range(n)]
    wt = [wide(N, K, 20 + e).t() for e in range(n)]
    for weights in (w, wt):
        store = torch.full((M, N + pad + shift), 7.0, dtype=TYPES[dt], device=cuda)
        check_mm(x, weights, counts, dt, out=store[:, shift:shift + N])
        assert torch.all(store[:, :shift] == 7.0) and torch.all(store[:, shift + N:] == 7.0)
    for tr in (False, True):
        stores = [torch.full((N, K + pad + shift) if tr else (K, N + pad + shift), 7.0, dtype=TYPES[dt], device=cuda)
                  for _ in range(n)]
        g = [s[:, shift:shift + (K if tr else N)] for s in stores]
        check_wgrad(x, d, counts, dt, out=[v.t() for v in g] if tr else g)
        for s in stores:
            assert torch.all(s[:, :shift] == 7.0) and torch.all(s[:, shift + (K if tr else N):] == 7.0)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("K,N", [(72, 88), (200, 264), (131, 77)])
def test_nan_stays_with_its_expert(cuda, dt, K, N):
    """NaN in the rows or weights of one expert, in rows of no expert and in
    the weights of an expert without rows reaches nobody else."""
    counts = [30, 1, 0, 100, 65]
    M, n = sum(counts), len(counts)
    x, d, w = randn((M + 20, K), dt, 7), randn((M + 20, N), dt, 8), randn((n, K, N), dt, 9)
    bad = slice(31, 131)
    for t in (x, d):
        t[bad] = float("nan")
        t[M:] = float("nan")
    w[2:4] = float("nan")
    print(f"nan {K}x{N} {dt}", flush=True)
    for stored in (w, w.transpose(1, 2).contiguous().transpose(1, 2)):
        y = H.himuon_grouped_mm(x, stored, ends_of(counts))
        assert torch.isnan(y[bad]).all() and torch.all(y[M:] == 0)
        for e, r in ((0, slice(0, 30)), (1, slice(30, 31)), (4, slice(131, M))):
            close(y[r], *product(x[r], w[e], dt))
    g = H.himuon_grouped_wgrad(x, d, ends_of(counts))
    assert torch.isnan(g[3]).all() and torch.all(g[2] == 0)
    for e, r in ((0, slice(0, 30)), (1, slice(30, 31)), (4, slice(131, M))):
        close(g[e], *product(x[r].t(), d[r], dt))


def guarded_block(rows, cols, dt, seed, before, after):
    """A column block whose neighbours, and the rows around it, hold NaN."""
    t = torch.full((rows + 2, before + cols + after), float("nan"), dtype=TYPES[dt], device="cuda")
    v = t[1:rows + 1, before:before + cols]
    v.copy_(randn((rows, cols), dt, seed))
    return v


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("K,N", [(1, 3), (3, 1), (5, 7), (9, 2), (65, 66), (71, 67), (130, 39), (513, 65), (519, 5), (1030, 129),
                                 (2047, 3)])
def test_narrow_and_long(cuda, K, N, dt):
    """Widths that end inside a 16-byte chunk or fall short of one, few tiles
    with long sums (along K and along the rows), NaN around every operand."""
    print(f"narrow {K}x{N} {dt}", flush=True)
    counts = [70, 0, 1200, 2]
    M, n = sum(counts), len(counts)
    x, d = guarded_block(M, K, dt, 5, 3, 2), guarded_block(M, N, dt, 6, 1, 4)
    w = [guarded_block(K, N, dt, 10 + e, 1, 4) for e in range(n)]
    wt = [guarded_block(N, K, dt, 20 + e, 5, 2).t() for e in range(n)]
    for ws in (w, wt):
        y = guarded_block(M, N, dt, 7, 2, 3)
        check_mm(x, ws, counts, dt, out=y)
        base = y._base.clone()
        base[1:M + 1, 2:2 + N] = float("nan")
        assert torch.isnan(base).all()
    g = [guarded_block(K, N, dt, 30 + e, 4, 1) for e in range(n)]
    check_wgrad(x, d, counts, dt, out=g)
    for v in g:
        base = v._base.clone()
        base[1:K + 1, 4:4 + N] = float("nan")
        assert torch.isnan(base).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("counts,K,N", [([5000], 40, 48), ([9, 0, 6001, 2000], 130, 65), ([2100, 2100], 128, 256), ([12345], 8, 3),
                                          ([9, 0, 13001, 5000], 130, 65)])
def test_rows_in_parts(cuda, counts, K, N, dt):
    """Weight gradients whose rows are cut into parts: experts with fewer rows
    than parts, rows past the last expert, the workspace given or not, and no
    write outside it."""
    print(f"rows in parts {counts} {K}x{N} {dt}", flush=True)
    M, n = sum(counts) + 77, len(counts)
    x, d = randn((M, K), dt, 40), randn((M, N), dt, 41)
    x[M - 77:] = float("nan")
    need = H.himuon_grouped_wgrad_workspace(x, d, n)
    first = check_wgrad(x, d, counts, dt)
    if need == 0:   # too few rows an expert
        assert M // n < 2560
        return
    ws = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    g = H.himuon_grouped_wgrad(x, d, ends_of(counts), workspace=ws)
    assert torch.equal(g, first) and torch.all(ws[need:] == 0x5a)
    with pytest.raises(H.HimuonError):
        H.himuon_grouped_wgrad(x, d, ends_of(counts), workspace=ws[:need - 16])


def test_many_experts_and_no_rows(cuda):
    """More experts than one launch holds, and calls without a row."""
    n, K, N = 600, 40, 24
    g = torch.Generator().manual_seed(11)
    counts = torch.randint(0, 5, (n,), generator=g).tolist()
    counts[254:258] = [0, 70, 0, 3]
    M = sum(counts)
    print("600 experts", flush=True)
    x, d, w = randn((M + 9, K), "bf16", 12), randn((M + 9, N), "bf16", 13), randn((n, K, N), "bf16", 14)
    check_mm(x, w, counts, "bf16")
    check_wgrad(x, d, counts, "bf16")
    none = [0] * 3
    assert H.himuon_grouped_mm(x[:0], w[:3], ends_of(none)).shape == (0, N)
    assert torch.all(H.himuon_grouped_wgrad(x[:0], d[:0], ends_of(none)) == 0)
    assert torch.all(H.himuon_grouped_mm(x, w[:3], ends_of(none)) == 0)
    assert torch.all(H.himuon_grouped_wgrad(x, d, ends_of(none)) == 0)


def test_ends_are_clamped(cuda):
    """End rows outside [0, M] are clamped to it."""
    x, w = randn((50, 32), "bf16", 15), randn((3, 32, 16), "bf16", 16)
    ends = torch.tensor([-5, 20, 1 << 30], dtype=torch.int32, device=cuda)
    y = H.himuon_grouped_mm(x, w, ends)
    close(y[:20], *product(x[:20], w[1], "bf16"))
    close(y[20:], *product(x[20:], w[2], "bf16"))
    g = H.himuon_grouped_wgrad(x, x, ends)
    assert torch.all(g[0] == 0)
    close(g[2], *product(x[20:].t(), x[20:], "bf16"))


def test_same_bits_and_other_streams(cuda):
    """The same call gives the same bits again, on a stream of the caller's
    choice, and from a captured graph replayed between eager calls."""
    counts = [100, 3, 0, 290, 41]
    x, d = randn((sum(counts), 256), "bf16", 17), randn((sum(counts), 136), "bf16", 18)
    w, ends = H.matrices(randn((5, 256, 136), "bf16", 19)), ends_of(counts)
    y0, g0 = H.himuon_grouped_mm(x, w, ends), H.himuon_grouped_wgrad(x, d, ends)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1 = H.himuon_grouped_mm(x, w, ends, stream=side)
    g1 = H.himuon_grouped_wgrad(x, d, ends, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(g0, g1)
    y2, g2 = torch.empty_like(y0), torch.empty_like(g0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H.himuon_grouped_mm(x, w, ends, out=y2)
        H.himuon_grouped_wgrad(x, d, ends, out=g2)
    for k in range(3):
        x.copy_(randn(tuple(x.shape), "bf16", 30 + k))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y2, H.himuon_grouped_mm(x, w, ends))
        assert torch.equal(g2, H.himuon_grouped_wgrad(x, d, ends))


def test_gradients_against_differences(cuda):
    """L = <Y, R>: its difference along a direction of X and of W against the
    input and weight gradients.  L is linear in each, so the difference is
    exact up to the rounding of the two products: for entries of size about 1
    it is sqrt(M N) K 2^-23 of their norm, taken ten times over."""
    counts, K, N = [40, 0, 77], 48, 56
    M = sum(counts)
    x, w, R = randn((M, K), "fp32", 20), randn((3, K, N), "fp32", 21), randn((M, N), "fp32", 22)
    u, v = randn((M, K), "fp32", 23), randn((3, K, N), "fp32", 24)
    ends = ends_of(counts)

    def loss(x, w):
        return float((H.himuon_grouped_mm(x, w, ends).double() * R.double()).sum())

    dx = H.himuon_grouped_mm(R, w.transpose(1, 2), ends)
    dw = H.himuon_grouped_wgrad(x, R, ends)
    tol = 10 * M * N * K * 2.0 ** -23
    assert abs((loss(x + u, w) - loss(x - u, w)) / 2 - float((dx.double() * u.double()).sum())) <= tol
    assert abs((loss(x, w + v) - loss(x, w - v)) / 2 - float((dw.double() * v.double()).sum())) <= tol


def test_large_products(cuda):
    """Column and row tiles at full size, against fp64 on sampled rows and columns."""
    counts, K, N = [700, 0, 1, 1100, 255], 1408, 2048
    M = sum(counts)
    print("large products", flush=True)
    x, d = randn((M, K), "bf16", 25), randn((M, N), "bf16", 26)
    w = randn((5, K, N), "bf16", 27)
    ends = ends_of(counts)
    rows = torch.tensor([0, 255, 256, 699, 700, 701, 956, 957, 1800, 1801, M - 1])
    for weights in (w, w.transpose(1, 2).contiguous().transpose(1, 2)):
        y = H.himuon_grouped_mm(x, weights, ends)
        for r in rows.tolist():
            e = int((ends.cpu() <= r).sum())
            close(y[r:r + 1], *product(x[r:r + 1], w[e], "bf16"))
    g = H.himuon_grouped_wgrad(x, d, ends)
    r = 0
    for e, c in enumerate(counts):
        for i in (0, 127, 128, 255, 256, 1279, 1280, 1407):
            if c:
                close(g[e][i:i + 1], *product(x[r:r + c, i:i + 1].t(), d[r:r + c], "bf16"))
        r += c
    assert torch.all(g[1] == 0)


def ragged(n, most, seed, none=0.1):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(1, most + 1, (n,), generator=g)
    c[torch.rand(n, generator=g) < none] = 0
    return c.tolist()


# (experts, most rows of one, K, N): many 256-wide tiles, K and N that end
# inside a step of 64 or a tile of 256, row tiles of one to four blocks of 64
TILED = [(64, 300, 200, 1416), (40, 700, 72, 2048), (64, 90, 520, 1408), (300, 60, 64, 264), (33, 260, 128, 1800)]


@pytest.mark.parametrize("stored", ["kn", "nk"])
@pytest.mark.parametrize("n,most,K,N", TILED)
def test_many_tiles(cuda, n, most, K, N, stored):
    """Enough tiles for the largest tile kernel, several to a workgroup."""
    counts = ragged(n, most, n)
    M = sum(counts)
    print(f"many tiles {n} x {most} x {K} x {N} {stored}, {M} rows", flush=True)
    x = randn((M + 11, K), "bf16", 40)
    w = randn((n, K, N), "bf16", 41) if stored == "kn" else randn((n, N, K), "bf16", 41).transpose(1, 2)
    # NaN beside the operands: in rows of no expert, in the weights of experts without rows
    x[M:] = float("nan")
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = float("nan")
    check_mm(x, w, counts, "bf16")


@pytest.mark.parametrize("n,most,K,N", [(64, 300, 200, 520), (20, 700, 1032, 776), (300, 40, 264, 72), (64, 130, 264, 640)])
def test_many_gradient_tiles(cuda, n, most, K, N):
    counts = ragged(n, most, n + 1)
    M = sum(counts)
    print(f"many gradient tiles {n} x {most} x {K} x {N}, {M} rows", flush=True)
    x, d = randn((M + 11, K), "bf16", 42), randn((M + 11, N), "bf16", 43)
    x[M:] = float("nan")
    d[M:] = float("nan")
    check_wgrad(x, d, counts, "bf16")


def test_many_tiles_strided_and_repeated(cuda):
    """Column blocks of wider tensors at 16-byte offsets whose other columns hold
    NaN, results into the middle of a wider tensor, the same bits again, and one
    expert that holds nearly all rows."""
    n, K, N = 48, 136, 1288
    counts = ragged(n, 200, 7)
    counts[5] = 9000
    M = sum(counts)
    big = torch.full((M, K + 24), float("nan"), dtype=torch.bfloat16, device=cuda)
    x = big[:, 8:8 + K]
    x.copy_(randn((M, K), "bf16", 44))
    wide = torch.full((n, K, N + 16), float("nan"), dtype=torch.bfloat16, device=cuda)
    w = wide[:, :, 8:8 + N]
    w.copy_(randn((n, K, N), "bf16", 45))
    store = torch.full((M, N + 16), 7.0, dtype=torch.bfloat16, device=cuda)
    y = check_mm(x, w, counts, "bf16", out=store[:, 8:8 + N])
    assert torch.all(store[:, :8] == 7.0) and torch.all(store[:, 8 + N:] == 7.0)
    ends = ends_of(counts)
    assert torch.equal(y, H.himuon_grouped_mm(x, w, ends))
    d = randn((M, N), "bf16", 46)
    g = check_wgrad(x, d, counts, "bf16")
    assert torch.equal(g, H.himuon_grouped_wgrad(x, d, ends))


def test_difference_quotients_tightly(cuda):
    """<Y, R> is linear in X and in W, so its difference along a direction differs
    from <gradient, direction> by roundings alone.  An element of Y is off by at
    most 2 K 2^-24 sum |x w| (as above), the gradients alike over N and over the
    rows; each is multiplied by its partner and summed in fp64."""
    counts, K, N = [40, 0, 77], 48, 56
    M = sum(counts)
    x, w, R = randn((M, K), "fp32", 20), randn((3, K, N), "fp32", 21), randn((M, N), "fp32", 22)
    u, v = randn((M, K), "fp32", 23), randn((3, K, N), "fp32", 24)
    ends = ends_of(counts)
    expert = torch.repeat_interleave(torch.arange(3), torch.tensor(counts))

    def loss(x, w):
        """(<Y, R>, bound of its error)"""
        y = H.himuon_grouped_mm(x, w, ends).double().cpu()
        size = torch.bmm(x.double().cpu().abs()[:, None], w.double().cpu().abs()[expert])[:, 0]
        r = R.double().cpu()
        return float((y * r).sum()), (2 * K * 2.0 ** -24) * float((size * r.abs()).sum())

    dx = H.himuon_grouped_mm(R, w.transpose(1, 2), ends).double().cpu()
    dw = H.himuon_grouped_wgrad(x, R, ends).double().cpu()
    wa, ra, xa = w.double().cpu().abs(), R.double().cpu().abs(), x.double().cpu().abs()
    bx = 2 * N * 2.0 ** -24 * float((torch.bmm(ra[:, None], wa.transpose(1, 2).contiguous()[expert])[:, 0] * u.double().cpu().abs()).sum())
    bw, r = 0.0, 0
    for e, c in enumerate(counts):
        bw += 2 * max(c, 1) * 2.0 ** -24 * float(((xa[r:r + c].t() @ ra[r:r + c]) * v[e].double().cpu().abs()).sum())
        r += c
    # the sums x + u and w + v are rounded to fp32 as well
    for up, down, grad, along, bound in ((loss(x + u, w), loss(x - u, w), dx, u, bx), (loss(x, w + v), loss(x, w - v), dw, v, bw)):
        diff = (up[0] - down[0]) / 2
        tol = (up[1] + down[1]) / 2 + bound + (up[1] + down[1]) / (2 * 2 * K)
        assert abs(diff - float((grad * along.double().cpu()).sum())) <= tol


@pytest.mark.parametrize("dt,K,N", [("bf16", 4096, 4096), ("bf16", 4095, 4097), ("fp32", 2048, 4100)])
def test_operands_past_2_to_the_31_elements(cuda, dt, K, N):
    """Rows and results whose offsets pass 32 bits: sampled rows and columns
    against fp64."""
    M = (1 << 31) // min(K, N) + 5000
    counts = [M // 3, 5, M - M // 3 - 5 - 100]
    print(f"past 2^31: {M} rows {K}x{N} {dt}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(50)

    def big(rows, cols):
        t = torch.empty((rows, cols), dtype=TYPES[dt], device="cuda")
        for r in range(0, rows, 1 << 16):
            t[r:r + (1 << 16)] = torch.randn((min(1 << 16, rows - r), cols), generator=g, device="cuda")
        return t

    x, w = big(M, K), big(3 * K, N).view(3, K, N)
    ends = ends_of(counts)
    sample = torch.tensor([0, M // 3 - 1, M // 3, M // 3 + 5, M // 2, M - 102, M - 101])
    for weights in (w, w.transpose(1, 2).contiguous().transpose(1, 2)):
        y = H.himuon_grouped_mm(x, weights, ends)
        for r in sample.tolist():
            e = int((ends.cpu() <= r).sum())
            close(y[r:r + 1], *product(x[r:r + 1], w[e], dt))
        assert torch.all(y[M - 100:] == 0)
        del weights
    d = y
    for r in range(0, M, 1 << 16):
        d[r:r + (1 << 16)] = torch.randn((min(1 << 16, M - r), N), generator=g, device="cuda")
    got = H.himuon_grouped_wgrad(x, d, ends)
    r = 0
    for e, c in enumerate(counts):
        rows = slice(r, r + c)
        for i in (0, K // 2, K - 1):
            a, b = x[rows, i].double(), d[rows][:, [0, 255, 256, N - 1]]
            want = torch.stack([(a * b[:, j].double()).sum() for j in range(4)]).cpu()
            size = torch.stack([(a.abs() * b[:, j].double().abs()).sum() for j in range(4)]).cpu()
            close(got[e, i, [0, 255, 256, N - 1]], want, 2 * c * 2.0 ** -24 * size + ROUND[dt] * want.abs())
        r += c
