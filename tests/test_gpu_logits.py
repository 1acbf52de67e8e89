"""Distillation and token log probabilities on the GPU against fp64.

Bounds.  With A the largest finite |s| of a row, s = z / temperature: s itself
carries a relative error of 2^-22 (the reciprocal of the temperature and one
product), an exponential of |x| <= 2 A + 8 a relative error of 2^-22 (2 A + 8)
(its argument's rounding and a few units of the instruction), and a sum of V
terms in parts of at most V / 64 + 64 additions (V / 64 + 64) 2^-24.  So log q
is off by at most

    d = 2^-20 (A + 8) + (V / 64 + 64) 2^-24,

q by d relative to itself, the entropy by d (2 A + 8 + log V), and likewise
with A_t, k for the teacher's p (d_p).  The loss is off by at most
P (d + d_p (1 + max |log p - log q|)), the gradient by
c (P q (d + d_p) + p d_p), c = |weight| / temperature, before it is rounded to
its type: 2^-8 (bf16), 2^-22 (fp32) of itself.
"""
import ctypes
import math

import pytest
import torch

import tiled_newton_schulz_amd as H

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -22}
INF = float("inf")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def logits(N, V, dt, seed, scale=3.0, mask=0.0):
    z = torch.randn((N, V), generator=gen(seed)) * scale
    if mask:
        z[torch.rand((N, V), generator=gen(seed + 1)) < mask] = -INF
        z[:, 0] = 1.0
    return z.to(TYPES[dt])


def strided(z, pad, shift):
    """The same values on the GPU inside a wider tensor of NaN."""
    t = torch.full((z.shape[0], z.shape[1] + pad + shift), float("nan"), dtype=z.dtype, device="cuda")
    v = t[:, shift:shift + z.shape[1]]
    v.copy_(z)
    return v


def row_bound(s, V):
    A = torch.where(torch.isfinite(s), s.abs(), 0.0).amax(1)
    return A, 2.0 ** -20 * (A + 8) + (V / 64 + 64) * 2.0 ** -24


def softmax64(z, tau):
    s = z.double() / tau
    lse = torch.logsumexp(s, 1)
    lq = s - lse[:, None]
    return s, lse, lq, torch.exp(lq)


def near(got, want, bound, what):
    got = got.double().cpu()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    ok = same | ((got - want).abs() <= bound)
    assert torch.all(ok), (what, float(torch.where(ok, 0.0, (got - want).abs() - bound).nan_to_num(9e99).max()))


# ---- token log probabilities -----------------------------------------------------

def check_logprobs(z, zg, tokens, top, tau, dt, r=None):
    N, V = z.shape
    if r is None:
        r = H.himuon_token_logprobs(zg, tokens.cuda(), top=top, temperature=tau)
    torch.cuda.synchronize()
    live = (tokens >= 0) & (tokens < V)
    s, lse, lq, q = softmax64(z, tau)
    A, d = row_bound(s, V)
    want = torch.where(live, lq.gather(1, tokens.long().clamp(0, V - 1)[:, None])[:, 0], 0.0)
    near(r.logp, want, d, "logp")
    H_ = -torch.where(q > 0, q * lq, 0.0).sum(1)
    near(r.entropy, torch.where(live, H_, 0.0), d * (2 * A + 8 + math.log(V)), "entropy")
    near(r.lse.double().sum(1), torch.where(live, lse, 0.0), d, "lse")
    if top:
        order = torch.sort(z.double(), dim=1, descending=True, stable=True)[1][:, :top]
        assert torch.equal(r.top_idx.cpu().long()[live], order[live])
        assert torch.all(r.top_idx.cpu()[~live] == -1) and torch.all(r.top_logp.cpu()[~live] == -INF)
        near(r.top_logp[live.cuda()], lq.gather(1, order)[live], d[live][:, None], "top_logp")
    return r, (s, lse, lq, q, H_, live, A, d)


def check_logprobs_grad(z, zg, tokens, tau, dt, r, ref, gl, gh, out=None):
    V = z.shape[1]
    s, lse, lq, q, H_, live, A, d = ref
    g = H.himuon_token_logprobs_grad(zg, tokens.cuda(), r.lse, r.entropy, None if gl is None else gl.cuda(),
                                     None if gh is None else gh.cuda(), temperature=tau, out=out)
    torch.cuda.synchronize()
    a = torch.zeros(z.shape[0]).double() if gl is None else gl.double()
    b = torch.zeros(z.shape[0]).double() if gh is None else gh.double()
    hot = torch.zeros_like(q)
    hot[torch.arange(z.shape[0]), tokens.long().clamp(0, V - 1)] = 1.0
    qlq = torch.where(q > 0, q * lq, 0.0)
    want = (a[:, None] * (hot - q) - b[:, None] * (qlq + q * H_[:, None])) / tau
    dH = d * (2 * A + 8 + math.log(V))
    # terms cancel: each carries its own rounding
    err = (a.abs()[:, None] * (q * d[:, None] + 2.0 ** -22 * (hot + q))
           + b.abs()[:, None] * (q * (d + dH)[:, None] + (qlq.abs() + q * H_[:, None].abs()) * (d[:, None] + 2.0 ** -21))) / tau
    want = torch.where(live[:, None], want, 0.0)
    near(g, want, err + ROUND[dt] * want.abs() + 1e-38, "grad")
    return g


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V,top", [(1, 1, 1), (3, 2, 2), (2, 64, 64), (5, 63, 5), (37, 1000, 20), (7, 5003, 3),
                                     (4, 32000, 64), (1, 131072, 20), (3, 131073, 1), (300, 257, 8), (2, 200001, 10)])
def test_logprobs(cuda, N, V, top, dt):
    print(f"logprobs {N}x{V} top {top} {dt}", flush=True)
    z = logits(N, V, dt, N + V, mask=0.1 if V > 2 else 0.0)
    tokens = torch.randint(0, V, (N,), generator=gen(1), dtype=torch.int64 if N % 2 else torch.int32)
    tau = [1.0, 0.7, 2.0][V % 3]
    zg = z.cuda()
    r, ref = check_logprobs(z, zg, tokens, top, tau, dt)
    gl, gh = torch.randn(N, generator=gen(2)), torch.randn(N, generator=gen(3))
    check_logprobs_grad(z, zg, tokens, tau, dt, r, ref, gl, gh)
    check_logprobs_grad(z, zg, tokens, tau, dt, r, ref, gl, None)
    check_logprobs_grad(z, zg, tokens, tau, dt, r, ref, None, gh)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (5, 1), (16, 8)])
def test_logprobs_strides_in_place(cuda, dt, pad, shift):
    """Rows inside a wider tensor of NaN; the gradient in place of the logits
    leaves the columns around them."""
    N, V = 9, 4099
    print(f"logprobs strides {pad} {shift} {dt}", flush=True)
    z = logits(N, V, dt, 5)
    zg = strided(z, pad, shift)
    tokens = torch.randint(0, V, (N,), generator=gen(6))
    tokens[3], tokens[4] = -100, V      # skipped rows
    r, ref = check_logprobs(z, zg, tokens, 11, 1.3, dt)
    gl, gh = torch.randn(N, generator=gen(7)), torch.randn(N, generator=gen(8))
    want = check_logprobs_grad(z, zg, tokens, 1.3, dt, r, ref, gl, gh)
    got = check_logprobs_grad(z, zg, tokens, 1.3, dt, r, ref, gl, gh, out=zg)
    assert torch.equal(got, want)
    base = zg._base
    assert torch.isnan(base[:, :shift]).all() and torch.isnan(base[:, shift + V:]).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [50, 2048, 40000])
def test_alternatives_with_ties_and_masks(cuda, dt, V):
    """Constant rows, rows of few distinct values, rows with fewer allowed ids
    than alternatives, ascending and descending rows, the largest in one run."""
    top = 40
    z = torch.zeros((8, V))
    z[1] = torch.randint(0, 3, (V,), generator=gen(1)).float()
    z[2] = -INF
    z[2, torch.randperm(V, generator=gen(2))[:7]] = torch.arange(7).float()
    z[3] = torch.arange(V).float() / 64
    z[4] = -torch.arange(V).float() / 64
    z[5, V // 2:] = 1.0
    z[6] = -INF                                             # nothing left
    z[7] = torch.finfo(TYPES[dt]).min                       # masked by the lowest value
    z[7, V // 3] = 2.0
    z[0, ::2] = -0.0                                        # -0 ranks with +0
    z = z.to(TYPES[dt])
    tokens = torch.full((8,), V // 3)
    print(f"ties {V} {dt}", flush=True)
    live = [0, 1, 2, 3, 4, 5, 7]
    r = H.himuon_token_logprobs(z.cuda(), tokens.cuda(), top=top)
    sub = type(r)(*[x[live] for x in r])
    check_logprobs(z[live], None, tokens[live], top, 1.0, dt, r=sub)
    assert r.lse[6, 0].item() == -INF and r.logp[6].item() == -INF and r.entropy[6].item() == 0.0
    assert r.top_idx[6].tolist() == list(range(top)) and torch.all(r.top_logp[6] == -INF)
    g = H.himuon_token_logprobs_grad(z.cuda(), tokens.cuda(), r.lse, r.entropy, torch.ones(8).cuda(), torch.ones(8).cuda())
    assert torch.isfinite(g).all()


def test_logprobs_nan_and_inf_stay_in_their_row(cuda):
    V = 3000
    z = logits(6, V, "fp32", 9)
    z[1, 17] = float("nan")
    z[2, 40] = INF
    z[3] = float("nan")
    z[4, 5] = float("nan")
    tokens = torch.tensor([4, 5, 6, 7, -1, 8])
    r = H.himuon_token_logprobs(z.cuda(), tokens.cuda(), top=4)
    for t in (r.logp, r.entropy, r.lse[:, 0]):
        assert torch.isnan(t[1:4]).all() and t[4].item() == 0.0 and torch.isfinite(t[[0, 5]]).all()
    keep = [0, 5]
    check_logprobs(z[keep], None, tokens[keep], 4, 1.0, "fp32", r=type(r)(*[x[keep] for x in r]))
    assert r.top_idx[2, 0].item() == 40
    assert r.top_idx[3].tolist() == [0, 1, 2, 3]
    g = H.himuon_token_logprobs_grad(z.cuda(), tokens.cuda(), r.lse, r.entropy, torch.ones(6).cuda())
    assert torch.isnan(g[1:4]).all() and torch.all(g[4] == 0) and torch.isfinite(g[keep]).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("V,top", [(600001, 64), (600001, 5), (131072, 64), (131071, 33), (40000, 64)])
def test_many_segments_and_alternatives(cuda, V, top, dt):
    """Rows of one value, of few, and masked but for some ids, next to ordinary
    ones: the alternatives are those of a stable sort, whatever the segments."""
    print(f"many segments {V} top {top} {dt}", flush=True)
    z = logits(4, V, dt, 60)
    z[1] = -2.5
    z[2] = torch.round(z[2])
    z[3] = -INF
    z[3, 17::V // 40] = 1.0
    r = H.himuon_token_logprobs(z.cuda(), top=top)
    order = torch.sort(z.float(), dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(r.top_idx.cpu().long(), order)
    s = z.double()
    want = (s - torch.logsumexp(s, 1, keepdim=True)).gather(1, order)
    _, d = row_bound(s, V)
    there = torch.isfinite(want)
    assert torch.equal(torch.isfinite(r.top_logp.cpu()), there)
    near(r.top_logp[there.cuda()], want[there], d[:, None].expand_as(want)[there], "top")


def test_logprobs_without_tokens_and_rows(cuda):
    z = logits(5, 777, "bf16", 10)
    r = H.himuon_token_logprobs(z.cuda(), top=3)
    assert r.logp is None
    full, _ = check_logprobs(z, z.cuda(), torch.zeros(5, dtype=torch.int64), 3, 1.0, "bf16")
    for a, b in ((r.entropy, full.entropy), (r.lse, full.lse), (r.top_idx, full.top_idx), (r.top_logp, full.top_logp)):
        assert torch.equal(a, b)
    e = H.himuon_token_logprobs(z.cuda()[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), top=3)
    assert e.logp.shape == (0,) and e.top_idx.shape == (0, 3)
    assert H.himuon_token_logprobs_grad(z.cuda()[:0], None, e.lse, e.entropy, None, e.entropy).shape == (0, 777)
    # entropy alone
    g = H.himuon_token_logprobs_grad(z.cuda(), None, r.lse, r.entropy, None, torch.ones(5).cuda())
    h = H.himuon_token_logprobs_grad(z.cuda(), torch.zeros(5, dtype=torch.int64).cuda(), r.lse, r.entropy, None, torch.ones(5).cuda())
    assert torch.equal(g, h)


# ---- distillation --------------------------------------------------------------------

def distill64(z, idx, t, tau, normalize, w):
    """(loss, dz, their bounds) in fp64."""
    V = z.shape[1]
    there = (idx >= 0) & (idx < V)
    u = torch.where(there, t.double() / tau if normalize else t.double(), -INF)
    if normalize:
        m = u.amax(1, keepdim=True)
        l = torch.where(m == -INF, 0.0, torch.logsumexp(u, 1, keepdim=True))
        lp = u - l
    else:
        lp = u
    p = torch.exp(lp)
    live = (w != 0) & ~(u == -INF).all(1)
    s, lse, lq, q = softmax64(z, tau)
    where = idx.long().clamp(0, V - 1)
    pick = lq.gather(1, where)
    term = torch.where(p > 0, p * (lp - pick), 0.0)
    loss = torch.where(live, w.double() * term.sum(1), 0.0)
    P = p.sum(1)
    dense = torch.zeros_like(q).scatter_add_(1, where, torch.where(there, p, 0.0))
    c = w.double() / tau
    grad = torch.where(live[:, None], c[:, None] * (P[:, None] * q - dense), 0.0)
    A, d = row_bound(s, V)
    At = torch.where(torch.isfinite(u), u.abs(), 0.0).amax(1)
    dp = 2.0 ** -20 * (At + 8) + (idx.shape[1] / 64 + 64) * 2.0 ** -24
    gap = torch.where(p > 0, (lp.abs() + pick.abs()), 0.0).amax(1)
    lb = w.double().abs() * P * (d + dp * (1 + gap))
    gb = c.abs()[:, None] * (P[:, None] * q * (d + dp)[:, None] + dense * dp[:, None])
    return loss, grad, torch.where(live, lse, 0.0), d, lb, gb


def check_distill(z, zg, idx, t, tau, normalize, w, dt):
    loss, grad, lse, d, lb, gb = distill64(z, idx, t, tau, normalize, w)
    ig, tg, wg = idx.cuda(), t.cuda(), w.cuda()
    kw = dict(temperature=tau, normalize=normalize)
    fused = H.himuon_distill(zg, ig, tg, weight=wg, grad=True, **kw)
    apart = H.himuon_distill(zg, ig, tg, weight=wg, **kw)
    g2 = H.himuon_distill_grad(zg, ig, tg, apart.lse, wg, **kw)
    torch.cuda.synchronize()
    for r in (fused, apart):
        near(r.loss, loss, lb, "loss")
        near(r.lse.double().sum(1), lse, d, "lse")
    for g in (fused.grad, g2):
        near(g, grad, gb + ROUND[dt] * grad.abs() + 1e-38, "grad")
    return fused


def teacher(N, V, k, seed, kind=torch.int64):
    idx = torch.stack([torch.randperm(V, generator=gen(seed + i))[:k] for i in range(N)]).to(kind)
    return idx, torch.randn((N, k), generator=gen(seed + 999)) * 3


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V,k", [(1, 1, 1), (2, 5, 5), (37, 1000, 8), (6, 5003, 64), (3, 32000, 100), (300, 263, 16),
                                   (2, 131072, 64), (2, 131073, 1024), (1, 200001, 7)])
@pytest.mark.parametrize("normalize", [True, False])
def test_distill(cuda, N, V, k, normalize, dt):
    print(f"distill {N}x{V} k {k} {normalize} {dt}", flush=True)
    z = logits(N, V, dt, N + V)
    idx, t = teacher(N, V, k, 50, torch.int64 if N % 2 else torch.int32)
    if not normalize:
        t = torch.log_softmax(t, 1) - 0.1
    w = torch.rand(N, generator=gen(4)) + 0.5
    check_distill(z, z.cuda(), idx, t, [1.0, 0.7, 2.0][V % 3], normalize, w, dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("V,pad,shift", [(3000, 0, 0), (4099, 3, 1), (70000, 8, 8)])
def test_distill_absent_repeated_masked(cuda, dt, V, pad, shift):
    """Absent entries, rows without any, weight 0 over a row of NaN, ids given
    more than once, p = 0, masked logits (some where the teacher has an entry),
    a strided teacher, and the gradient in place."""
    N, k = 8, 12
    z = logits(N, V, dt, 70)
    idx, t = teacher(N, V, k, 71)
    wide = torch.full((N, k + 4), float("nan"))
    wide[:, :k] = t
    idx[0, 5:] = -1
    idx[1] = V + 3
    idx[2, 3:6] = idx[2, 0]
    idx[3, :] = idx[3, 0]
    t[4, 2:] = -INF
    t[5] = -INF
    wide[:, :k] = t
    z[6, ::3] = -INF
    z[6, idx[6, 1]] = 0.5
    z[7] = float("nan")
    w = torch.ones(N)
    w[7] = 0.0
    blocked = (z[6, idx[6]] == -INF)
    idx[6, blocked] = -1
    print(f"distill special {V} {dt}", flush=True)
    zg = strided(z, pad, shift)
    tg = wide.cuda()[:, :k]
    for normalize in (True, False):
        u = t if normalize else t - 3.0
        zz = z.clone()
        zz[7] = 0.0                       # the weight makes it count nothing; 0 * NaN would spread in the reference
        loss, grad, lse, d, lb, gb = distill64(zz, idx, u, 1.5, normalize, w)
        tt = tg if normalize else tg - 3.0
        r = H.himuon_distill(zg, idx.cuda(), tt, 1.5, normalize, w.cuda(), grad=True)
        near(r.loss, loss, lb, "loss")
        near(r.grad, grad, gb + ROUND[dt] * grad.abs() + 1e-38, "grad")
        assert r.loss[[1, 5, 7]].tolist() == [0.0, 0.0, 0.0] and torch.all(r.grad[[1, 5, 7]] == 0)
        g2 = H.himuon_distill_grad(zg, idx.cuda(), tt, r.lse, w.cuda(), 1.5, normalize)
        near(g2, grad, gb + ROUND[dt] * grad.abs() + 1e-38, "grad")
    # in place, both ways
    z1, z2 = strided(z, pad, shift), strided(z, pad, shift)
    a = H.himuon_distill(z1, idx.cuda(), tg, 1.5, True, w.cuda(), grad=z1)
    assert a.grad is z1
    r = H.himuon_distill(zg, idx.cuda(), tg, 1.5, True, w.cuda(), grad=True)
    assert torch.equal(z1, r.grad) and torch.equal(a.loss, r.loss)
    H.himuon_distill_grad(z2, idx.cuda(), tg, r.lse, w.cuda(), 1.5, True, out=z2)
    assert torch.equal(z2, H.himuon_distill_grad(zg, idx.cuda(), tg, r.lse, w.cuda(), 1.5, True))
    for v in (z1, z2):
        if v._base is not None:
            assert torch.isnan(v._base[:, :shift]).all() and torch.isnan(v._base[:, shift + V:]).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("threads,chunks", [(256, 1), (256, 2), (256, 3), (256, 4), (256, 6), (256, 8), (512, 6), (512, 8),
                                            (1024, 6), (1024, 8), (1024, 12), (1024, 16), (1024, 18), (1024, 20)])
def test_distill_row_sizes(cuda, threads, chunks, dt):
    """Rows around the sizes that workgroups hold, on and off the 16-byte grid,
    the gradient on the logits' grid and on another one; nothing outside it is
    written."""
    epc = 8 if dt == "bf16" else 4
    N, full = 5, threads * chunks * epc
    for V in (full - epc, full - epc - 3, full):
        idx, t = teacher(N, V, 6, 90)
        idx[1, 0], idx[2, 0] = 0, V - 1
        z = logits(N, V, dt, 91)
        w = torch.tensor([1.0, 0.5, 2.0, 0.0, 1.0])
        loss, grad, lse, d, lb, gb = distill64(z, idx, t, 1.0, True, w)
        tol = gb + ROUND[dt] * grad.abs() + 1e-38
        for (zp, zs), (gp, gs) in (((epc, 0), (2 * epc, epc)), ((3, 1), (3, 1)), ((2, 1), (2, 1)), ((3, 1), (4, 2))):
            print(f"distill {N}x{V} logits {zp} {zs} gradient {gp} {gs} {dt}", flush=True)
            out = strided(torch.full((N, V), float("nan"), dtype=TYPES[dt]), gp, gs)
            r = H.himuon_distill(strided(z, zp, zs), idx.cuda(), t.cuda(), weight=w.cuda(), grad=out)
            near(r.loss, loss, lb, "loss")
            near(r.lse.double().sum(1)[w != 0], lse[w != 0], d[w != 0], "lse")
            near(out, grad, tol, "grad")
            assert torch.isnan(out._base[:, :gs]).all() and torch.isnan(out._base[:, gs + V:]).all()


def test_distill_extremes(cuda):
    """A masked logit under an entry gives the loss +inf and a finite gradient;
    NaN and +inf make their own row NaN; a row of the lowest value is uniform."""
    V = 2500
    z = logits(5, V, "fp32", 80)
    idx, t = teacher(5, V, 4, 81)
    z[1, idx[1, 2]] = -INF
    z[2, 9] = float("nan")
    z[3, 9] = INF
    z[4] = torch.finfo(torch.float32).min
    r = H.himuon_distill(z.cuda(), idx.cuda(), t.cuda(), grad=True)
    assert r.loss[1].item() == INF and torch.isfinite(r.grad[1]).all()
    assert torch.isnan(r.loss[2:4]).all() and torch.isnan(r.grad[2:4]).all()
    keep = [0, 4]
    zz = z.clone()
    zz[4] = 0.0
    loss, grad, lse, d, lb, gb = distill64(zz, idx, t, 1.0, True, torch.ones(5))
    near(r.loss[keep], loss[keep], lb[keep], "loss")
    near(r.grad[keep], grad[keep], (gb + ROUND["fp32"] * grad.abs())[keep] + 1e-38, "grad")


def test_distill_no_rows(cuda):
    z = torch.zeros((0, 100), device="cuda")
    r = H.himuon_distill(z, torch.zeros((0, 3), dtype=torch.int64, device="cuda"), torch.zeros((0, 3), device="cuda"), grad=True)
    assert r.loss.shape == (0,) and r.grad.shape == (0, 100)


def test_gradients_against_differences(cuda):
    """Central differences of the forward results along a direction v of unit
    entries: the third derivative of each is at most 8 times the sum of its
    weights, so the difference is off by 8 h^2 and the rounding of the two
    losses by 2 d / (2 h)."""
    N, V, h = 4, 300, 2.0 ** -6
    z = logits(N, V, "fp32", 90, scale=1.5)
    v = torch.sign(torch.randn((N, V), generator=gen(91)))
    idx, t = teacher(N, V, 6, 92)
    tol = N * (8 * h * h + 2.0 ** -15 / h)
    up, down = (z + h * v).cuda(), (z - h * v).cuda()

    def loss(x):
        return H.himuon_distill(x, idx.cuda(), t.cuda()).loss.double().sum()

    g = H.himuon_distill(z.cuda(), idx.cuda(), t.cuda(), grad=True).grad
    assert abs(float((loss(up) - loss(down)) / (2 * h)) - float((g.double().cpu() * v).sum())) <= tol
    tokens = torch.tensor([5, 17, 0, 299])
    one = torch.ones(N, device="cuda")
    r = H.himuon_token_logprobs(z.cuda(), tokens.cuda())
    for pick, args in (("logp", (one, None)), ("entropy", (None, one))):
        f = lambda x: getattr(H.himuon_token_logprobs(x, tokens.cuda()), pick).double().sum()
        g = H.himuon_token_logprobs_grad(z.cuda(), tokens.cuda(), r.lse, r.entropy, *args)
        assert abs(float((f(up) - f(down)) / (2 * h)) - float((g.double().cpu() * v).sum())) <= tol


@pytest.mark.parametrize("N,V", [(3, 100000), (600, 2048)])
def test_same_bits_streams_graph(cuda, N, V):
    z = logits(N, V, "bf16", 95).cuda()
    idx, t = teacher(N, V, 9, 96)
    idx, t = idx.cuda(), t.cuda()
    tokens = torch.randint(0, V, (N,), generator=gen(97)).cuda()
    w = torch.ones(N, device="cuda")

    def calls(stream=None):
        a = H.himuon_distill(z, idx, t, weight=w, grad=True, stream=stream)
        b = H.himuon_token_logprobs(z, tokens, top=12, stream=stream)
        c = H.himuon_token_logprobs_grad(z, tokens, b.lse, b.entropy, w, w, stream=stream)
        e = H.himuon_distill_grad(z, idx, t, a.lse, w, stream=stream)
        return [*a, *b, c, e]

    ref = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        got = calls(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for k in range(3):
        z.copy_(logits(N, V, "bf16", 100 + k))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(calls(), got))


# ---- logits of large magnitude ---------------------------------------------------------
# Differences of equal logits are exactly zero whatever their size, and the next
# other value of the rows below is so far off that its q is 0 in fp32.  So q is
# 1 / n over the n largest, and the bounds are those of a row with A = 0.
FAR = {"-1e9": -1e9, "1e9": 1e9, "lowest": None}


def far_rows(V, dt, base):
    """All at base; one id far above; two values, the larger one on a third of
    the ids (both past fp32's range under a temperature below 1 for the lowest
    value); base among -inf; an ordinary row."""
    low = torch.finfo(TYPES[dt]).min
    b = low if base is None else base
    z = torch.full((5, V), b)
    z[1, V // 2] = 2.0 if b < 0 else 1.5 * b
    z[2] = b * (0.875 if b < 0 else 1.25)
    z[2, torch.arange(V) % 3 != 0] = b
    z[3, torch.arange(V) % 7 != 0] = -INF
    z[4] = torch.randn(V, generator=gen(200)) * 3
    return z.to(TYPES[dt])


def far_softmax(z, tau):
    """log q and q in fp64, from differences."""
    x = z.double()
    s = (x - x.amax(1, keepdim=True)) / tau
    lq = s - torch.logsumexp(s, 1, keepdim=True)
    return lq, torch.exp(lq)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("tau", [0.7, 1.0, 1.5])
@pytest.mark.parametrize("base", list(FAR))
@pytest.mark.parametrize("V", [1000, 40001])
def test_gradients_of_far_logits(cuda, V, base, tau, dt):
    print(f"far logits {V} {base} {tau} {dt}", flush=True)
    z = far_rows(V, dt, FAR[base])
    N, k = z.shape[0], 4
    zg = z.cuda()
    lq, q = far_softmax(z, tau)
    d = 2.0 ** -20 * (8 + math.log(V) + 40) + (V / 64 + 64) * 2.0 ** -24   # 40: the ordinary row's s
    # entries among the largest logits of each row (other losses are as large as the logits)
    best = torch.sort(z.float(), dim=1, descending=True, stable=True).indices[:, :k]
    best[1, 1:] = -1
    t = torch.randn((N, k), generator=gen(201))
    w = torch.rand(N, generator=gen(202)) + 0.5
    there = best >= 0
    u = torch.where(there, t.double() / tau, -INF)
    lp = torch.log_softmax(u, 1)
    p = torch.exp(lp)
    pick = lq.gather(1, best.clamp(min=0))
    loss = w.double() * torch.where(there, p * (lp - pick), 0.0).sum(1)
    dp = 2.0 ** -20 * 16 + 65 * 2.0 ** -24
    gap = torch.where(there, lp.abs() + pick.abs(), 0.0).amax(1)
    lb = w.double() * (d + dp * (1 + gap))
    dense = torch.zeros_like(q).scatter_add_(1, best.clamp(min=0), torch.where(there, p, 0.0))
    c = (w.double() / tau)[:, None]
    grad = c * (q - dense)
    gb = c * (q * (d + dp) + dense * dp) + ROUND[dt] * grad.abs() + 1e-38
    args = (zg, best.cuda(), t.cuda())
    fused = H.himuon_distill(*args, tau, weight=w.cuda(), grad=True)
    apart = H.himuon_distill(*args, tau, weight=w.cuda())
    g2 = H.himuon_distill_grad(*args, apart.lse, w.cuda(), tau)
    in_place = zg.clone()
    H.himuon_distill_grad(in_place, best.cuda(), t.cuda(), apart.lse, w.cuda(), tau, out=in_place)
    assert torch.equal(in_place, g2)
    for r in (fused, apart):
        near(r.loss, loss, lb, "loss")
        assert torch.isfinite(r.lse).all()
    near(fused.grad, grad, gb, "fused gradient")
    near(g2, grad, gb, "gradient")

    tokens = best[:, 0].clone()
    r = H.himuon_token_logprobs(zg, tokens.cuda(), top=4, temperature=tau)
    Hq = -torch.where(q > 0, q * lq, 0.0).sum(1)
    dH = d * (8 + math.log(V) + 40)
    near(r.logp, lq.gather(1, tokens[:, None])[:, 0], d, "logp")
    near(r.entropy, Hq, dH, "entropy")
    gl, gh = torch.randn(N, generator=gen(203)), torch.randn(N, generator=gen(204))
    hot = torch.zeros_like(q)
    hot[torch.arange(N), tokens] = 1.0
    qlq = torch.where(q > 0, q * lq, 0.0)
    for a, b in ((gl, gh), (gl, None), (None, gh)):
        got = H.himuon_token_logprobs_grad(zg, tokens.cuda(), r.lse, r.entropy, None if a is None else a.cuda(),
                                           None if b is None else b.cuda(), temperature=tau)
        A = torch.zeros(N).double() if a is None else a.double()
        B = torch.zeros(N).double() if b is None else b.double()
        want = (A[:, None] * (hot - q) - B[:, None] * (qlq + q * Hq[:, None])) / tau
        err = (A.abs()[:, None] * (q * d + 2.0 ** -22 * (hot + q))
               + B.abs()[:, None] * (q * (d + dH) + (qlq.abs() + q * Hq[:, None]) * (d + 2.0 ** -21))) / tau
        near(got, want, err + ROUND[dt] * want.abs() + 1e-38, "gradient of logp and entropy")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [700, 60000])
def test_teacher_without_probability(cuda, V, dt):
    """Teacher's log probabilities whose exponentials are 0 in fp32: the row has
    no entry with p > 0 and counts nothing, whatever its logits are; next to an
    entry that counts they add nothing."""
    print(f"teacher without probability {V} {dt}", flush=True)
    N, k = 6, 5
    z = logits(N, V, dt, 210)
    z[1, 7] = float("nan")
    z[2, 7] = INF
    z[3] = -INF
    idx, t = teacher(N, V, k, 211)
    t = torch.log_softmax(t, 1)
    t[:4] = torch.tensor([-200.0, -1e4, -1e30, -INF, -150.0])
    t[4, 2:] = -300.0
    w = torch.ones(N)
    args = (z.cuda(), idx.cuda(), t.cuda(), 1.0, False)
    fused = H.himuon_distill(*args, w.cuda(), grad=True)
    apart = H.himuon_distill(*args, w.cuda())
    g2 = H.himuon_distill_grad(z.cuda(), idx.cuda(), t.cuda(), apart.lse, w.cuda(), 1.0, False)
    loss, grad, lse, d, lb, gb = distill64(z[4:], idx[4:], t[4:], 1.0, False, w[4:])
    for r, g in ((fused, fused.grad), (apart, g2)):
        assert torch.all(r.loss[:4] == 0) and torch.all(r.lse[:4] == 0) and torch.all(g[:4] == 0)
        near(r.loss[4:], loss, lb, "loss")
        near(r.lse[4:].double().sum(1), lse, d, "lse")
        near(g[4:], grad, gb + ROUND[dt] * grad.abs() + 1e-38, "grad")


@pytest.mark.parametrize("shift", [0, 1])
def test_more_rows_than_a_launch_holds(cuda, shift):
    """A row a workgroup of 256 threads: 2^24 rows and a few take two launches,
    whose results and skipped rows meet where the first ends."""
    N, V, cut = (1 << 24) + 300, 8, (1 << 24) - 1
    print(f"{N} rows, shift {shift}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(220)
    z = torch.randn((N, V + shift), generator=g, device="cuda").bfloat16()[:, shift:]
    tokens = torch.randint(0, V, (N,), generator=g, device="cuda")
    tokens[cut + 1], tokens[cut + 7] = -1, V
    idx = torch.randint(0, V, (N, 1), generator=g, device="cuda")
    t = torch.rand((N, 1), generator=g, device="cuda") - 1.0
    gl, gh = torch.randn(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
    r = H.himuon_token_logprobs(z, tokens, top=2)
    dz = H.himuon_token_logprobs_grad(z, tokens, r.lse, r.entropy, gl, gh)
    a = H.himuon_distill(z, idx, t, normalize=False, weight=gl)
    da = H.himuon_distill_grad(z, idx, t, a.lse, gl, normalize=False)
    f = H.himuon_distill(z, idx, t, normalize=False, weight=gl, grad=True)
    torch.cuda.synchronize()
    for rows in (slice(0, 1000), slice(cut - 500, cut + 500), slice(N - 200, N)):
        zz, tk, ll, hh = z[rows].cpu(), tokens[rows].cpu(), gl[rows].cpu(), gh[rows].cpu()
        part = type(r)(*[x[rows] for x in r])
        _, ref = check_logprobs(zz, None, tk, 2, 1.0, "bf16", r=part)
        want = H.himuon_token_logprobs_grad(z[rows], tokens[rows], part.lse.contiguous(), part.entropy.contiguous(),
                                            gl[rows], gh[rows])
        assert torch.equal(dz[rows], want)
        check_logprobs_grad(zz, z[rows], tk, 1.0, "bf16", part, ref, ll, hh)
        loss, grad, lse, d, lb, gb = distill64(zz, idx[rows].cpu(), t[rows].cpu(), 1.0, False, ll)
        for res, dres in ((a, da), (f, f.grad)):
            near(res.loss[rows], loss, lb, "loss")
            near(res.lse[rows].double().sum(1), lse, d, "lse")
            near(dres[rows], grad, gb + ROUND["bf16"] * grad.abs() + 1e-38, "grad")


# ---- sizes at which a workgroup takes several rows, or long segments ----------------------
# Every row against fp64 on the GPU, in blocks of rows.
def on_gpu(got, want, bound, what):
    got = got.double()
    ok = (got == want) | (torch.isnan(got) & torch.isnan(want)) | ((got - want).abs() <= bound)
    assert torch.all(ok), (what, float(torch.where(ok, 0.0, (got - want).abs() - bound).nan_to_num(9e99).max()))


def gpu_logits(N, V, dt, seed, shift):
    """(logits on the GPU inside a wider tensor of NaN if shift, else contiguous)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.full((N, V + 2 * shift), float("nan"), dtype=TYPES[dt], device="cuda")[:, shift:shift + V]
    for r in range(0, N, 256):
        z[r:r + 256] = torch.randn((min(256, N - r), V), generator=g, device="cuda") * 3
    return z, g


def gpu_teacher(N, V, k, g):
    """Ids spread over the row, all different; some absent."""
    at = torch.rand((N, k), generator=g, device="cuda")
    idx = ((torch.arange(k, device="cuda") + at) * (V / k)).long().clamp(max=V - 1)
    idx[torch.rand((N, k), generator=g, device="cuda") < 0.1] = -1
    idx[::11] = V
    return idx, torch.randn((N, k), generator=g, device="cuda") * 3


def gpu_weights(N, g):
    w = torch.rand(N, generator=g, device="cuda") + 0.5
    w[torch.arange(N, device="cuda") % 7 == 3] = 0.0
    return w


@pytest.mark.parametrize("N,V,dt,shift,out_shift", [
    (700, 70000, "bf16", 0, 0), (700, 70001, "bf16", 1, 1), (700, 70001, "bf16", 1, 2), (600, 131072, "bf16", 0, 0),
    (600, 40000, "fp32", 0, 0), (600, 40003, "fp32", 1, 1), (600, 40003, "fp32", 1, 2),
    (5000, 1003, "bf16", 1, 1), (5000, 3000, "bf16", 0, 0), (5000, 1003, "fp32", 1, 2), (5000, 3000, "fp32", 0, 0)])
def test_distill_several_rows_a_workgroup(cuda, N, V, dt, shift, out_shift):
    """More rows than workgroups: rows of weight 0 over NaN and rows without an
    entry between the others, apart and in place."""
    print(f"several rows {N}x{V} {dt} {shift} {out_shift}", flush=True)
    z, g = gpu_logits(N, V, dt, 300 + N, shift)
    idx, t = gpu_teacher(N, V, 9, g)
    w = gpu_weights(N, g)
    z[w == 0] = float("nan")
    out = torch.full((N, V + 2 * out_shift), float("nan"), dtype=TYPES[dt], device="cuda")[:, out_shift:out_shift + V]
    r = H.himuon_distill(z, idx, t, 1.5, weight=w, grad=out)
    torch.cuda.synchronize()
    for r0 in range(0, N, 200):
        rows = slice(r0, min(N, r0 + 200))
        zz = torch.where((w[rows] == 0)[:, None], torch.zeros((), dtype=z.dtype, device="cuda"), z[rows])
        loss, grad, lse, d, lb, gb = distill64(zz, idx[rows], t[rows], 1.5, True, w[rows])
        on_gpu(r.loss[rows], loss, lb, "loss")
        on_gpu(r.lse[rows].double().sum(1), lse, d, "lse")
        on_gpu(out[rows], grad, gb + ROUND[dt] * grad.abs() + 1e-38, "gradient")
    base = out._base
    assert torch.isnan(base[:, :out_shift]).all() and torch.isnan(base[:, out_shift + V:]).all()
    if shift == out_shift:
        again = H.himuon_distill(z, idx, t, 1.5, weight=w, grad=z)
        assert torch.equal(z, out) and torch.equal(again.loss, r.loss) and torch.equal(again.lse, r.lse)
        base = z._base
        assert torch.isnan(base[:, :shift]).all() and torch.isnan(base[:, shift + V:]).all()


LONG = [(1100, 16000, "bf16", 0), (600, 16000, "bf16", 0), (1100, 20001, "bf16", 1), (1100, 8000, "fp32", 0),
        (600, 8000, "fp32", 0), (1100, 20001, "fp32", 1), (1030, 70000, "bf16", 0)]


@pytest.mark.parametrize("top", [0, 5, 40])
@pytest.mark.parametrize("N,V,dt,shift", LONG)
def test_logprobs_of_long_segments(cuda, N, V, dt, shift, top):
    """Segments of four and eight chunks a thread: rows of one value, of few,
    ascending and descending, masked but for some ids, low in the chunks of one
    wave (the others' all lie above its bound), and ordinary ones."""
    print(f"long segments {N}x{V} {dt} {shift} top {top}", flush=True)
    z, g = gpu_logits(N, V, dt, 400 + N, shift)
    v = torch.arange(V, device="cuda")
    epc = 8 if dt == "bf16" else 4
    for r in (1, 333, N - 1):   # (each kind in several rows)
        z[r] = -2.5
    z[2] = torch.round(z[2])
    z[4], z[5] = v / 64, -(v / 64)
    z[6] = -INF
    z[6, 17::V // 60] = 1.0
    z[7] = torch.finfo(TYPES[dt]).min
    z[7, V // 3] = 2.0
    for r in (8, N // 2):
        z[r] = torch.where(v // epc % 256 < 64, z[r].float() - 50.0, z[r].float())
    z[9] = (v * 37 % 1009) / 16
    tokens = torch.randint(0, V, (N,), generator=g, device="cuda")
    tokens[6] = 17
    tokens[torch.arange(N, device="cuda") % 13 == 3] = -1
    tau = 1.3
    r = H.himuon_token_logprobs(z, tokens, top=top, temperature=tau)
    gl, gh = torch.randn(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
    dz = H.himuon_token_logprobs_grad(z, tokens, r.lse, r.entropy, gl, gh, temperature=tau)
    torch.cuda.synchronize()
    for r0 in range(0, N, 200):
        rows = slice(r0, min(N, r0 + 200))
        zz, tok = z[rows], tokens[rows]
        live = tok >= 0
        s, lse, lq, q = softmax64(zz, tau)
        # (logits masked by the lowest value: their q is 0, and their own log q
        # carries the relative error of s)
        A, d = row_bound(torch.where(s < -1e30, 0.0, s), V)
        ids = tok.clamp(min=0)[:, None]
        own = torch.where(lq < -1e30, 2.0 ** -20 * lq.abs(), 0.0)
        on_gpu(r.logp[rows], torch.where(live, lq.gather(1, ids)[:, 0], 0.0), d + own.gather(1, ids)[:, 0], "logp")
        qlq = torch.where(q > 0, q * lq, 0.0)
        Hq = -qlq.sum(1)
        dH = d * (2 * A + 8 + math.log(V))
        on_gpu(r.entropy[rows], torch.where(live, Hq, 0.0), dH, "entropy")
        on_gpu(r.lse[rows].double().sum(1), torch.where(live, lse, 0.0), d, "lse")
        if top:
            order = torch.sort(zz.float(), dim=1, descending=True, stable=True).indices[:, :top]
            assert torch.equal(r.top_idx[rows].long()[live], order[live])
            got = r.top_logp[rows].double()
            on_gpu(got[live], lq.gather(1, order)[live], (d[:, None] + own.gather(1, order))[live], "alternatives")
            assert torch.all(r.top_idx[rows][~live] == -1) and torch.all(got[~live] == -INF)
        a, b = torch.where(live, gl[rows], 0.0).double()[:, None], torch.where(live, gh[rows], 0.0).double()[:, None]
        hot = torch.zeros_like(q).scatter_(1, ids, 1.0)
        want = (a * (hot - q) - b * (qlq + q * Hq[:, None])) / tau
        # (a q below 2^-126 may be 0, and |q log q| is below 88 2^-126 there)
        err = (a.abs() * (q * d[:, None] + 2.0 ** -22 * (hot + q) + 2.0 ** -126)
               + b.abs() * (q * (d + dH)[:, None] + (qlq.abs() + q * Hq[:, None].abs()) * (d[:, None] + 2.0 ** -21)
                            + 2.0 ** -126 * (88 + Hq[:, None]))) / tau
        on_gpu(dz[rows], want, err + ROUND[dt] * want.abs() + 1e-38, "gradient")
    H.himuon_token_logprobs_grad(z, tokens, r.lse, r.entropy, gl, gh, temperature=tau, out=z)
    assert torch.equal(z, dz)


@pytest.mark.parametrize("N,V,dt,shift", LONG)
def test_distill_of_long_segments_in_two_calls(cuda, N, V, dt, shift):
    """The loss, and from its lse the gradient, apart and in place."""
    print(f"two calls {N}x{V} {dt} {shift}", flush=True)
    z, g = gpu_logits(N, V, dt, 500 + N, shift)
    w = gpu_weights(N, g)
    z[w == 0] = float("nan")
    for k in (9, 70):
        idx, t = gpu_teacher(N, V, k, g)
        t = torch.log_softmax(t, 1) - 0.1
        r = H.himuon_distill(z, idx, t, 0.7, False, w)
        dz = H.himuon_distill_grad(z, idx, t, r.lse, w, 0.7, False)
        for r0 in range(0, N, 200):
            rows = slice(r0, min(N, r0 + 200))
            zz = torch.where((w[rows] == 0)[:, None], torch.zeros((), dtype=z.dtype, device="cuda"), z[rows])
            loss, grad, lse, d, lb, gb = distill64(zz, idx[rows], t[rows], 0.7, False, w[rows])
            on_gpu(r.loss[rows], loss, lb, "loss")
            on_gpu(r.lse[rows].double().sum(1), lse, d, "lse")
            on_gpu(dz[rows], grad, gb + ROUND[dt] * grad.abs() + 1e-38, "gradient")
    H.himuon_distill_grad(z, idx, t, r.lse, w, 0.7, False, out=z)
    assert torch.equal(z, dz)


@pytest.mark.parametrize("V", [131072, 131073])
def test_logits_past_2_to_the_32_elements(cuda, V):
    """Rows whose offsets pass 32 bits, in bytes and in elements, on and off the
    16-byte grid, the gradients in place: sampled rows against fp64."""
    N, k = 33000, 5
    print(f"{N}x{V}", flush=True)
    assert N * V > 1 << 32
    z, g = gpu_logits(N, V, "bf16", 600, 0)
    rows = torch.tensor([0, 16383, 16384, 32767, 32768, N - 2, N - 1], device="cuda")
    zz = z[rows].cpu()
    idx, t = gpu_teacher(N, V, k, g)
    tokens = torch.randint(0, V, (N,), generator=g, device="cuda")
    w = torch.rand(N, generator=g, device="cuda") + 0.5
    r = H.himuon_token_logprobs(z, tokens, top=3)
    part = type(r)(*[x[rows] for x in r])
    _, ref = check_logprobs(zz, None, tokens[rows].cpu(), 3, 1.0, "bf16", r=part)
    loss, grad, lse, d, lb, gb = distill64(zz, idx[rows].cpu(), t[rows].cpu(), 1.0, True, w[rows].cpu())
    a = H.himuon_distill(z, idx, t, weight=w)
    near(a.loss[rows], loss, lb, "loss")
    kept = z.clone()
    H.himuon_distill_grad(kept, idx, t, a.lse, w, out=kept)
    near(kept[rows], grad, gb + ROUND["bf16"] * grad.abs() + 1e-38, "gradient")
    kept.copy_(z)
    f = H.himuon_distill(kept, idx, t, weight=w, grad=kept)
    near(f.loss[rows], loss, lb, "fused loss")
    near(kept[rows], grad, gb + ROUND["bf16"] * grad.abs() + 1e-38, "fused gradient")
    gl, gh = torch.randn(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
    want = H.himuon_token_logprobs_grad(z[rows], tokens[rows], part.lse.contiguous(), part.entropy.contiguous(), gl[rows], gh[rows])
    check_logprobs_grad(zz, z[rows], tokens[rows].cpu(), 1.0, "bf16", part, ref, gl[rows].cpu(), gh[rows].cpu())
    H.himuon_token_logprobs_grad(z, tokens, r.lse, r.entropy, gl, gh, out=z)
    assert torch.equal(z[rows], want)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [3000, 170001, 170008])
def test_distill_without_weights_or_lse(cuda, V, dt):
    """No weights are weights of 1, and no lse wanted changes nothing else,
    whether a row is kept on chip or read twice."""
    print(f"distill without weights {V} {dt}", flush=True)
    N, k = 5, 6
    z = logits(N, V, dt, 700)
    idx, t = teacher(N, V, k, 701)
    idx[2] = -1
    zg, ig, tg = z.cuda(), idx.cuda(), t.cuda()
    loss, grad, lse, d, lb, gb = distill64(z, idx, t, 1.5, True, torch.ones(N))
    tol = gb + ROUND[dt] * grad.abs() + 1e-38
    r = H.himuon_distill(zg, ig, tg, 1.5, grad=True)
    near(r.loss, loss, lb, "loss")
    near(r.lse.double().sum(1), lse, d, "lse")
    near(r.grad, grad, tol, "grad")
    ones = H.himuon_distill(zg, ig, tg, 1.5, weight=torch.ones(N, device="cuda"), grad=True)
    assert torch.equal(ones.loss, r.loss) and torch.equal(ones.grad, r.grad)
    in_place = zg.clone()
    H.himuon_distill(in_place, ig, tg, 1.5, grad=in_place)
    assert torch.equal(in_place, r.grad)
    # the C entry without lse
    got, l2 = torch.empty_like(zg), torch.empty(N, device="cuda")
    ws = torch.empty(max(H.himuon_distill_workspace(zg, True), 16), dtype=torch.uint8, device="cuda")
    dz, do, dt_ = H._rows(zg), H._rows(got), H._rows(tg)
    at = lambda x: ctypes.c_void_p(x.data_ptr())
    code = H.lib.himuon_distill(ctypes.byref(dz), at(ig), H.I64, ctypes.byref(dt_), 1.5, 1, None, at(l2), None,
                                ctypes.byref(do), H._dtype_code(zg), at(ws), ws.numel(),
                                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert code == 0 and torch.equal(got, r.grad) and torch.equal(l2, r.loss)


@pytest.mark.parametrize("V", [1000, 60000])
def test_logprobs_optional_results(cuda, V):
    """Each result of the C entry may be left out; the others stay the same."""
    N, top = 6, 4
    print(f"optional results {V}", flush=True)
    zg = logits(N, V, "bf16", 710).cuda()
    tokens = torch.randint(0, V, (N,), generator=gen(711)).cuda()
    tokens[2] = -1
    want = H.himuon_token_logprobs(zg, tokens, top=top)
    ws = torch.empty(max(H.himuon_token_logprobs_workspace(zg, top), 16), dtype=torch.uint8, device="cuda")
    dz = H._rows(zg)
    for left_out in range(4):
        res = [torch.full_like(x, 7) for x in want]
        at = [None if i == left_out else ctypes.c_void_p(x.data_ptr()) for i, x in enumerate(res)]
        code = H.lib.himuon_token_logprobs(ctypes.byref(dz), ctypes.c_void_p(tokens.data_ptr()), H.I64, 1.0,
                                           0 if left_out == 3 else top, at[0], at[1], at[2], at[3],
                                           None if left_out == 3 else at[4], H.BF16, ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                           ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert code == 0
        for i, (x, y) in enumerate(zip(res, want)):
            if i == left_out or (left_out == 3 and i == 4):
                assert torch.all(x == 7)
            else:
                assert torch.equal(x, y)
