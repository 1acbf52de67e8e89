"""What is measured of the operators around the optimiser step: the experts' products (forward, input gradient, weight
gradient), distillation from a teacher's top logits, and log probabilities of given tokens.

Where `own` is false, `run` computes them from elementary torch operations in 32 bits; where it is true, through
tiled_newton_schulz_amd.  Shapes come from this repository's mixture-of-experts workload (64 experts of 4096 x 1408 and
1408 x 4096), its smaller matrices, and generic vocabulary sizes.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}

# Every listed and drawn case of the experts' products stays below these.
MOST_FLOPS = 2 * 32768 * 4096 * 1408
MOST_WEIGHTS = 64 * 4096 * 1408
# ... and of the two losses.
MOST_LOGITS = 2048 * 131072


def listed():
    return [
        # a small experiment's layer, a handful of tokens: launch latency
        dict(name="mm_small", op="mm", dtype="bf16", experts=8, rows=40, inner=512, cols=256, stored="kn"),
        # a few dozen tokens decoded through the 64 experts: one or two rows an expert, the weights' bytes count
        dict(name="mm_decode", op="mm", dtype="bf16", experts=64, rows=96, inner=4096, cols=1408, stored="kn"),
        # the up product of one training step, weights kept as the optimiser holds them
        dict(name="mm_up", op="mm", dtype="bf16", experts=64, rows=16384, inner=4096, cols=1408, stored="kn"),
        # the gradient of that product's input: the same weights read transposed
        dict(name="mm_dgrad", op="mm", dtype="bf16", experts=64, rows=32768, inner=1408, cols=4096, stored="nk"),
        # the gradient of those weights, which the Muon step takes
        dict(name="mm_wgrad", op="wgrad", dtype="bf16", experts=64, rows=32768, inner=4096, cols=1408, stored="kn"),
        # fp32 experts of odd sizes (rows that start off any alignment)
        dict(name="wgrad_fp32_odd", op="wgrad", dtype="fp32", experts=6, rows=1001, inner=515, cols=261, stored="kn"),
        # a short test run's distillation: few rows, small odd vocabulary, fp32
        dict(name="distill_small", op="distill", dtype="fp32", rows=37, vocab=5003, entries=8, temperature=2.0,
             normalize=True, fused=True),
        # one micro-batch against stored teacher logits, loss and gradient in one call
        dict(name="distill_train", op="distill", dtype="bf16", rows=2048, vocab=131072, entries=64, temperature=1.0,
             normalize=True, fused=True),
        # forward and backward as two calls, the teacher's probabilities taken as they stand
        dict(name="distill_two_calls", op="distill", dtype="bf16", rows=2048, vocab=32000, entries=32, temperature=1.5,
             normalize=False, fused=False),
        # a server answers four sequences with 20 alternatives for each token: latency
        dict(name="logprobs_decode", op="logprobs", dtype="bf16", rows=4, vocab=131072, top=20, temperature=0.7,
             backward=False),
        # a long prompt scored at an odd vocabulary, five alternatives each
        dict(name="logprobs_score", op="logprobs", dtype="bf16", rows=4000, vocab=65537, top=5, temperature=1.0,
             backward=False),
        # a policy-gradient step: log probabilities and entropy, and the gradient of the logits through both
        dict(name="logprobs_policy", op="logprobs", dtype="fp32", rows=1024, vocab=65536, top=0, temperature=1.0,
             backward=True),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["mm", "mm", "wgrad", "distill", "logprobs"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("mm", "wgrad"):
        # fp32 products are a sixteenth as fast: less work
        flops = MOST_FLOPS if dtype == "bf16" else MOST_FLOPS // 16
        while True:
            experts = _spread(rng, 1, 96)
            rows = _spread(rng, 1, 32768)
            inner, cols = _spread(rng, 32, 4096), _spread(rng, 32, 4096)
            if rng.random() < 0.6:   # most widths are multiples of eight, some are odd
                inner, cols = 8 * max(1, inner // 8), 8 * max(1, cols // 8)
            if 3072 in (experts, rows, inner, cols):
                continue
            if 2 * rows * inner * cols <= flops and experts * inner * cols <= MOST_WEIGHTS:
                return dict(op=op, dtype=dtype, experts=experts, rows=rows, inner=inner, cols=cols,
                            stored=rng.choice(["kn", "nk"]) if op == "mm" else "kn")
    while True:
        rows, vocab = _spread(rng, 1, 4096), _spread(rng, 1000, 160000)
        if rng.random() < 0.6:
            vocab = 8 * (vocab // 8)
        if rows * vocab * BYTES[dtype] <= 2 * MOST_LOGITS and 3072 not in (rows, vocab):
            break
    temperature = rng.choice([1.0, 1.0, 0.7, 2.0])
    if op == "distill":
        return dict(op=op, dtype=dtype, rows=rows, vocab=vocab, entries=_spread(rng, 1, 128), temperature=temperature,
                    normalize=rng.random() < 0.7, fused=rng.random() < 0.6)
    backward = rng.random() < 0.4
    return dict(op=op, dtype=dtype, rows=rows, vocab=vocab, top=0 if backward else rng.choice([0, 1, 5, 20, 64]),
                temperature=temperature, backward=backward)


# ---- inputs ------------------------------------------------------------------------------------

def _counts(case):
    """Rows of each expert, before they are shuffled: a router's uneven choice, some experts without a row."""
    rng = random.Random(case["experts"] * 1000003 + case["rows"])
    share = [rng.gammavariate(2.0, 1.0) if rng.random() > 0.05 else 0.0 for _ in range(case["experts"])]
    if sum(share) == 0.0:
        share[0] = 1.0
    total, out, left = sum(share), [], 0.0
    for s in share:   # largest whole parts first, the rest carried on, so the sum is exact
        left += s * case["rows"] / total
        c = int(left + 1e-9)
        out.append(c)
        left -= c
    out[max(range(len(out)), key=lambda i: share[i])] += case["rows"] - sum(out)
    return out


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(gen, shape, dtype, scale=1.0):
    t = torch.empty(shape, dtype=TYPES[dtype], device="cuda")
    t.normal_(generator=gen)
    return t.mul_(scale) if scale != 1.0 else t


def prepare(case, seed):
    gen = _generator(seed)
    state = {"case": case}
    if case["op"] in ("mm", "wgrad"):
        counts = _counts(case)
        random.Random(int(seed)).shuffle(counts)
        n, m, k, c = case["experts"], case["rows"], case["inner"], case["cols"]
        state["counts"] = counts
        state["ends"] = torch.tensor(counts, device="cuda").cumsum(0).to(torch.int32)
        state["x"] = _normal(gen, (m, k), case["dtype"])
        if case["op"] == "mm":
            # weights [inner, cols] of every expert, stored that way or transposed
            shape = (n, k, c) if case["stored"] == "kn" else (n, c, k)
            w = _normal(gen, shape, case["dtype"], 1.0 / math.sqrt(k))
            state["w"] = w if case["stored"] == "kn" else w.transpose(1, 2)
        else:
            state["dy"] = _normal(gen, (m, c), case["dtype"], 0.1)
        if own:
            import tiled_newton_schulz_amd as himuon
            state["himuon"] = himuon
            if case["op"] == "mm":
                state["experts"] = himuon.matrices(state["w"])
        return state

    n, v = case["rows"], case["vocab"]
    z = _normal(gen, (n, v), case["dtype"], 2.5)
    # some ids that no text uses are ruled out in every row
    z[:, torch.randint(0, v, (max(1, v // 500),), generator=gen, device="cuda")] = float("-inf")
    state["z"] = z
    # the token that came next: mostly a likely one, so raise it
    tokens = torch.randint(0, v, (n,), generator=gen, device="cuda")
    z.scatter_(1, tokens[:, None], 9.0)
    if case["op"] == "distill":
        k = case["entries"]
        # the teacher's top entries, best first; a row holds fewer where the rest was cut off (-1)
        idx = torch.rand((n, k), generator=gen, device="cuda")
        idx = ((torch.arange(k, device="cuda") + idx) * (v / k)).to(torch.int64).clamp_(0, v - 1)
        z.scatter_(1, idx, 4.0 + torch.rand((n, k), generator=gen, device="cuda").to(z.dtype))
        t = (torch.rand((n, k), generator=gen, device="cuda") * 8.0).sort(dim=1, descending=True)[0]
        if not case["normalize"]:   # log probabilities whose sum stays below one
            t = t - t.exp().sum(1, keepdim=True).log() - 0.05
        kept = torch.randint(1, k + 1, (n, 1), generator=gen, device="cuda")
        full = torch.rand((n, 1), generator=gen, device="cuda") < 0.9
        cut = (torch.arange(k, device="cuda")[None] >= kept) & ~full
        state["idx"] = idx.masked_fill(cut, -1).to(torch.int32)
        state["t"] = t.contiguous()
        # rows of the prompt or the padding count nothing
        weight = torch.rand((n,), generator=gen, device="cuda") + 0.5
        weight[torch.rand((n,), generator=gen, device="cuda") < 0.05] = 0.0
        state["weight"] = weight / n
    else:
        # a negative id marks a row that is not scored
        tokens[torch.rand((n,), generator=gen, device="cuda") < 0.02] = -1
        state["tokens"] = tokens
        if case["backward"]:
            state["g_logp"] = torch.randn((n,), generator=gen, device="cuda") / n
            state["g_entropy"] = torch.full((n,), -0.01 / n, device="cuda")
    if own:
        import tiled_newton_schulz_amd as himuon
        state["himuon"] = himuon
    return state


# ---- the operators in their plain form ------------------------------------------------------------

def _plain_mm(state):
    x, w, counts = state["x"], state["w"], state["counts"]
    parts, r = [], 0
    for e, c in enumerate(counts):
        if c:
            parts.append(x[r:r + c].float() @ w[e].float())
        r += c
    return torch.cat(parts).to(x.dtype)


def _plain_wgrad(state):
    x, dy, counts = state["x"], state["dy"], state["counts"]
    out = torch.zeros((len(counts), x.shape[1], dy.shape[1]), dtype=x.dtype, device=x.device)
    r = 0
    for e, c in enumerate(counts):
        if c:
            out[e] = x[r:r + c].float().t() @ dy[r:r + c].float()
        r += c
    return out


def _plain_softmax(z, temperature):
    s = z.float() / temperature
    m = s.amax(dim=1, keepdim=True)
    e = torch.exp(s - m)
    total = e.sum(dim=1, keepdim=True)
    return s, e / total, m + torch.log(total)


def _plain_distill(state):
    case, z = state["case"], state["z"]
    s, q, lse = _plain_softmax(z, case["temperature"])
    there = state["idx"] >= 0
    idx = state["idx"].long().clamp(min=0)
    if case["normalize"]:
        u = (state["t"] / case["temperature"]).masked_fill(~there, float("-inf"))
        u = u - u.amax(dim=1, keepdim=True)
        logp = u - torch.log(torch.exp(u).sum(dim=1, keepdim=True))
    else:
        logp = state["t"].masked_fill(~there, float("-inf"))
    p = torch.exp(logp)
    terms = p * (logp - (s.gather(1, idx) - lse))
    loss = torch.where(there & (p > 0), terms, torch.zeros_like(terms)).sum(dim=1) * state["weight"]
    scale = (state["weight"] / case["temperature"])[:, None]
    grad = q.mul_(p.sum(dim=1, keepdim=True) * scale)
    grad.scatter_add_(1, idx, -(p * scale))
    grad = torch.where(state["weight"][:, None] != 0, grad, torch.zeros_like(grad))
    return loss, grad.to(z.dtype)


def _plain_logprobs(state):
    case, z, tokens = state["case"], state["z"], state["tokens"]
    live = tokens >= 0
    ids = tokens.clamp(min=0)[:, None]
    s, q, lse = _plain_softmax(z, case["temperature"])
    logq = s - lse
    zero = torch.zeros((), device=z.device)
    weighted = torch.where(q > 0, q * logq, zero)
    entropy = torch.where(live, -weighted.sum(dim=1), zero)
    logp = torch.where(live, logq.gather(1, ids)[:, 0], zero)
    out = {"logp": logp, "entropy": entropy}
    if case["top"]:
        best, where = [], []
        order = torch.arange(z.shape[1], device=z.device)
        rest = z.float().clone()
        taken = torch.zeros_like(rest, dtype=torch.bool)
        for _ in range(case["top"]):   # the largest left, the lowest id among equals
            top = rest.amax(dim=1, keepdim=True)
            i = torch.where((rest == top) & ~taken, order, z.shape[1]).amin(dim=1, keepdim=True)
            best.append(logq.gather(1, i))
            where.append(i)
            rest.scatter_(1, i, float("-inf"))
            taken.scatter_(1, i, True)
        out["top_logp"] = torch.where(live[:, None], torch.cat(best, 1), torch.full_like(zero, float("-inf")))
        out["top_idx"] = torch.where(live[:, None], torch.cat(where, 1), torch.full_like(order[:1], -1)).to(torch.int32)
    if case["backward"]:
        gl = torch.where(live, state["g_logp"], zero)[:, None] / case["temperature"]
        gh = torch.where(live, state["g_entropy"], zero)[:, None] / case["temperature"]
        grad = -q * gl - gh * (weighted + q * entropy[:, None])
        grad.scatter_add_(1, ids, gl)
        out["grad"] = grad.to(z.dtype)
    return out


# ---- one pass --------------------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if not own:
        plain = {"mm": _plain_mm, "wgrad": _plain_wgrad, "distill": _plain_distill, "logprobs": _plain_logprobs}
        return plain[case["op"]](state)
    himuon = state["himuon"]
    if case["op"] == "mm":
        return himuon.himuon_grouped_mm(state["x"], state["experts"], state["ends"])
    if case["op"] == "wgrad":
        return himuon.himuon_grouped_wgrad(state["x"], state["dy"], state["ends"])
    z = state["z"]
    if case["op"] == "distill":
        args = dict(temperature=case["temperature"], normalize=case["normalize"])
        if case["fused"]:
            r = himuon.himuon_distill(z, state["idx"], state["t"], weight=state["weight"], grad=True, **args)
            return r.loss, r.grad
        r = himuon.himuon_distill(z, state["idx"], state["t"], weight=state["weight"], **args)
        return r.loss, himuon.himuon_distill_grad(z, state["idx"], state["t"], r.lse, state["weight"], **args)
    r = himuon.himuon_token_logprobs(z, state["tokens"], top=case["top"], temperature=case["temperature"])
    out = {"logp": r.logp, "entropy": r.entropy}
    if case["top"]:
        out["top_logp"], out["top_idx"] = r.top_logp, r.top_idx
    if case["backward"]:
        out["grad"] = himuon.himuon_token_logprobs_grad(z, state["tokens"], r.lse, r.entropy, state["g_logp"],
                                                        state["g_entropy"], temperature=case["temperature"])
    return out


def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] in ("mm", "wgrad"):
        m, k, c = case["rows"], case["inner"], case["cols"]
        # weights of experts that have rows are read; a weight gradient is written for every expert
        n = sum(1 for x in _counts(case) if x) if case["op"] == "mm" else case["experts"]
        return {"bytes": b * (m * k + m * c + n * k * c) + 4 * case["experts"], "flops": 2 * m * k * c}
    n, v = case["rows"], case["vocab"]
    if case["op"] == "distill":
        # as two calls the logits are read twice
        passes = 2 if case["fused"] else 3
        return {"bytes": passes * n * v * b + n * (8 * case["entries"] + 8), "flops": 8 * n * v}
    passes = 3 if case["backward"] else 1
    return {"bytes": passes * n * v * b + n * (8 * case["top"] + 16), "flops": (12 if case["backward"] else 6) * n * v}


# ---- the definitions in 64 bits ----------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "mm":
        ends = [0] + state["ends"].tolist()
        y = torch.zeros((case["rows"], case["cols"]), dtype=f64, device="cuda")
        for e in range(case["experts"]):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                torch.mm(state["x"][lo:hi].to(f64), state["w"][e].to(f64).contiguous(), out=y[lo:hi])
        return y
    if case["op"] == "wgrad":
        ends = [0] + state["ends"].tolist()
        g = []
        for e in range(case["experts"]):
            rows = slice(ends[e], ends[e + 1])
            g.append(state["x"][rows].to(f64).t().contiguous() @ state["dy"][rows].to(f64))
        return torch.stack(g)

    tau = case["temperature"]
    losses, grads, outs = [], [], []
    step = max(1, (1 << 27) // case["vocab"])
    for r0 in range(0, case["rows"], step):   # in blocks of rows, to bound the memory
        rows = slice(r0, r0 + step)
        s = state["z"][rows].to(f64) / tau
        lse = torch.logsumexp(s, dim=1)
        q = torch.exp(s - lse[:, None])
        if case["op"] == "distill":
            idx, t, w = state["idx"][rows].long(), state["t"][rows].to(f64), state["weight"][rows].to(f64)
            p = torch.where(idx >= 0, torch.exp(t / tau if case["normalize"] else t), torch.zeros((), dtype=f64, device="cuda"))
            if case["normalize"]:
                p = p / p.sum(dim=1, keepdim=True)
            where = idx.clamp(min=0)
            # entropy of p and its cross entropy against q, apart
            inside = torch.special.xlogy(p, p).sum(dim=1)
            picked = s.gather(1, where) - lse[:, None]
            cross = torch.where(p > 0, p * picked, torch.zeros_like(p)).sum(dim=1)
            losses.append(w * (inside - cross))
            dense = torch.zeros_like(s).scatter_add_(1, where, p)
            g = (q * p.sum(dim=1)[:, None] - dense) * (w / tau)[:, None]
            g[w == 0] = 0.0
            grads.append(g)
            continue
        ids = state["tokens"][rows]
        live = ids >= 0
        pick = torch.nn.functional.one_hot(ids.clamp(min=0), case["vocab"]).to(torch.bool)
        logq = s - lse[:, None]
        entropy = -torch.special.xlogy(q, q).sum(dim=1)
        got = {"logp": torch.where(live, logq[pick], 0.0), "entropy": torch.where(live, entropy, 0.0)}
        if case["top"]:
            value, order = torch.sort(s, dim=1, descending=True, stable=True)
            top = order[:, :case["top"]].to(torch.int32)
            got["top_logp"] = value[:, :case["top"]] - lse[:, None]
            got["top_logp"][~live] = float("-inf")
            top[~live] = -1
            got["top_idx"] = top
            del value, order
        if case["backward"]:
            gl, gh = state["g_logp"][rows].to(f64)[:, None], state["g_entropy"][rows].to(f64)[:, None]
            g = gl * (pick.to(f64) - q) - gh * (torch.special.xlogy(q, q) + q * entropy[:, None])
            g[~live] = 0.0
            got["grad"] = g / tau
        outs.append(got)
    if case["op"] == "distill":
        return torch.cat(losses), torch.cat(grads)
    return {k: torch.cat([o[k] for o in outs]) for k in outs[0]}
