"""What is measured of a training step's other operators: the gated experts' block (forward, and backward through the
down product and the gate), layer normalisation with its gradients, and AdamW steps over many tensors with states in 32
or 8 bits.

Where `own` is false, `run` computes them from elementary torch operations in 32 bits; where it is true, through
tiled_newton_schulz_amd.  Shapes come from this repository's mixture-of-experts workload (64 experts of 4096 x 1408 and
1408 x 4096), its layers (24, of width 2048), and generic vocabulary sizes.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
BLOCK = 256    # elements that share a scale where states are held in 8 bits

# Every listed and drawn case of the gated experts stays below these.
MOST_FLOPS = 4 * 16384 * 4096 * 1408
MOST_WEIGHTS = 64 * 4096 * 2 * 1408
# ... of layer normalisation, and of an optimiser step.
MOST_ROWS = 16384 * 4096
MOST_PARAMETERS = 2 * 32000 * 4096


def listed():
    return [
        # a small experiment's gated layer, a handful of tokens, kept for its gradient: launch latency
        dict(name="gated_small", op="gated", dtype="bf16", experts=8, rows=40, inner=512, cols=256, act="silu", keep=True),
        # a few dozen tokens decoded through the 64 experts: the weights' bytes count
        dict(name="gated_decode", op="gated", dtype="bf16", experts=64, rows=96, inner=4096, cols=1408, act="silu",
             keep=False),
        # one training step's forward pass
        dict(name="gated_train", op="gated", dtype="bf16", experts=64, rows=16384, inner=4096, cols=1408, act="silu",
             keep=True),
        # ... and its way back through the down product and the gate
        dict(name="gated_grad_train", op="gated_grad", dtype="bf16", experts=64, rows=16384, inner=4096, cols=1408,
             act="silu"),
        # fp32 experts of odd sizes (rows that start off any alignment), another activation
        dict(name="gated_grad_fp32_odd", op="gated_grad", dtype="fp32", experts=6, rows=1001, inner=515, cols=261,
             act="gelu_tanh"),
        # a server normalises four sequences' tokens: latency
        dict(name="norm_decode", op="norm", dtype="bf16", rows=4, cols=4096),
        # the rows of one training step, forward and backward
        dict(name="norm_train", op="norm", dtype="bf16", rows=16384, cols=4096),
        dict(name="norm_grad_train", op="norm_grad", dtype="bf16", rows=16384, cols=4096),
        # fp32 rows of an odd width
        dict(name="norm_grad_odd", op="norm_grad", dtype="fp32", rows=3001, cols=1409),
        # two norms' weights and biases in each of 24 layers: 96 small tensors, launch and host time
        dict(name="adamw_norms", op="adamw", dtype="fp32", grads="fp32", bits=32, tensors=96, numel=96 * 2048, even=True,
             step=100),
        # an embedding and a head, states in 8 bits
        dict(name="adamw_embed", op="adamw", dtype="bf16", grads="bf16", bits=8, tensors=2, numel=2 * 32000 * 4096,
             even=True, step=5000),
        # fp32 master weights of many uneven tensors from bf16 gradients
        dict(name="adamw_master", op="adamw", dtype="fp32", grads="bf16", bits=32, tensors=50, numel=20000003, even=False,
             step=1),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "gated_grad", "norm", "norm_grad", "adamw", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("gated", "gated_grad"):
        # fp32 products are a sixteenth as fast: less work
        flops = MOST_FLOPS if dtype == "bf16" else MOST_FLOPS // 16
        while True:
            experts = _spread(rng, 1, 96)
            rows = _spread(rng, 1, 32768)
            inner, cols = _spread(rng, 32, 4096), _spread(rng, 32, 4096)
            if rng.random() < 0.6:   # most widths are multiples of eight, some are odd
                inner, cols = 8 * max(1, inner // 8), 8 * max(1, cols // 8)
            if 4 * rows * inner * cols <= flops and 2 * experts * inner * cols <= MOST_WEIGHTS:
                break
        case = dict(op=op, dtype=dtype, experts=experts, rows=rows, inner=inner, cols=cols,
                    act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]))
        if op == "gated":
            case["keep"] = rng.random() < 0.5
        return case
    if op in ("norm", "norm_grad"):
        while True:
            rows, cols = _spread(rng, 1, 65536), _spread(rng, 16, 16384)
            if rng.random() < 0.6:
                cols = 8 * max(1, cols // 8)
            if rows * cols * BYTES[dtype] <= 2 * MOST_ROWS:
                return dict(op=op, dtype=dtype, rows=rows, cols=cols)
    tensors = _spread(rng, 1, 300)
    most = MOST_PARAMETERS if dtype == "bf16" else MOST_PARAMETERS // 2
    return dict(op="adamw", dtype=dtype, grads="bf16" if dtype == "bf16" else rng.choice(["bf16", "fp32"]),
                bits=rng.choice([8, 8, 32]), tensors=tensors, numel=_spread(rng, 4 * tensors, most // 4),
                even=rng.random() < 0.3, step=_spread(rng, 1, 100000))


# ---- inputs ------------------------------------------------------------------------------------

def _shares(parts, total, even, least):
    """Whole parts of `total`: equal ones, or uneven ones of at least `least`."""
    if even:
        return [total // parts] * parts
    rng = random.Random(parts * 1000003 + total)
    share = [rng.gammavariate(2.0, 1.0) if rng.random() > 0.05 else 0.0 for _ in range(parts)]
    if sum(share) == 0.0:
        share[0] = 1.0
    whole, out, left = sum(share), [], 0.0
    for s in share:   # the fractions are carried on, so the sum is exact
        left += s * (total - least * parts) / whole
        c = int(left + 1e-9)
        out.append(least + c)
        left -= c
    out[max(range(parts), key=lambda i: share[i])] += total - sum(out)
    return out


def _counts(case):
    """Rows of each expert, before they are shuffled: a router's uneven choice, some experts without a row."""
    return _shares(case["experts"], case["rows"], False, 0)


def _sizes(case):
    """Elements of each tensor of an optimiser step, and where they begin in a flat buffer (in whole blocks)."""
    if case["even"]:
        sizes = _shares(case["tensors"], case["numel"], True, 1)
    else:   # a few large tensors and many small ones
        sizes = _shares(case["tensors"], case["numel"], False, 1)
        sizes.sort()
        for i in range(len(sizes) // 2):
            moved = sizes[i] - max(1, sizes[i] // (3 << (i % 11)))
            sizes[i] -= moved
            sizes[-1 - i // 4] += moved
        random.Random(case["numel"]).shuffle(sizes)
    starts, at = [], 0
    for s in sizes:
        starts.append(at)
        at += -(-s // BLOCK) * BLOCK
    return sizes, starts, at


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(gen, shape, dtype, scale=1.0):
    t = torch.empty(shape, dtype=TYPES[dtype], device="cuda")
    t.normal_(generator=gen)
    return t.mul_(scale) if scale != 1.0 else t


def _uniform(gen, n, lo, hi):
    return torch.empty(n, dtype=torch.float32, device="cuda").uniform_(lo, hi, generator=gen)


def prepare(case, seed):
    gen = _generator(seed)
    state = {"case": case}
    himuon = None
    if own:
        import tiled_newton_schulz_amd as himuon
        state["himuon"] = himuon
    dtype = case["dtype"]
    if case["op"] in ("gated", "gated_grad"):
        counts = _counts(case)
        random.Random(int(seed)).shuffle(counts)
        n, m, k, c = case["experts"], case["rows"], case["inner"], case["cols"]
        state["counts"] = counts
        state["ends"] = torch.tensor(counts, device="cuda").cumsum(0).to(torch.int32)
        if case["op"] == "gated":
            # both projections of an expert side by side, gate first
            state["x"] = _normal(gen, (m, k), dtype)
            state["w"] = _normal(gen, (n, k, 2 * c), dtype, 1.5 / math.sqrt(k))
        else:
            # the down projection, the gradient behind it, and what the forward pass kept
            state["dy"] = _normal(gen, (m, k), dtype, 0.1)
            state["w"] = _normal(gen, (n, c, k), dtype, 1.0 / math.sqrt(c))
            state["pre"] = _normal(gen, (m, 2 * c), dtype, 1.5)
        if own:
            state["experts"] = himuon.matrices(state["w"])
        return state
    if case["op"] in ("norm", "norm_grad"):
        n, c = case["rows"], case["cols"]
        # activations of a residual stream: rows of their own size and offset, a few large columns
        x = torch.empty((n, c), dtype=torch.float32, device="cuda").normal_(generator=gen)
        x[:, torch.randint(0, c, (max(1, c // 200),), generator=gen, device="cuda")] *= 20.0
        x.mul_(_uniform(gen, n, 0.5, 4.0)[:, None]).add_(_uniform(gen, n, -2.0, 2.0)[:, None])
        state["x"] = x.to(TYPES[dtype])
        state["weight"] = _normal(gen, (c,), dtype, 0.2) + 1.0
        state["bias"] = _normal(gen, (c,), dtype, 0.1)
        if case["op"] == "norm_grad":
            state["dy"] = _normal(gen, (n, c), dtype, 0.1)
            mean = state["x"].float().mean(dim=1, keepdim=True)
            var = (state["x"].float() - mean).square_().mean(dim=1, keepdim=True)
            state["stats"] = torch.cat([mean, torch.rsqrt(var + 1e-5)], dim=1).contiguous()
        return state

    # an optimiser step: weights and gradients in flat buffers, as training programs keep them, and a tensor for each part
    sizes, starts, total = _sizes(case)
    kept = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, s in zip(starts, sizes):
        kept[a:a + s] = True
    state["w"] = _normal(gen, (total,), dtype, 0.05).mul_(kept)
    state["g"] = _normal(gen, (total,), case["grads"], 0.01).mul_(kept)
    # rows of an embedding that no token of the batch met
    state["g"].mul_((_uniform(gen, total // BLOCK, 0.0, 1.0) > 0.3).repeat_interleave(BLOCK))
    if case["bits"] == 32:
        state["m"] = _normal(gen, (total,), "fp32", 0.003).mul_(kept)
        state["v"] = _normal(gen, (total,), "fp32", 0.01).square_().mul_(kept)
    else:
        f8 = torch.float8_e4m3fn
        state["m"] = _normal(gen, (total,), "fp32", 100.0).clamp_(-448.0, 448.0).mul_(kept).to(f8)
        state["v"] = _normal(gen, (total,), "fp32", 120.0).abs_().clamp_(1.0, 448.0).mul_(kept).to(f8)
        state["m_scale"] = _uniform(gen, total // BLOCK, 1e-5, 5e-5)
        state["v_scale"] = _uniform(gen, total // BLOCK, 5e-5, 1e-4)
    # the factor that holds the gradients' norm down, computed on the GPU
    state["grad_scale"] = _uniform(gen, 1, 0.5, 1.0)
    state["starts"], state["sizes"] = starts, sizes
    if own:
        # each tensor as the model has it
        state["weights"] = himuon.tensors([state["w"][a:a + s] for a, s in zip(starts, sizes)])
        state["gradients"] = himuon.tensors([state["g"][a:a + s] for a, s in zip(starts, sizes)])
        held = himuon.adamw_state(state["weights"], bits=case["bits"])
        held.m.copy_(state["m"])
        held.v.copy_(state["v"])
        if case["bits"] == 8:
            held.m_scale.copy_(state["m_scale"])
            held.v_scale.copy_(state["v_scale"])
        state["held"] = held
        for name in ("m", "v", "m_scale", "v_scale"):
            state.pop(name, None)
    return state


LR, BETAS, EPS, DECAY = 3e-4, (0.9, 0.999), 1e-8, 0.1


# ---- the operators in their plain form ------------------------------------------------------------

def _plain_act(act, g, with_slope):
    """act(g), and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s)) if with_slope else None
    if act == "relu":
        return torch.clamp(g, min=0.0), (g > 0).float() if with_slope else None
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi) if with_slope else None
    a, b = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(a * (g + b * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * a * (1.0 + 3.0 * b * g * g) if with_slope else None


def _by_expert(counts, rows, w, product):
    parts, r = [], 0
    for e, c in enumerate(counts):
        if c:
            parts.append(product(rows[r:r + c].float(), w[e].float()))
        r += c
    return torch.cat(parts)


def _plain_gated(state):
    case, c = state["case"], state["case"]["cols"]
    pre = _by_expert(state["counts"], state["x"], state["w"], lambda x, w: x @ w)
    h = _plain_act(case["act"], pre[:, :c], False)[0] * pre[:, c:]
    return (h.to(state["x"].dtype), pre.to(state["x"].dtype)) if case["keep"] else (h.to(state["x"].dtype),)


def _plain_gated_grad(state):
    case, c, dtype = state["case"], state["case"]["cols"], state["dy"].dtype
    dh = _by_expert(state["counts"], state["dy"], state["w"], lambda dy, w: dy @ w.t())
    g, u = state["pre"][:, :c].float(), state["pre"][:, c:].float()
    a, slope = _plain_act(case["act"], g, True)
    return torch.cat([dh * u * slope, dh * a], dim=1).to(dtype), (a * u).to(dtype)


def _plain_norm(state):
    x = state["x"].float()
    mean = x.mean(dim=1, keepdim=True)
    d = x - mean
    r = 1.0 / torch.sqrt(d.square().mean(dim=1, keepdim=True) + 1e-5)
    y = d * r * state["weight"].float() + state["bias"].float()
    return y.to(state["x"].dtype), torch.cat([mean, r], dim=1)


def _plain_norm_grad(state):
    dtype = state["x"].dtype
    mean, r = state["stats"][:, :1], state["stats"][:, 1:]
    xh, dy = (state["x"].float() - mean) * r, state["dy"].float()
    dyw = dy * state["weight"].float()
    dx = r * (dyw - dyw.mean(dim=1, keepdim=True) - xh * (dyw * xh).mean(dim=1, keepdim=True))
    return dx.to(dtype), (dy * xh).sum(dim=0).to(dtype), dy.sum(dim=0).to(dtype)


def _dither(state, device):
    """16 random bits of every element, from its place in its tensor and the step: for sqrt(v), and for m."""
    total = state["w"].numel()
    starts = torch.tensor(state["starts"], device=device)
    widths = torch.tensor([-(-s // BLOCK) * BLOCK for s in state["sizes"]], device=device)
    i = torch.arange(total, device=device) - torch.repeat_interleave(starts, widths, output_size=total)
    low = 0xFFFFFFFF
    h = ((i >> 1) * 0xB890E049 + _key(state["case"]["step"])) & low
    h = ((h ^ (h >> 15)) * 0xB4A1B41D) & low
    h = ((h ^ (h >> 13)) * 0xF5BBB081) & low
    u = torch.where((i & 1) == 0, h & 0xFFFF, h >> 16)
    return u, ((u << 8) | (u >> 8)) & 0xFFFF


def _key(step):
    low = 0xFFFFFFFF
    k = (step * 0x9AD24435 + 0xB3B07CC5) & low
    return ((k ^ (k >> 16)) * 0xB06A350D) & low


def _plain_codes(y, u):
    """e4m3 codes of y (0 to 448), rounded down after u / 65536 of a step was added."""
    small = y < 0.015625
    z = torch.where(small, y + 0.015625, y)
    bits = (z.view(torch.int32) + (u << 4).to(torch.int32)) >> 20
    return torch.where(small, bits - 968, bits - 960).clamp(max=126)


def _plain_adamw(state):
    case, w = state["case"], state["w"]
    b1, b2 = BETAS
    g = state["g"].float() * state["grad_scale"]
    if case["bits"] == 32:
        m0, r0, v0 = state["m"], None, state["v"]
    else:
        m0 = (state["m"].float().view(-1, BLOCK) * state["m_scale"][:, None]).view(-1)
        r0 = (state["v"].float().view(-1, BLOCK) * state["v_scale"][:, None]).view(-1)
        v0 = r0 * r0
    m = m0 * b1 + g * (1.0 - b1)
    v = v0 * b2 + (g * g) * (1.0 - b2)
    r = torch.sqrt(v)
    c1 = LR / (1.0 - b1 ** case["step"])
    c2 = 1.0 / math.sqrt(1.0 - b2 ** case["step"])
    new = w.float() * (1.0 - LR * DECAY) - c1 * m / (r * c2 + EPS)
    w.copy_(new.to(w.dtype))
    if case["bits"] == 32:
        state["m"].copy_(m)
        state["v"].copy_(v)
        return w, state["m"], state["v"]
    uv, um = _dither(state, w.device)
    for name, value, u in (("m", m, um), ("v", r, uv)):
        most = value.abs().view(-1, BLOCK).amax(dim=1).clamp(min=1e-30)
        y = (value.abs().view(-1, BLOCK) * (most.reciprocal() * 448.0)[:, None]).view(-1)
        code = _plain_codes(y, u)
        if name == "v":   # what is not zero stays so
            code = torch.where((value > 0) & (code == 0), 1, code)
        code = torch.where(value < 0, code + 128, code).to(torch.uint8)
        state[name].copy_(code.view(torch.float8_e4m3fn))
        state[name + "_scale"].copy_(most * (1.0 / 448.0))
    return w, state["m"], state["v"], state["m_scale"], state["v_scale"]


# ---- one pass --------------------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if not own:
        plain = {"gated": _plain_gated, "gated_grad": _plain_gated_grad, "norm": _plain_norm,
                 "norm_grad": _plain_norm_grad, "adamw": _plain_adamw}
        return plain[case["op"]](state)
    himuon = state["himuon"]
    if case["op"] == "gated":
        r = himuon.himuon_grouped_gated_mm(state["x"], state["experts"], state["ends"], act=case["act"], keep=case["keep"])
        return (r.h, r.pre) if case["keep"] else (r.h,)
    if case["op"] == "gated_grad":
        r = himuon.himuon_grouped_gated_mm_grad(state["dy"], state["experts"], state["ends"], state["pre"], act=case["act"],
                                                hidden=True)
        return r.grad, r.h
    if case["op"] == "norm":
        r = himuon.himuon_layer_norm(state["x"], state["weight"], state["bias"], eps=1e-5)
        return r.y, r.stats
    if case["op"] == "norm_grad":
        r = himuon.himuon_layer_norm_grad(state["x"], state["weight"], state["stats"], state["dy"])
        return r.dx, r.dweight, r.dbias
    held = state["held"]
    himuon.himuon_adamw_step(state["weights"], state["gradients"], held, lr=LR, step=case["step"], betas=BETAS, eps=EPS,
                             weight_decay=DECAY, grad_scale=state["grad_scale"])
    if case["bits"] == 32:
        return state["w"], held.m, held.v
    return state["w"], held.m, held.v, held.m_scale, held.v_scale


def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] in ("gated", "gated_grad"):
        m, k, c = case["rows"], case["inner"], case["cols"]
        # weights of experts that have rows are read
        n = sum(1 for x in _counts(case) if x)
        if case["op"] == "gated":
            return {"bytes": b * (m * k + (3 if case["keep"] else 1) * m * c + n * k * 2 * c) + 4 * case["experts"],
                    "flops": 4 * m * k * c + 8 * m * c}
        return {"bytes": b * (m * k + 5 * m * c + n * k * c) + 4 * case["experts"], "flops": 2 * m * k * c + 16 * m * c}
    if case["op"] in ("norm", "norm_grad"):
        n, c = case["rows"], case["cols"]
        if case["op"] == "norm":
            return {"bytes": b * (2 * n * c + 2 * c) + 8 * n, "flops": 8 * n * c}
        return {"bytes": b * (3 * n * c + 3 * c) + 8 * n, "flops": 14 * n * c}
    held = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    numel = sum(_sizes(case)[0])
    return {"bytes": numel * (2 * b + BYTES[case["grads"]] + held), "flops": 16 * numel}


# ---- the definitions in 64 bits ----------------------------------------------------------------------

def _slopes(act, g):
    """act(g), and its derivative by autograd."""
    g = g.detach().requires_grad_()
    with torch.enable_grad():
        if act == "silu":
            y = g * torch.sigmoid(g)
        elif act == "relu":
            y = torch.relu(g)
        else:
            y = torch.nn.functional.gelu(g, approximate="tanh" if act == "gelu_tanh" else "none")
        slope, = torch.autograd.grad(y.sum(), g)
    return y.detach(), slope


def exact(case, seed):
    state = prepare(case, seed)
    f64 = torch.float64
    if case["op"] in ("gated", "gated_grad"):
        c = case["cols"]
        ends = [0] + state["ends"].tolist()
        rows = state["x"] if case["op"] == "gated" else state["dy"]
        outs = []
        for e in range(case["experts"]):
            part = slice(ends[e], ends[e + 1])
            if ends[e + 1] == ends[e]:
                continue
            w = state["w"][e].to(f64)
            if case["op"] == "gated":
                gate, up = rows[part].to(f64) @ w[:, :c].contiguous(), rows[part].to(f64) @ w[:, c:].contiguous()
                h = _slopes(case["act"], gate)[0] * up
                outs.append((h, torch.cat([gate, up], dim=1)) if case["keep"] else (h,))
            else:
                dh = torch.mm(rows[part].to(f64), w.t().contiguous())
                gate, up = state["pre"][part].to(f64).split(c, dim=1)
                y, slope = _slopes(case["act"], gate)
                outs.append((torch.cat([slope * up * dh, y * dh], dim=1), y * up))
        return tuple(torch.cat(o) for o in zip(*outs))
    if case["op"] == "norm":
        ys, stats = [], []
        for x in state["x"].split(4096):   # in blocks of rows, to bound the memory
            x = x.to(f64)
            var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
            r = (var + 1e-5) ** -0.5
            ys.append((x - mean) * (state["weight"].to(f64) * r) + state["bias"].to(f64))
            stats.append(torch.cat([mean, r], dim=1))
        return torch.cat(ys), torch.cat(stats)
    if case["op"] == "norm_grad":
        c, w = case["cols"], state["weight"].to(f64)
        dxs, dw, db = [], torch.zeros(c, dtype=f64, device="cuda"), torch.zeros(c, dtype=f64, device="cuda")
        for x, dy, st in zip(state["x"].split(4096), state["dy"].split(4096), state["stats"].split(4096)):
            xh = (x.to(f64) - st[:, :1]) * st[:, 1:].to(f64)
            dy = dy.to(f64)
            a, b = dy @ w, ((dy * xh) @ w)
            dxs.append(st[:, 1:].to(f64) * (dy * w - (a[:, None] + xh * b[:, None]) / c))
            dw += (dy * xh).sum(dim=0)
            db += dy.sum(dim=0)
        return torch.cat(dxs), dw, db

    (b1, b2), t = BETAS, case["step"]
    g = state["g"].to(f64) * state["grad_scale"].to(f64)
    if case["bits"] == 32:
        m0, v0 = state["m"].to(f64), state["v"].to(f64)
    else:
        wide = lambda name: state[name].to(f64) * state[name + "_scale"].to(f64).repeat_interleave(BLOCK)
        m0, v0 = wide("m"), wide("v") ** 2
    m, v = torch.lerp(g, m0, b1), torch.lerp(g * g, v0, b2)
    update = (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + EPS)
    w = state["w"].to(f64)
    w = w - LR * (update + DECAY * w)
    if case["bits"] == 32:
        return w, m, v
    del update, g, m0, v0
    uv, um = _dither(state, "cuda")
    out = [w]
    scales = []
    for x, u in ((m, um), (v.sqrt(), uv)):
        most = torch.linalg.vector_norm(x.view(-1, BLOCK), ord=float("inf"), dim=1).clamp(min=1e-30)
        scales.append(most / 448)
        y = (x.abs().view(-1, BLOCK) / scales[-1][:, None]).view(-1)
        step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)   # between neighbours of y
        q = torch.floor(y / step + u / 65536) * step
        if x.min() >= 0:   # sqrt(v)
            q = torch.where(x > 0, q.clamp(min=2.0 ** -9), q)
        out.append(torch.copysign(q.clamp(max=448), x))
    return (*out, *scales)
