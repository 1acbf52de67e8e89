"""Distilling a mixture-of-experts student from a teacher's top logits, trained
by Muon: the library's operators in one training loop.

A model is a residual block of experts between an embedding and a head,

    x = embed[token],   h = x + relu(x up_e)^2 down_e,   logits = h head,

with e the token's expert (argmax of x route; embedding and routes are fixed).
One step (Distiller.step):

1. the teacher's logits give its `top` entries of every row
   (himuon_token_logprobs);
2. the student's forward pass: its rows sorted by expert, one himuon_grouped_mm
   for each of the two products, whatever the experts' shares;
3. loss and gradient of the logits in one call, the gradient in place of the
   logits (himuon_distill);
4. backward: himuon_grouped_mm with the transposed weights for the input's
   gradient, himuon_grouped_wgrad for the experts';
5. himuon_muon_step on every expert's matrices (and plain gradient descent on
   the head).

GatedMoe normalises the experts' input and gates them,

    n = layer_norm(x),   h = x + (silu(n gate_e) * (n up_e)) down_e,

with himuon_layer_norm, himuon_grouped_gated_mm and their gradients in steps 2
and 4, and in step 5 one himuon_adamw_step on the head and the norm's weight and
bias, which Muon is not for.

Nothing waits for the device: the experts' shares stay there as end rows.

    python -m tiled_newton_schulz_amd.moe_distill --steps 20
    python -m tiled_newton_schulz_amd.moe_distill --steps 20 --gated --state-bits 8
"""
from __future__ import annotations

import argparse

from . import (adamw_state, himuon_adamw_step, himuon_distill, himuon_grouped_gated_mm, himuon_grouped_gated_mm_grad,
               himuon_grouped_mm, himuon_grouped_wgrad, himuon_layer_norm, himuon_layer_norm_grad, himuon_muon_step,
               himuon_token_logprobs)


class Moe:
    """Weights of the model above: embed V x d, route d x E, up E x d x f, down
    E x f x d, head d x V."""

    def __init__(self, vocab: int, dim: int, hidden: int, experts: int, dtype, seed: int, device="cuda"):
        import torch
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=g) * scale).to(dtype).to(device)

        self.embed = normal(vocab, dim, scale=1.0)
        self.route = normal(dim, experts, scale=dim ** -0.5)
        self.up = normal(experts, dim, hidden, scale=dim ** -0.5)
        self.down = normal(experts, hidden, dim, scale=hidden ** -0.5)
        self.head = normal(dim, vocab, scale=2 * dim ** -0.5)

    def forward(self, tokens):
        """(logits, what the backward pass needs)."""
        import torch
        x = self.embed[tokens]
        expert = (x @ self.route).argmax(1)
        order = torch.argsort(expert, stable=True)
        ends = torch.searchsorted(expert[order], torch.arange(len(self.up), device=x.device), right=True).int()
        xs = x[order]
        pre = himuon_grouped_mm(xs, self.up, ends)
        act = torch.relu(pre).square()
        h = x.index_add(0, order, himuon_grouped_mm(act, self.down, ends))
        return h @ self.head, (order, ends, xs, pre, act, h)

    def backward(self, kept, dlogits):
        """Gradients of (up, down, head)."""
        import torch
        order, ends, xs, pre, act, h = kept
        dy = (dlogits @ self.head.t())[order]
        dact = himuon_grouped_mm(dy, self.down.transpose(1, 2), ends)
        dpre = dact * (2 * torch.relu(pre))
        g_up, g_down = torch.empty_like(self.up), torch.empty_like(self.down)
        himuon_grouped_wgrad(xs, dpre, ends, g_up)
        himuon_grouped_wgrad(act, dy, ends, g_down)
        return g_up, g_down, h.t() @ dlogits

    def matrices(self, up, down):
        """What Muon orthogonalises one by one, of these weights or gradients."""
        return [*up, *down]


class GatedMoe(Moe):
    """As Moe, with a layer norm (norm_weight, norm_bias: d) and gated experts: up
    is E x d x 2f, the gate's projection in its first f columns."""

    def __init__(self, vocab: int, dim: int, hidden: int, experts: int, dtype, seed: int, device="cuda", act: str = "silu"):
        import torch
        super().__init__(vocab, dim, hidden, experts, dtype, seed, device)
        g = torch.Generator().manual_seed(seed + 1000)
        gate = (torch.randn((experts, dim, hidden), generator=g) * dim ** -0.5).to(dtype).to(device)
        self.up = torch.cat([gate, self.up], dim=2)
        self.norm_weight = torch.ones(dim, dtype=dtype, device=device)
        self.norm_bias = torch.zeros(dim, dtype=dtype, device=device)
        self.act = act

    def forward(self, tokens):
        """(logits, what the backward pass needs)."""
        import torch
        x = self.embed[tokens]
        n, stats = himuon_layer_norm(x, self.norm_weight, self.norm_bias)
        expert = (x @ self.route).argmax(1)
        order = torch.argsort(expert, stable=True)
        ends = torch.searchsorted(expert[order], torch.arange(len(self.up), device=x.device), right=True).int()
        ns = n[order]
        hidden, pre = himuon_grouped_gated_mm(ns, self.up, ends, act=self.act, keep=True)
        h = x.index_add(0, order, himuon_grouped_mm(hidden, self.down, ends))
        return h @ self.head, (order, ends, x, stats, ns, pre, h)

    def backward(self, kept, dlogits):
        """Gradients of (up, down, head, norm_weight, norm_bias); what was kept is used up."""
        import torch
        order, ends, x, stats, ns, pre, h = kept
        dy = (dlogits @ self.head.t())[order]
        dpre, hidden = himuon_grouped_gated_mm_grad(dy, self.down, ends, pre, act=self.act, hidden=True, out=pre)
        g_up, g_down = torch.empty_like(self.up), torch.empty_like(self.down)
        himuon_grouped_wgrad(ns, dpre, ends, g_up)
        himuon_grouped_wgrad(hidden, dy, ends, g_down)
        dn = torch.empty_like(x)
        dn[order] = himuon_grouped_mm(dpre, self.up.transpose(1, 2), ends)
        norm = himuon_layer_norm_grad(x, self.norm_weight, stats, dn, dx=False)   # (the embedding is fixed)
        return g_up, g_down, h.t() @ dlogits, norm.dweight, norm.dbias

    def matrices(self, up, down):
        """The gate's and the up projection each on its own."""
        f = self.down.shape[1]
        return [*up[:, :, :f], *up[:, :, f:], *down]


class Distiller:
    """head_rate: of a Moe's head; rate, state_bits: of AdamW on what Muon leaves of a
    GatedMoe."""

    def __init__(self, student: Moe, teacher: Moe, top: int = 16, temperature: float = 1.0, tile: int = 128,
                 eta: float = 0.02, head_rate: float = 0.5, rate: float = 1e-3, state_bits: int = 32):
        import torch
        self.student, self.teacher = student, teacher
        self.top, self.temperature, self.tile, self.eta, self.head_rate = top, temperature, tile, eta, head_rate
        self.momenta = [torch.zeros_like(w) for w in student.matrices(student.up, student.down)]
        self.rate, self.steps = rate, 0
        self.state = adamw_state(self._others(), bits=state_bits) if isinstance(student, GatedMoe) else None

    def _others(self):
        return [self.student.head, self.student.norm_weight, self.student.norm_bias]

    def targets(self, tokens):
        """(ids, log probabilities) of the teacher's top entries, best first."""
        logits, _ = self.teacher.forward(tokens)
        r = himuon_token_logprobs(logits, top=self.top)
        return r.top_idx, r.top_logp

    def gradients(self, tokens, idx, logp):
        """(loss of every token, gradients of their mean)."""
        import torch
        n = len(tokens)
        logits, kept = self.student.forward(tokens)
        mean = torch.full((n,), 1.0 / n, device=logits.device)
        # (normalised over the entries, the teacher's log probabilities are as
        # good as its logits)
        r = himuon_distill(logits, idx, logp, temperature=self.temperature, weight=mean, grad=logits)
        return r.loss, self.student.backward(kept, r.grad)

    def step(self, tokens):
        """Trains on a batch of tokens; the mean loss before the update (on the device)."""
        loss, (g_up, g_down, *others) = self.gradients(tokens, *self.targets(tokens))
        self.steps += 1
        weights = self.student.matrices(self.student.up, self.student.down)
        himuon_muon_step(weights, self.momenta, self.student.matrices(g_up, g_down), self.tile, 5, eta=self.eta)
        if self.state is None:
            self.student.head.sub_(self.head_rate * others[0])
        else:
            himuon_adamw_step(self._others(), others, self.state, lr=self.rate, step=self.steps)
        return loss.sum()

    def score(self, tokens):
        """Mean log probability the student gives to the teacher's first choice."""
        idx, _ = self.targets(tokens)
        logits, _ = self.student.forward(tokens)
        return himuon_token_logprobs(logits, idx[:, 0].contiguous()).logp.mean()


def main(argv=None):
    import torch
    ap = argparse.ArgumentParser(description="distil a mixture-of-experts student, trained by Muon")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=4096, help="tokens of a batch")
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--dim", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=1408)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top", type=int, default=16, help="teacher entries of a row")
    ap.add_argument("--tile", type=int, default=128)
    ap.add_argument("--gated", action="store_true", help="a layer norm and gated experts, AdamW on the rest")
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=32, help="of AdamW's states (--gated)")
    a = ap.parse_args(argv)
    shape = (a.vocab, a.dim, a.hidden, a.experts, torch.bfloat16)
    model = GatedMoe if a.gated else Moe
    teacher, student = model(*shape, seed=1), model(*shape, seed=2)
    student.embed, student.route = teacher.embed, teacher.route
    d = Distiller(student, teacher, a.top, tile=a.tile, state_bits=a.state_bits)
    g = torch.Generator(device="cuda").manual_seed(3)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps):
        tokens = torch.randint(0, a.vocab, (a.tokens,), device="cuda", generator=g)
        start.record()
        loss = d.step(tokens)
        end.record()
        end.synchronize()
        print(f"step {i}: loss {loss.item():.4f}, log probability of the teacher's choice {d.score(tokens).item():.4f}, "
              f"{start.elapsed_time(end):.2f} ms", flush=True)


if __name__ == "__main__":
    main()
