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

Nothing waits for the device: the experts' shares stay there as end rows.

    python -m tiled_newton_schulz_amd.moe_distill --steps 20
"""
from __future__ import annotations

import argparse

from . import himuon_distill, himuon_grouped_mm, himuon_grouped_wgrad, himuon_muon_step, himuon_token_logprobs


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


class Distiller:
    def __init__(self, student: Moe, teacher: Moe, top: int = 16, temperature: float = 1.0, tile: int = 128,
                 eta: float = 0.02, head_rate: float = 0.5):
        import torch
        self.student, self.teacher = student, teacher
        self.top, self.temperature, self.tile, self.eta, self.head_rate = top, temperature, tile, eta, head_rate
        self.momenta = [torch.zeros_like(w) for w in (*student.up, *student.down)]

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
        loss, (g_up, g_down, g_head) = self.gradients(tokens, *self.targets(tokens))
        weights = [*self.student.up, *self.student.down]
        himuon_muon_step(weights, self.momenta, [*g_up, *g_down], self.tile, 5, eta=self.eta)
        self.student.head.sub_(self.head_rate * g_head)
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
    a = ap.parse_args(argv)
    shape = (a.vocab, a.dim, a.hidden, a.experts, torch.bfloat16)
    teacher, student = Moe(*shape, seed=1), Moe(*shape, seed=2)
    student.embed, student.route = teacher.embed, teacher.route
    d = Distiller(student, teacher, a.top, tile=a.tile)
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
