"""The training loop with a layer norm, gated experts and AdamW: gradients of one step
against autograd in fp64, steps that run, and one step captured into a graph."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

import tiled_newton_schulz_amd as H
from tiled_newton_schulz_amd import moe_distill


def pair(vocab, dim, hidden, experts, dtype, **more):
    teacher, student = (moe_distill.GatedMoe(vocab, dim, hidden, experts, dtype, seed=s, **more) for s in (1, 2))
    student.embed, student.route = teacher.embed, teacher.route
    return teacher, student


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("tokens,vocab,dim,hidden,experts", [(200, 501, 64, 96, 5), (3, 1000, 40, 33, 8)])
def test_gradients(cuda, tokens, vocab, dim, hidden, experts, act):
    """fp32: each of the chain's products errs by less than sqrt(K) 2^-24 of its
    result's norm, the norm, the gate and the losses by 2^-20, so 1e-4 of a gradient's
    norm holds all of them with room for the norms that grow along the chain."""
    teacher, student = pair(vocab, dim, hidden, experts, torch.float32, act=act)
    student.norm_weight.mul_(1.0 + 0.3 * torch.randn(dim, generator=torch.Generator().manual_seed(3)).cuda())
    student.norm_bias.add_(0.1)
    d = moe_distill.Distiller(student, teacher, top=7, temperature=1.5)
    ids = torch.randint(0, vocab, (tokens,), generator=torch.Generator().manual_seed(5)).cuda()
    idx, logp = d.targets(ids)
    print(f"gated distillation step {tokens} tokens, {vocab} x {dim} x {hidden}, {experts} experts", flush=True)
    loss, grads = d.gradients(ids, idx, logp)

    expert = (student.embed[ids] @ student.route).argmax(1).cpu()
    x = student.embed[ids].cpu().double()
    up, down, head, nw, nb = ws = [w.cpu().double().requires_grad_() for w in (student.up, student.down, *d._others())]
    n = torch.nn.functional.layer_norm(x, (dim,), nw, nb, eps=1e-5)
    fn = torch.nn.functional.silu if act == "silu" else lambda t: torch.nn.functional.gelu(t, approximate="tanh")
    h = torch.stack([x[i] + (fn(n[i] @ up[e][:, :hidden]) * (n[i] @ up[e][:, hidden:])) @ down[e]
                     for i, e in enumerate(expert.tolist())])
    lq = torch.log_softmax(h @ head / 1.5, 1).gather(1, idx.cpu().long())
    lp = torch.log_softmax(logp.cpu().double() / 1.5, 1)
    want = (lp.exp() * (lp - lq)).sum(1) / tokens
    want.sum().backward()
    want = want.detach()
    assert (loss.cpu().double() - want).norm() <= 1e-4 * want.norm()
    for got, w in zip(grads, ws):
        assert (got.cpu().double() - w.grad).norm() <= 1e-4 * w.grad.norm()
        unused = torch.ones(experts, dtype=torch.bool)
        unused[expert] = False
        if got.dim() == 3:
            assert torch.all(got[unused.cuda()] == 0)


@pytest.mark.parametrize("bits", [32, 8])
def test_steps(cuda, bits):
    """Steps run, change every weight and leave finite ones."""
    teacher, student = pair(1000, 128, 192, 4, torch.bfloat16)
    d = moe_distill.Distiller(student, teacher, top=8, tile=64, state_bits=bits, rate=0.02)
    ids = torch.randint(0, 1000, (512,), generator=torch.Generator().manual_seed(6)).cuda()
    weights = (student.up, student.down, *d._others())
    before = [w.clone() for w in weights]
    for i in range(3):
        loss = d.step(ids).item()
        print(f"step {i}: loss {loss:.4f}", flush=True)
        assert math.isfinite(loss)
    for a, b in zip(weights, before):
        assert torch.all(torch.isfinite(a)) and not torch.equal(a, b)


def test_command(cuda, capsys):
    moe_distill.main(["--steps", "2", "--tokens", "64", "--vocab", "500", "--dim", "64", "--hidden", "64", "--experts", "4",
                      "--top", "4", "--tile", "32", "--gated", "--state-bits", "8"])
    assert capsys.readouterr().out.count("loss") == 2


def test_one_captured_step(cuda):
    """Norm, gated block, its backward and the optimiser as one graph: every replay's
    weights are those of the same calls made one by one, with other inputs each time."""
    M, d, f, n = 300, 64, 72, 5
    gen = torch.Generator().manual_seed(7)
    r = lambda *s, k=1.0: (torch.randn(s, generator=gen) * k).bfloat16().cuda()
    ends = torch.tensor([50, 50, 130, 260, 300], dtype=torch.int32, device=cuda)
    x, dy = r(M, d), r(M, d, k=0.1)

    def make():
        g = torch.Generator().manual_seed(8)
        t = lambda *s, k: (torch.randn(s, generator=g) * k).bfloat16().cuda()
        up, down, nw, nb = t(n, d, 2 * f, k=0.1), t(n, f, d, k=0.1), torch.ones(d, device=cuda).bfloat16(), t(d, k=0.1)
        return up, down, nw, nb, H.adamw_state([up, down, nw, nb], bits=8)

    def step(up, down, nw, nb, state):
        y, stats = H.himuon_layer_norm(x, nw, nb)
        h, pre = H.himuon_grouped_gated_mm(y, up, ends, keep=True)
        dpre, h = H.himuon_grouped_gated_mm_grad(dy, down, ends, pre, hidden=True, out=pre)
        g_up, g_down = H.himuon_grouped_wgrad(y, dpre, ends), H.himuon_grouped_wgrad(h, dy, ends)
        norm = H.himuon_layer_norm_grad(x, nw, stats, H.himuon_grouped_mm(dpre, up.transpose(1, 2), ends))
        H.himuon_adamw_step([up, down, nw, nb], [g_up, g_down, norm.dweight, norm.dbias], state, lr=1e-2, step=2)
        return norm.dx

    print("captured step", flush=True)
    one, two = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*make())   # (first calls outside the capture)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx = step(*one)
    for k in range(3):
        x.copy_(r(M, d))
        dy.copy_(r(M, d, k=0.1))
        want = step(*two)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want), k
        for a, b in zip(one[:4], two[:4]):
            assert torch.equal(a, b), k
        assert torch.equal(one[4].m.view(torch.uint8), two[4].m.view(torch.uint8))
