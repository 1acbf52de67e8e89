"""The training loop that runs the operators together: gradients of one step
against autograd in fp64, and a loss that falls."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from tiled_newton_schulz_amd import moe_distill


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def pair(vocab, dim, hidden, experts, dtype):
    teacher, student = (moe_distill.Moe(vocab, dim, hidden, experts, dtype, seed=s) for s in (1, 2))
    student.embed, student.route = teacher.embed, teacher.route
    return teacher, student


@pytest.mark.parametrize("tokens,vocab,dim,hidden,experts", [(200, 501, 64, 96, 5), (3, 1000, 40, 33, 8)])
def test_gradients(cuda, tokens, vocab, dim, hidden, experts):
    """fp32: each of the chain's products errs by less than sqrt(K) 2^-24 of its
    result's norm and the losses by 2^-20, so 1e-4 of a gradient's norm holds all
    of them with room for the norms that grow along the chain."""
    teacher, student = pair(vocab, dim, hidden, experts, torch.float32)
    d = moe_distill.Distiller(student, teacher, top=7, temperature=1.5)
    ids = torch.randint(0, vocab, (tokens,), generator=torch.Generator().manual_seed(5)).cuda()
    idx, logp = d.targets(ids)
    print(f"distillation step {tokens} tokens, {vocab} x {dim} x {hidden}, {experts} experts", flush=True)
    loss, grads = d.gradients(ids, idx, logp)

    expert = (student.embed[ids] @ student.route).argmax(1).cpu()
    x = student.embed[ids].cpu().double()
    up, down, head = (w.cpu().double().requires_grad_() for w in (student.up, student.down, student.head))
    h = torch.stack([x[i] + torch.relu(x[i] @ up[e]).square() @ down[e] for i, e in enumerate(expert.tolist())])
    lq = torch.log_softmax(h @ head / 1.5, 1).gather(1, idx.cpu().long())
    lp = torch.log_softmax(logp.cpu().double() / 1.5, 1)
    want = (lp.exp() * (lp - lq)).sum(1) / tokens
    want.sum().backward()
    want = want.detach()
    assert (loss.cpu().double() - want).norm() <= 1e-4 * want.norm()
    for got, w in zip(grads, (up, down, head)):
        assert (got.cpu().double() - w.grad).norm() <= 1e-4 * w.grad.norm()
        unused = torch.ones(experts, dtype=torch.bool)
        unused[expert] = False
        if got.dim() == 3:
            assert torch.all(got[unused.cuda()] == 0)


def test_training(cuda):
    """Thirty steps on one batch: the loss halves, and the student comes to give
    the teacher's choice more."""
    teacher, student = pair(1000, 128, 192, 4, torch.bfloat16)
    d = moe_distill.Distiller(student, teacher, top=8, tile=64)
    ids = torch.randint(0, 1000, (512,), generator=torch.Generator().manual_seed(6)).cuda()
    before = d.score(ids).item()
    losses = []
    for i in range(30):
        losses.append(d.step(ids).item())
        print(f"step {i}: loss {losses[-1]:.4f}", flush=True)
    assert losses[-1] < 0.5 * losses[0]
    assert d.score(ids).item() > before


def test_command(cuda, capsys):
    moe_distill.main(["--steps", "2", "--tokens", "64", "--vocab", "500", "--dim", "64", "--hidden", "64", "--experts", "4",
                      "--top", "4", "--tile", "32"])
    assert capsys.readouterr().out.count("loss") == 2


def test_replaced_weights_are_used(cuda):
    """Weights given to a model after it was made are those of its products,
    and of the step that trains them."""
    vocab, dim, hidden, experts = 400, 64, 96, 4
    teacher, student = pair(vocab, dim, hidden, experts, torch.float32)
    d = moe_distill.Distiller(student, teacher, top=5, tile=32)
    other = moe_distill.Moe(vocab, dim, hidden, experts, torch.float32, seed=9)
    ids = torch.arange(100, device="cuda")
    student.up, student.down, student.head = (w.clone() for w in (other.up, other.down, other.head))
    other.embed, other.route = student.embed, student.route
    assert torch.equal(student.forward(ids)[0], other.forward(ids)[0])
    targets = d.targets(ids)
    want = moe_distill.Distiller(other, teacher, top=5, tile=32).gradients(ids, *targets)
    got = d.gradients(ids, *targets)
    assert torch.equal(got[0], want[0]) and all(torch.equal(a, b) for a, b in zip(got[1], want[1]))
    before = [w.clone() for w in (student.up, student.down, student.head)]
    d.step(ids)
    for a, b in zip((student.up, student.down, student.head), before):
        assert not torch.equal(a, b)
