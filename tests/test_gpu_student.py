"""The workers' distillation step (student.StudentStep): its losses and
gradients against 64-bit autograd of the same model without quantisation, and
a few steps of descent on the averaged gradients.

Tolerance: rounding a value to e4m3 is off by 2.6% in the mean square (2^-4
over sqrt 3, and the significand's spread), to e5m2 by 5.3%.  The logits carry
two e4m3 roundings, a weight gradient an e4m3 and an e5m2 one and, through the
probabilities, the logits' own errors: 15% of the gradient's norm covers them."""
import numpy as np
import pytest

from helpers import need_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return need_cuda()


def make(torch, P, T, H, V, E, n, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    head = torch.randn((V, H), generator=g, device="cuda") * 0.2
    router = torch.randn((E, H), generator=g, device="cuda") * 0.2
    hidden = [torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(P)]
    index = [torch.stack([torch.randperm(V, generator=g, device="cuda")[:n] for _ in range(T)]).int() for _ in range(P)]
    teacher = [torch.randn((T, n), generator=g, device="cuda") * 2 for _ in range(P)]
    return head, router, hidden, index, teacher


def exact(torch, step, head, router, hidden, index, teacher, k, alpha, tau, valid=None):
    """(mean distillation loss, balance loss, head's and router's gradient) in fp64, with the step's own choices."""
    W, R = head.double().requires_grad_(), router.double().requires_grad_()
    P, E = len(hidden), router.shape[0]
    total = 0.0
    probs, n = [], 0
    for w in range(P):
        x = hidden[w].double()
        logq = torch.log_softmax(x @ W.t() / tau, 1).gather(1, index[w].long())
        p = torch.softmax(teacher[w].double() / tau, 1)
        total = total + (p * (torch.log(p) - logq)).sum(1).mean() / P
        probs.append(torch.softmax(x @ R.t(), 1))
        n += x.shape[0]
    c = step.counts.sum(0).double()
    bal = alpha * E * ((c / (k * n)) * (sum(q.sum(0) for q in probs) / n)).sum()
    (total + bal).backward()
    return total.item(), bal.item(), W.grad, R.grad


@pytest.mark.parametrize("P,T,H,V,E,k", [(2, 150, 200, 900, 12, 2), (3, 300, 256, 9001, 40, 4)])
def test_losses_and_gradients(env, P, T, H, V, E, k):
    torch, g = env
    from gradient_allreduce_homomorphic_gb300.student import StudentStep

    head, router, hidden, index, teacher = make(torch, P, T, H, V, E, 8, 61)
    step = StudentStep(head, router, workers=P, tokens=T, k=k, alpha=2.0, tau=1.5)
    step.run(1, hidden, index, teacher)
    torch.cuda.synchronize()
    loss, bal, dW, dR = exact(torch, step, head, router, hidden, index, teacher, k, 2.0, 1.5)
    got = torch.stack(step.loss).double().mean().item()
    assert abs(got - loss) <= 0.05 * loss
    assert abs(step.balance.item() / P - bal) <= 0.02 * bal  # run with P alpha
    avg = step.averaging.ring_flat[0]
    mine = avg[:V * H].view(V, H).double(), avg[step.router_grad[0].storage_offset():][:E * H].view(E, H).double()
    for a, b in zip(mine, (dW, dR)):
        assert ((a - b).norm() / b.norm()).item() <= 0.15
    want = torch.stack([t for t in step.grads]).double().mean(0)
    assert torch.allclose(avg.double(), want, rtol=1e-5, atol=1e-9)
    thc = step.averaging.thc_flat.double()
    nmse = ((avg.double() - thc).square().sum() / avg.double().square().sum()).item()
    assert abs(step.averaging.nmse.item() - nmse) <= 1e-5 * nmse and g.gar_sync_status() == 0


def test_descent_and_repeatability(env):
    torch, g = env
    from gradient_allreduce_homomorphic_gb300.student import StudentStep

    P, T, H, V, E = 2, 256, 128, 2000, 16
    head, router, hidden, index, teacher = make(torch, P, T, H, V, E, 16, 62)
    step = StudentStep(head, router, workers=P, tokens=T, k=2, alpha=0.1)
    losses = []
    for i in range(8):
        step.run(i, hidden, index, teacher)
        losses.append(torch.stack(step.loss).mean().item())
        avg = step.averaging.ring_flat[0]
        if i == 0:
            before = avg.clone()
            step.run(i, hidden, index, teacher)
            assert torch.equal(before, avg)
        head -= 4.0 * avg[:V * H].view(V, H)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_padding_tokens_do_not_count(env):
    """Tokens without weight and validity: the same losses and weight gradients whatever the teacher says of them."""
    torch, g = env
    from gradient_allreduce_homomorphic_gb300.student import StudentStep

    P, T, H, V, E = 2, 140, 64, 700, 9
    head, router, hidden, index, teacher = make(torch, P, T, H, V, E, 4, 63)
    weight = [torch.full((T,), 0.01, device="cuda") for _ in range(P)]
    valid = [torch.ones(T, dtype=torch.uint8, device="cuda") for _ in range(P)]
    weight[1][100:], valid[1][100:] = 0.0, 0
    outs = []
    for change in (False, True):
        if change:
            teacher[1][100:], index[1][100:] = float("nan"), -1
        step = StudentStep(head, router, workers=P, tokens=T)
        step.run(3, hidden, index, teacher, weight, valid)
        torch.cuda.synchronize()
        outs.append((step.grads, step.counts, step.balance, step.loss))
    for a, b in zip(outs[0][0] + outs[0][3], outs[1][0] + outs[1][3]):
        assert torch.equal(a, b)
    assert torch.equal(outs[0][1], outs[1][1]) and torch.equal(outs[0][2], outs[1][2])
    assert outs[0][1][1].sum().item() == 100 * 2


@pytest.mark.parametrize("P,T,H,V,E,k,weighted", [(1, 150, 200, 900, 12, 2, False), (3, 300, 256, 9001, 40, 4, True)])
def test_reported_losses_and_gradient_of_the_hidden_states(env, P, T, H, V, E, k, weighted):
    """What the class says of its results, in 64 bits: balance is P alpha B, dx the gradient of P F over the hidden states
    (its router's share is checked apart, with a balance loss that outweighs the distillation)."""
    torch, g = env
    from gradient_allreduce_homomorphic_gb300.student import StudentStep

    head, router, hidden, index, teacher = make(torch, P, T, H, V, E, 8, 64)
    weight = valid = None
    gen = torch.Generator(device="cuda").manual_seed(65)
    if weighted:
        weight = [torch.rand(T, generator=gen, device="cuda") / T for _ in range(P)]
        valid = [(torch.rand(T, generator=gen, device="cuda") < 0.9).to(torch.uint8) for _ in range(P)]
    for alpha in (0.5, 5000.0):
        step = StudentStep(head, router, workers=P, tokens=T, k=k, alpha=alpha, tau=1.5)
        step.run(1, hidden, index, teacher, weight, valid)
        torch.cuda.synchronize()
        x = [h.double().requires_grad_() for h in hidden]
        W, R = head.double(), router.double()
        on = [torch.ones(T, device="cuda").double() if valid is None else v.double() for v in valid or hidden]
        n = sum(o.sum() for o in on)
        D, mean_p = [], 0.0
        for w in range(P):
            logq = torch.log_softmax(x[w] @ W.t() / 1.5, 1).gather(1, index[w].long())
            p = torch.softmax(teacher[w].double() / 1.5, 1)
            share = torch.full((T,), 1.0 / T, device="cuda").double() if weight is None else weight[w].double()
            D.append((share * (p * (torch.log(p) - logq)).sum(1)).sum())
            mean_p = mean_p + (on[w][:, None] * torch.softmax(x[w] @ R.t(), 1)).sum(0) / n
            losses = (share * step.loss[w].double()).sum().item()
            assert abs(losses - D[w].item()) <= 0.05 * D[w].item()
        B = E * ((step.counts.sum(0).double() / (k * n)) * mean_p).sum()
        assert abs(step.balance.item() - P * alpha * B.item()) <= 0.02 * P * alpha * B.item()
        (sum(D) / P + alpha * B).backward()
        for w in range(P):
            assert ((step.dx[w].double() - P * x[w].grad).norm() / (P * x[w].grad).norm()).item() <= 0.15
    assert g.gar_sync_status() == 0
