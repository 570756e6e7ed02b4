"""The workers' language-model step (language.LanguageStep) and the averaging step's
clipping: losses and gradients against 64-bit autograd of the same model without
quantisation, with the step's own choices.

Tolerance: rounding a value to e4m3 is off by 2.6% in the mean square (2^-4 over sqrt
3, and the significand's spread), to e5m2 by 5.3%.  The experts' rows and the router's
logits carry two e4m3 roundings, a weight gradient an e4m3 and an e5m2 one besides:
15% of the gradient's norm covers them.  The head's gradient is exact but for bf16 h
and the experts' rows."""
import numpy as np
import pytest

from helpers import need_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return need_cuda()


def make(torch, P, T, H, V, E, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    head = (torch.randn((V, H), generator=g, device="cuda") * 0.2).bfloat16()
    router = torch.randn((E, H), generator=g, device="cuda") * 0.2
    experts = torch.randn((E, H, H), generator=g, device="cuda") * H ** -0.5
    hidden = [torch.randn((T, H), generator=g, device="cuda").bfloat16() for _ in range(P)]
    target = [torch.randint(0, V, (T,), generator=g, device="cuda").int() for _ in range(P)]
    for t in target:
        t[::17] = -100
    return head, router, experts, hidden, target


def exact(torch, step, head, router, experts, hidden, target, weight):
    """Losses per worker, P F, and its gradient over head, router, experts and hidden states, in fp64."""
    leaves = [t.double().requires_grad_() for t in (head, router, experts)]
    W, R, U = leaves
    xs = [h.double().requires_grad_() for h in hidden]
    P, E, k, n = len(xs), R.shape[0], step.k, sum(h.shape[0] for h in hidden)
    total, mean_p, losses = 0.0, 0.0, []
    for w, x in enumerate(xs):
        r = x @ R.t()
        choice = step.choice[w].long()
        share = torch.softmax(r.gather(1, choice), 1) * (step.position[w] >= 0)
        h = x
        for j in range(k):
            h = h + share[:, j:j + 1] * torch.einsum("th,toh->to", x, U[choice[:, j]])
        on = (target[w] >= 0) & (weight[w] != 0)
        logp = torch.log_softmax(h @ W.t(), 1).gather(1, target[w].long().clamp(min=0)[:, None])[:, 0]
        losses.append(torch.where(on, -logp, 0.0))
        total = total + (losses[-1] * weight[w].double()).sum()
        mean_p = mean_p + torch.softmax(r, 1).sum(0) / n
    bal = step.alpha * E * ((step.counts.sum(0).double() / (k * n)) * mean_p).sum()
    (total + P * bal).backward()
    return losses, P * bal.item(), [t.grad / P for t in leaves], [x.grad for x in xs]


def near(a, b, tol):
    return ((a.double() - b).norm() / b.norm()).item() <= tol


@pytest.mark.parametrize("P,T,H,V,E,k,capacity,alpha", [(2, 150, 64, 900, 8, 2, 0, 1.0), (3, 260, 136, 3001, 12, 3, 50, 0.1)])
def test_losses_and_gradients(env, P, T, H, V, E, k, capacity, alpha):
    torch, g = env
    from gradient_allreduce_homomorphic_gb300.language import LanguageStep

    head, router, experts, hidden, target = make(torch, P, T, H, V, E, 71)
    weight = [torch.rand(T, device="cuda") / T for _ in range(P)]
    step = LanguageStep(head, router, experts, workers=P, tokens=T, k=k, capacity=capacity, alpha=alpha)
    step.run(1, hidden, target, weight)
    torch.cuda.synchronize()
    if capacity:
        assert bool((torch.stack(step.position) < 0).any())  # some choices are over it
    losses, bal, (dW, dR, dU), dx = exact(torch, step, head, router, experts, hidden, target, weight)
    for w in range(P):
        assert near(step.loss[w], losses[w], 0.05) and bool((step.loss[w][target[w] < 0] == 0).all())
        assert near(step.dx[w], dx[w], 0.15)
    assert abs(step.balance.item() - bal) <= 0.02 * bal
    avg = step.averaging.ring_flat[0]
    at = lambda v: avg[v.storage_offset():][:v.numel()].view(v.shape)  # noqa: E731
    for view, want in ((step.head_grad[0], dW), (step.router_grad[0], dR), (step.expert_grad[0], dU)):
        assert near(at(view), want, 0.15)
    assert g.gar_sync_status() == 0


def test_the_same_bits_again_and_in_a_graph(env):
    torch, g = env
    from gradient_allreduce_homomorphic_gb300.language import LanguageStep

    P, T, H, V, E = 2, 200, 64, 1000, 8
    head, router, experts, hidden, target = make(torch, P, T, H, V, E, 72)
    step = LanguageStep(head, router, experts, workers=P, tokens=T, max_norm=0.05)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (*step.averaging.ring_flat, step.averaging.thc_flat, *step.dx, *step.loss, step.counts,
                                    step.averaging.norm)]

    step.run(5, hidden, target)
    want = results()
    step.run(5, hidden, target)
    assert all(torch.equal(a, b) for a, b in zip(want, results()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run(5, hidden, target)
    for t in (*step.averaging.ring_flat, *step.dx, *step.loss):
        t.fill_(7.0)
    for _ in range(2):
        graph.replay()
        got = results()
    flat = step.averaging  # the gaps between the tensors were filled too: only what the step writes is compared
    for a, b, is_flat in zip(want, got, [True] * (P + 1) + [False] * (len(want) - P - 1)):
        if is_flat:
            assert all(torch.equal(x, y) for x, y in zip(flat._views(a), flat._views(b)))
        else:
            assert torch.equal(a, b)
    assert g.gar_sync_status() == 0


def test_padding_tokens_do_not_count(env):
    """Tokens without weight and validity: whatever their targets and (finite) hidden states, the others' results stay."""
    torch, g = env
    from gradient_allreduce_homomorphic_gb300.language import LanguageStep

    P, T, H, V, E = 2, 140, 64, 700, 8
    head, router, experts, hidden, target = make(torch, P, T, H, V, E, 73)
    weight = [torch.full((T,), 0.01, device="cuda") for _ in range(P)]
    valid = [torch.ones(T, dtype=torch.uint8, device="cuda") for _ in range(P)]
    weight[1][100:], valid[1][100:] = 0.0, 0
    outs = []
    for change in (False, True):
        if change:
            target[1][100:] = 3
            hidden[1][100:] = hidden[1][100:] * 0.5
        step = LanguageStep(head, router, experts, workers=P, tokens=T)
        step.run(3, hidden, target, weight, valid)
        torch.cuda.synchronize()
        outs.append((step.loss, [d[:100] for d in step.dx], [step.counts, step.balance]))
        assert bool((step.choice[1][100:] == -1).all()) and bool((step.position[1][100:] == -1).all())
        assert bool((step.loss[1][100:] == 0).all()) and bool((step.dx[1][100:] == 0).all())
    for a, b in zip(outs[0], outs[1]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("nmse", ["fused", "separate"])
def test_averages_clipped(env, nmse):
    """max_norm scales both averages by their own norms, after the NMSE; what was not above it stays bit for bit."""
    torch, g = env
    from gradient_allreduce_homomorphic_gb300.pipeline import AveragingStep, flat_offsets

    sizes = np.array([1000, 37, 70000, 5], np.int64)
    offs = flat_offsets(sizes)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    grads = [torch.randn(int(offs[-1]), generator=gen, device="cuda") for _ in range(3)]
    for f in grads:
        for i, s in enumerate(sizes):
            f[int(offs[i] + s):int(offs[i + 1])] = 0.0
    plain = AveragingStep(grads, sizes, offs, nmse=nmse)
    plain.run(4)
    torch.cuda.synchronize()
    norms = [math_norm(f) for f in (plain.ring_flat[0], plain.thc_flat)]
    for max_norm, schedule in ((0.5 * norms[0], "overlap"), (0.5 * norms[0], "serial"), (2 * max(norms), "overlap")):
        step = AveragingStep(grads, sizes, offs, nmse=nmse, max_norm=max_norm)
        step.run(4, schedule=schedule)
        torch.cuda.synchronize()
        assert step.nmse.item() == plain.nmse.item()
        for norm, want, flats, base in ((step.norm, norms[0], step.ring_flat, plain.ring_flat),
                                        (step.thc_norm, norms[1], [step.thc_flat], [plain.thc_flat])):
            assert abs(norm.item() - want) <= 4 * 2.0 ** -24 * want
            for a, b in zip(flats, base):
                if want <= max_norm:
                    assert torch.equal(a, b)
                else:
                    c = b.double() * (max_norm / want)
                    assert bool(((a.double() - c).abs() <= 8 * 2.0 ** -24 * c.abs()).all())
    step.setup_host()
    with pytest.raises(RuntimeError):
        step.run_from_host(1, [])
    with pytest.raises(ValueError):
        AveragingStep(grads, sizes, offs, max_norm=-1.0)
    assert g.gar_sync_status() == 0


def math_norm(t):
    return t.double().square().sum().sqrt().item()
