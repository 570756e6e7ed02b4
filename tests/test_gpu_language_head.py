"""The language step's head, whose gradient no 8-bit product meets: against 64 bits
from the step's own hidden states h (bf16), its targets and weights.

Tolerance: g is the sum of two bf16 values (2^-16 of it at most, mean square below
2^-17), exp(z - lse) is within 1e-6 at these logits, the sums' truncation within 2^-23 a
term of a few hundred; the averages over the workers add u each.  1e-5 of the gradient's
norm covers them.  Of the loss: 2^-23 hidden of the logits' products, 300 u of lse."""
import pytest

from helpers import need_cuda
from test_gpu_language import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,T,H,V,E,k,weighted", [(2, 150, 64, 900, 8, 2, False), (3, 260, 136, 3001, 12, 3, True)])
def test_heads_gradient_and_losses(P, T, H, V, E, k, weighted):
    torch, g = need_cuda()
    from gradient_allreduce_homomorphic_gb300.language import LanguageStep

    head, router, experts, hidden, target = make(torch, P, T, H, V, E, 74)
    weight = [torch.rand(T, device="cuda") / T for _ in range(P)] if weighted else None
    if weighted:
        weight[0][5:9] = 0.0
    step = LanguageStep(head, router, experts, workers=P, tokens=T, k=k)
    step.run(1, hidden, target, weight)
    torch.cuda.synchronize()
    W, total = head.double(), 0.0
    for w in range(P):
        share = (weight[w] if weighted else torch.full((T,), 1.0 / T, device="cuda")).double()
        on = (target[w] >= 0) & (share != 0)
        x = step.h[w].double()
        z = x @ W.t()
        at = target[w].long().clamp(min=0)[:, None]
        loss = torch.logsumexp(z, 1) - z.gather(1, at)[:, 0]
        tol = 4 * H * 2.0 ** -24 * (x.abs() @ W.abs().t()).amax(1) + 300 * 2.0 ** -24 * (1 + loss)
        assert ((step.loss[w].double() - torch.where(on, loss, 0.0)).abs() <= tol).all()
        G = torch.softmax(z, 1).scatter_add(1, at, -torch.ones_like(at, dtype=torch.float64)) * (share * on)[:, None]
        want = G.t() @ x
        assert (step.head_grad[w].double() - want).norm() <= 1e-5 * want.norm()
        rows = G.abs().t() @ x.abs()  # and no row far off on its own
        assert ((step.head_grad[w].double() - want).abs() <= 1e-4 * rows + 1e-12).all()
        total = total + want / P
    view = step.head_grad[0]
    average = step.averaging.ring_flat[0][view.storage_offset():][:view.numel()].view(V, H)
    assert (average.double() - total).norm() <= 1e-5 * total.norm()
    assert g.gar_sync_status() == 0
