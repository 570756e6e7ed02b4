"""Sure targets of the vocabulary layer's cross entropy: losses near 0 and their
gradients, against the closed form in 64 bits.

x is 1 in its first column alone, so that the logits are w's first column, exactly.
Tolerances, u = 2^-24:
  rest   the sum over all entries but the target, relative to the largest of them: an
         exponential 2^-22 and 2 u log2(e) times its distance (3 at most) from the
         maximum, a batch's 11 additions, the additions of all batches 4 u together,
         30 joins of pairs at most, 7 u each: under 260 u
  d      its logarithm (2 u of it), the maxima's difference and their sum: 4 u |d|
  loss   log1p(exp(d)): relative to exp(d) the above and 8 u; no more of the loss
  g      of the target: the loss's, and 8 u for exp(-loss) - 1 and its weight; of the others:
         lse's absolute error, its rounding u |lse|, 2^-22 and 4 u log2(e) |z - lse|
  dw     g as two bf16 values 2^-16, 2 u a term of the sum (2 for each row)
  dx     g as a bf16 value and the result 2^-8, 2 u a term of the sum  lse    the loss's absolute error or the above, and 2 u of itself"""
import math

import pytest

from helpers import need_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
CASES = [(100.0, 75.0, 32000), (0.0, -20.0, 131072), (30.0, 12.0, 32000), (64.0, 50.0, 5000), (-3.0, -20.0, 131072),
         (40.0, 30.0, 33)]


@pytest.fixture(scope="module")
def env():
    return need_cuda()


def problem(torch, rows, sure, others, vocab, at=7):
    """Logits `sure` for entry `at`, others .. others - 3 in steps of an eighth for the rest; their sum beside the maximum."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(vocab)
    z = others - torch.randint(0, 25, (vocab,), generator=gen, device="cuda") / 8
    z[(at + 1) % vocab] = others
    z[at] = sure
    w = torch.randn((vocab, 8), generator=gen, device="cuda")
    w[:, 0] = z
    x = torch.zeros((rows, 8), device="cuda")
    x[:, 0] = 1.0
    w, x = w.bfloat16(), x.bfloat16()
    z = w[:, 0].double()
    rest = z.clone()
    rest[at] = -math.inf
    return x, w, z, torch.logsumexp(rest, 0).item()


def loss_of(torch, g, x, w, target):
    rows = x.shape[0]
    t = torch.full((rows,), target, dtype=torch.int32, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ws = torch.full((g.gar_vocab_workspace_bytes(rows, w.shape[0], 8, torch.float32),), 255, dtype=torch.uint8, device="cuda")
    g.gar_vocab_loss(x, w, t, loss, lse, ws)
    torch.cuda.synchronize()
    return t, loss, lse, ws


@pytest.mark.parametrize("rows", [1, 300, 19456])
@pytest.mark.parametrize("sure,others,vocab", CASES)
def test_losses_near_zero(env, sure, others, vocab, rows):
    """Of many rows a run takes a row's whole vocabulary: what it adds to a sum of 1 must not be lost."""
    torch, g = env
    x, w, z, rest = problem(torch, rows, sure, others, vocab)
    _, loss, lse, _ = loss_of(torch, g, x, w, 7)
    d = rest - z[7].item()
    want = math.log1p(math.exp(d))
    rel = (260 + 4 * abs(d) + 2 * math.log(vocab) + 8) * U
    assert (loss.double() - want).abs().max().item() <= rel * want
    assert (lse.double() - (z[7].item() + want)).abs().max().item() <= rel * want + 2 * U * abs(z[7].item() + want)


@pytest.mark.parametrize("rows", [1, 19456])
def test_a_sure_mistake(env, rows):
    """All but one entry's probability lies with an entry that is not the target."""
    torch, g = env
    x, w, z, _ = problem(torch, rows, 20.0, 0.0, 131072)
    _, loss, lse, _ = loss_of(torch, g, x, w, 9)
    whole = torch.logsumexp(z, 0).item()
    want = whole - z[9].item()
    assert (lse.double() - whole).abs().max().item() <= 260 * U + 4 * U * whole
    assert (loss.double() - want).abs().max().item() <= 260 * U + 8 * U * want


@pytest.mark.parametrize("dw_type", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("sure,others,vocab", CASES)
def test_gradients_of_sure_targets(env, sure, others, vocab, rows, dw_type):
    """The target's share, of 1e-7 to 1e-2, and with it g's sum of 0 over the vocabulary."""
    torch, g = env
    x, w, z, rest = problem(torch, rows, sure, others, vocab)
    target, loss, lse, ws = loss_of(torch, g, x, w, 7)
    weight = torch.full((rows,), 1.0 / 1024, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(w.shape, dtype=torch.float32 if dw_type == "f32" else torch.bfloat16, device="cuda")
    g.gar_vocab_grad_with_loss(x, w, target, loss, lse, dx, dw, ws, weight=weight)
    torch.cuda.synchronize()
    d = rest - z[7].item()
    want_loss = math.log1p(math.exp(d))
    want = torch.exp(z - (z[7] + want_loss)) / 1024
    want[7] = math.expm1(-want_loss) / 1024
    of_loss = (260 + 4 * abs(d) + 2 * math.log(vocab) + 8) * U
    rel = torch.full_like(z, of_loss * want_loss + 2 * U * (z[7].item() + want_loss) + 2 ** -22)
    rel += 4 * U * 1.4426950408889634 * (z - z[7] - want_loss).abs() + 4 * U
    rel[7] = of_loss + 8 * U
    parts, half = (2 ** -16, U) if dw_type == "f32" else (2 ** -8, 2 ** -8)
    got = dw[:, 0].double()
    assert ((got - rows * want).abs() <= 1.02 * (rel + parts + half + 4 * U * rows) * rows * want.abs()).all()
    tol = ((1.02 * rel + 2 ** -8 + 2 * U * vocab) * want.abs()) @ w.double().abs() * 1.02
    want_dx = want @ w.double()
    assert ((dx.double() - want_dx).abs() <= tol + 2 ** -8 * want_dx.abs()).all()


def test_losses_given_or_not(env):
    """Where no target is sure the losses change nothing but the target's entry, by lse's rounding; rows that do not
    count and NaN among the losses stay theirs."""
    torch, g = env
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randn((200, 96), generator=gen, device="cuda").bfloat16()
    w = (torch.randn((1000, 96), generator=gen, device="cuda") * 0.2).bfloat16()
    target = torch.randint(0, 1000, (200,), generator=gen, device="cuda").int()
    target[::7] = -100
    x[5] = float("inf")
    loss, lse = torch.empty(200, device="cuda"), torch.empty(200, device="cuda")
    ws = torch.empty(g.gar_vocab_workspace_bytes(200, 1000, 96, torch.bfloat16), dtype=torch.uint8, device="cuda")
    g.gar_vocab_loss(x, w, target, loss, lse, ws)
    a, b = torch.empty_like(x), torch.empty_like(x)
    g.gar_vocab_grad(x, w, target, lse, a, None, ws)
    g.gar_vocab_grad_with_loss(x, w, target, loss, lse, b, None, ws)
    torch.cuda.synchronize()
    assert bool((b[::7] == 0).all()) and bool(b[5].isnan().all()) and bool(loss[5].isnan())
    rest = torch.arange(200, device="cuda") != 5
    g64 = torch.softmax(x[rest].double() @ w.double().t(), 1)
    g64.scatter_add_(1, target[rest].clamp(min=0).long()[:, None], -torch.ones((199, 1), dtype=torch.float64, device="cuda"))
    size = g64.abs() @ w.double().abs()  # both: g's rounding and the result's, sums, and lse's error far below them
    assert ((a[rest].double() - b[rest].double()).abs() <= (4 * 2 ** -8 + 1e-3) * size).all()


def test_logits_of_minus_infinity(env):
    """Probability 0: the loss of another target is as if the entry were not there, its own is +inf; its share of dw is
    -weight x where it is the target and 0 elsewhere."""
    torch, g = env
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    x = torch.randn((300, 64), generator=gen, device="cuda").abs().add_(0.5).bfloat16()
    w = (torch.randn((900, 64), generator=gen, device="cuda") * 0.2).bfloat16()
    gone = [3, 700]
    w[gone, 5] = float("-inf")
    target = torch.randint(4, 700, (300,), generator=gen, device="cuda").int()
    target[::9] = 700
    lost = target == 700
    loss, lse = torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
    ws = torch.empty(g.gar_vocab_workspace_bytes(300, 900, 64, torch.float32), dtype=torch.uint8, device="cuda")
    g.gar_vocab_loss(x, w, target, loss, lse, ws)
    kept = torch.ones(900, dtype=torch.bool, device="cuda")
    kept[gone] = False
    z = x.double() @ w.double()[kept].t()
    size = x.double().abs() @ w.double()[kept].abs().t()
    ez = 2 * U * 64 * size.amax(1)
    want = torch.logsumexp(z, 1)
    tol = 2 * ez + 260 * U + 8 * U * (1 + want.abs())
    assert ((lse.double() - want).abs() <= tol).all() and bool((loss[lost] == float("inf")).all())
    place = torch.cumsum(kept, 0)[target.long()] - 1
    of_row = want - z.gather(1, place[:, None])[:, 0]
    assert ((loss.double() - of_row).abs() <= tol + 2 * ez + 8 * U * of_row)[~lost].all()
    for grad in (lambda dw: g.gar_vocab_grad(x, w, target, lse, None, dw, ws),
                 lambda dw: g.gar_vocab_grad_with_loss(x, w, target, loss, lse, None, dw, ws)):
        dw = torch.empty((900, 64), device="cuda")
        grad(dw)
        want_dw = -x[lost].double().sum(0)
        assert bool(torch.isfinite(dw).all()) and bool((dw[3] == 0).all())
        assert ((dw[700].double() - want_dw).abs() <= (2 ** -16 + 2 * U * 600) * want_dw.abs()).all()
