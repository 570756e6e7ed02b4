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
  lse    the loss's absolute error or the above, and 2 u of itself"""
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
