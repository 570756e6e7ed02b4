"""The vocabulary layer's cross entropy and its gradient (gar_vocab_loss,
gar_vocab_grad) against the plain form in 64 bits.

Tolerances, each counted from the roundings on the way.  u = 2^-24 is fp32's half
step; the tensor cores' additions round toward zero, 2u each.
  z      h products, exact, added one by one at most: 2 u h sum_h |x w| = ez
  exp    2^-22 of itself from the instruction, and its exponent (z - m) log2(e) is
         formed in two roundings: 2 u log2(e) |z - m|
  sums   a batch of 32 columns adds 11 terms after one another and may be scaled
         once (2^-22): V / 64 batches of (11 u + 2^-22) at most
  lse    the above relative to the sum, so absolute in its logarithm, and the
         rounding of the logarithm, of m and of their sum
  g      weight p (2 ez + else + 2^-22 + 2 u (1 + |z - lse| log2(e))), and rounded to
         bf16 (2^-8 of it), or to two bf16 values (2^-16)
  dx, dw the products' share of g's error, 2 u a term of the sums, one rounding to
         the result's type (half of its eps)."""
import numpy as np
import pytest

from helpers import need_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LOG2E = 1.4426950408889634


@pytest.fixture(scope="module")
def env():
    return need_cuda()


class Problem:
    """Inputs (views into wider buffers where pad > 0) and the outputs' and bounds' 64-bit values."""

    def __init__(self, torch, rows, vocab, hidden, seed=0, pad=0, scale=2.0, masked=0.1, weighted=True):
        self.torch, self.rows, self.vocab, self.hidden = torch, rows, vocab, hidden
        g = torch.Generator(device="cuda")
        g.manual_seed(1000 * seed + rows + vocab + hidden)
        ld = (hidden + 7) // 8 * 8 + pad

        def matrix(n, s):
            return (torch.randn((n, ld), generator=g, device="cuda") * s).bfloat16()[:, :hidden]

        self.x, self.w = matrix(rows, 1.0), matrix(vocab, scale / hidden ** 0.5)
        target = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        away = torch.rand(rows, generator=g, device="cuda") < masked
        target[away] = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, -100, vocab)[away]
        self.target = target.to(torch.int32)
        self.weight = (torch.rand(rows, generator=g, device="cuda") + 0.5) / rows if weighted else None
        if weighted and rows > 3:
            self.weight[3] = 0.0
        self.gen = g

    def live(self):
        ok = (self.target >= 0) & (self.target < self.vocab)
        return ok if self.weight is None else ok & (self.weight != 0)

    def reference(self):
        torch = self.torch
        on = self.live()
        x = torch.where(on[:, None], self.x, 0).double()
        w = self.w.double()
        weight = torch.where(on, 1.0 if self.weight is None else self.weight.double(), 0.0)
        z = x @ w.t()
        ez = 2 * U * self.hidden * (x.abs() @ w.abs().t())
        lse = torch.logsumexp(z, 1)
        at = self.target.long().clamp(0, self.vocab - 1)[:, None]
        top = z.amax(1)
        low = (top[:, None] - z).clamp(max=60.0)  # powers below that are nothing
        p = torch.exp(z - lse[:, None])
        e_exp = 2 ** -22 + 2 * U * LOG2E * low + 2 * ez
        e_lse = (p * e_exp).sum(1) + (self.vocab / 64 + 40) * (11 * U + 2 ** -22) + 4 * U * (lse.abs() + top.abs() + 1)
        self.lse, self.e_lse = torch.where(on, lse, 0.0), torch.where(on, e_lse, 0.0)
        self.loss = torch.where(on, lse - z.gather(1, at)[:, 0], 0.0)
        self.e_loss = torch.where(on, e_lse + ez.gather(1, at)[:, 0] + 4 * U * self.loss.abs(), 0.0)
        g = p.clone()
        g.scatter_add_(1, at, -torch.ones_like(at, dtype=torch.float64))
        g *= weight[:, None]
        e_g = weight.abs()[:, None] * p * (2 * ez + e_lse[:, None] + 2 ** -22 + 4 * U * (1 + LOG2E * (lse[:, None] - z).abs()))
        e_g += 4 * U * g.abs()
        self.g, self.e_g, self.x64, self.w64 = g, e_g, x, w
        return self

    def gradients(self, dw_type, addend=None):
        """dx, dw and their bounds."""
        torch = self.torch
        half = torch.finfo(dw_type).eps / 2
        of_g = 2.0 ** -16 if dw_type == torch.float32 else 2.0 ** -8
        dx, dw = self.g @ self.w64, self.g.t() @ self.x64
        big_dx, big_dw = self.g.abs() @ self.w64.abs(), self.g.abs().t() @ self.x64.abs()
        e_dx = 1.02 * (self.e_g @ self.w64.abs()) + (2.0 ** -8 * 1.02 + 2 * U * (self.vocab + 80)) * big_dx
        e_dw = 1.02 * (self.e_g.t() @ self.x64.abs()) + (of_g * 1.02 + 2 * U * (2 * self.rows + 80)) * big_dw
        if addend is not None:
            dw = dw + addend.double()
            e_dw = e_dw + 2 * U * addend.double().abs()
        return dx, e_dx * 1.01 + 2.0 ** -8 * dx.abs(), dw, e_dw * 1.01 + half * dw.abs()


def within(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol + 1e-30)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, the first {got[bad][0].item()} for " \
                                f"{want[bad][0].item()} (within {tol[bad][0].item()})"


def workspace(torch, g, p, dw_type):
    n = g.gar_vocab_workspace_bytes(p.rows, p.vocab, p.hidden, dw_type)
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN as any float


def outputs(torch, p, dw_type, pad=0):
    full = lambda n, t: torch.full((n, p.hidden + pad), 7.0, dtype=t, device="cuda")  # noqa: E731
    return (torch.full((p.rows,), 7.0, device="cuda"), torch.full((p.rows,), 7.0, device="cuda"), full(p.rows, torch.bfloat16),
            full(p.vocab, dw_type))


def run(torch, g, p, dw_type, addend=None, pad=0, stream=None):
    loss, lse, dx, dw = outputs(torch, p, dw_type, pad)
    ws = workspace(torch, g, p, dw_type)
    h = p.hidden
    torch.cuda.synchronize()
    g.gar_vocab_loss(p.x, p.w, p.target, loss, lse, ws, weight=p.weight, stream=stream)
    g.gar_vocab_grad(p.x, p.w, p.target, lse, dx[:, :h], dw[:, :h], ws, weight=p.weight, addend=addend, stream=stream)
    torch.cuda.synchronize()
    assert g.gar_sync_status() == 0
    assert bool((dx[:, h:] == 7).all()) and bool((dw[:, h:] == 7).all()), "written past a row"
    return loss, lse, dx[:, :h], dw[:, :h]


def check(torch, g, p, dw_type, addend=None, pad=0, stream=None):
    loss, lse, dx, dw = run(torch, g, p, dw_type, addend, pad, stream)
    p.reference()
    within(loss, p.loss, p.e_loss, "loss")
    within(lse, p.lse, p.e_lse, "lse")
    want_dx, e_dx, want_dw, e_dw = p.gradients(dw_type, addend)
    within(dx, want_dx, e_dx, "dx")
    within(dw, want_dw, e_dw, "dw")
    off = ~p.live()
    assert bool((loss[off] == 0).all()) and bool((lse[off] == 0).all()) and bool((dx[off] == 0).all())
    return loss, lse, dx, dw


SIZES = [(1, 1, 1), (1, 300, 8), (3, 257, 64), (2, 33, 7), (255, 256, 72), (256, 255, 120), (257, 1000, 1000), (130, 4099, 264),
         (129, 512, 513), (64, 32, 2056), (700, 2049, 100)]


@pytest.mark.parametrize("dw", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,hidden", SIZES)
def test_against_64_bits(env, rows, vocab, hidden, dw):
    torch, g = env
    check(torch, g, Problem(torch, rows, vocab, hidden), torch.float32 if dw == "f32" else torch.bfloat16)


@pytest.mark.parametrize("dw", ["f32", "bf16"])
def test_strides_and_addend(env, dw):
    torch, g = env
    t = torch.float32 if dw == "f32" else torch.bfloat16
    p = Problem(torch, 300, 777, 200, seed=1, pad=24)
    add = (torch.randn((777, 211), generator=p.gen, device="cuda") * 1e-3).to(t)[:, 5:205]
    check(torch, g, p, t, addend=add, pad=3)


@pytest.mark.parametrize("dw", ["f32", "bf16"])
def test_addend_in_place(env, dw):
    torch, g = env
    t = torch.float32 if dw == "f32" else torch.bfloat16
    p = Problem(torch, 100, 520, 128, seed=2, weighted=False).reference()
    before = (torch.randn((520, 128), generator=p.gen, device="cuda")).to(t)
    acc, ws = before.clone(), workspace(torch, g, p, t)
    loss, lse, dx, _ = outputs(torch, p, t)
    g.gar_vocab_loss(p.x, p.w, p.target, loss, lse, ws)
    g.gar_vocab_grad(p.x, p.w, p.target, lse, None, acc, ws, addend=acc)
    g.gar_vocab_grad(p.x, p.w, p.target, lse, dx, None, ws)
    want_dx, e_dx, want_dw, e_dw = p.gradients(t, before)
    within(dx, want_dx, e_dx, "dx alone")
    within(acc, want_dw, e_dw, "dw alone")


@pytest.mark.parametrize("dw", ["f32", "bf16"])
def test_several_pieces_of_the_vocabulary(env, dw):
    """g of 4500 x 31000 takes more than a piece's 256 MB, so dx is a sum over pieces."""
    torch, g = env
    check(torch, g, Problem(torch, 4500, 31000, 40), torch.float32 if dw == "f32" else torch.bfloat16)


def test_long_sums_of_an_fp32_dw(env):
    """More rows than one accumulator adds up; x with a mean, so that the sums grow all along."""
    torch, g = env
    p = Problem(torch, 9000, 700, 64, seed=3)
    p.x.add_(0.5)
    check(torch, g, p, torch.float32)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_that_do_not_count_are_not_seen(env, bad):
    torch, g = env
    p = Problem(torch, 260, 900, 136, seed=4, masked=0.3)
    p.x[~p.live()] = bad
    loss, lse, dx, dw = run(torch, g, p, torch.bfloat16)
    q = Problem(torch, 260, 900, 136, seed=4, masked=0.3).reference()
    want_dx, e_dx, want_dw, e_dw = q.gradients(torch.bfloat16)
    within(loss, q.loss, q.e_loss, "loss")
    within(dx, want_dx, e_dx, "dx")
    within(dw, want_dw, e_dw, "dw")


def test_no_row_counts(env):
    torch, g = env
    p = Problem(torch, 70, 600, 96, seed=5)
    p.target.fill_(-1)
    p.x.fill_(float("nan"))
    loss, lse, dx, dw = run(torch, g, p, torch.float32)
    for t in (loss, lse, dx, dw):
        assert bool((t == 0).all())


@pytest.mark.parametrize("dw", ["f32", "bf16"])
def test_no_rows(env, dw):
    torch, g = env
    t = torch.float32 if dw == "f32" else torch.bfloat16
    p = Problem(torch, 0, 100, 40)
    add = torch.randn((100, 40), device="cuda").to(t)
    assert torch.equal(run(torch, g, p, t, addend=add)[3], add)
    assert bool((run(torch, g, p, t)[3] == 0).all())


def test_a_nan_stays_in_its_row_of_the_loss(env):
    torch, g = env
    p = Problem(torch, 300, 700, 64, seed=6, masked=0.0)
    clean, _, _, _ = run(torch, g, p, torch.bfloat16)
    p.x[17, 5] = float("nan")
    p.x[18, 5] = float("inf")
    loss, lse, dx, dw = run(torch, g, p, torch.bfloat16)
    hit = torch.zeros(300, dtype=torch.bool, device="cuda")
    hit[17:19] = True
    assert bool(loss[hit].isnan().all()) and torch.equal(loss[~hit], clean[~hit])
    assert bool(dx[17].isnan().all()) and not bool(dx[~hit].isnan().any()) and bool(dw.isnan().all())


@pytest.mark.parametrize("scale", [60.0, 1e-4])
def test_large_and_small_logits(env, scale):
    torch, g = env
    check(torch, g, Problem(torch, 200, 1500, 128, seed=7, scale=scale), torch.float32)


def test_a_vocabulary_of_one_and_sure_targets(env):
    """Loss and gradient 0 exactly where the target has all the probability, however large its logit."""
    torch, g = env
    p = Problem(torch, 40, 1, 64, seed=12, scale=30.0)
    for t in run(torch, g, p, torch.bfloat16)[::2]:
        assert bool((t == 0).all())
    q = Problem(torch, 40, 300, 64, seed=12, masked=0.0, weighted=False)
    q.w.zero_()
    q.w[7] = 4.0
    q.x.copy_(q.x.abs() + 1)  # z = 4 sum |x| + 256 for entry 7, 0 for all others
    q.target.fill_(7)
    loss, lse, dx, dw = run(torch, g, q, torch.float32)
    assert bool((loss == 0).all()) and bool((dx == 0).all()) and bool((dw[7] == 0).all())
    assert bool((lse == (q.x.double() @ q.w.double()[7]).float()).all())


def test_rows_far_apart(env):
    """Offsets past 2^31 elements in w and dw."""
    torch, g = env
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")
    p = Problem(torch, 40, 2100, 72, seed=8)
    wide = torch.empty((2100, 1 << 20), dtype=torch.bfloat16, device="cuda")
    w, wide[:, :72] = p.w, p.w
    p.w = wide[:, :72]
    loss, lse, dx, _ = outputs(torch, p, torch.bfloat16)
    ws = workspace(torch, g, p, torch.bfloat16)
    dw = wide[:, 80:152]
    g.gar_vocab_loss(p.x, p.w, p.target, loss, lse, ws, weight=p.weight)
    g.gar_vocab_grad(p.x, p.w, p.target, lse, dx, dw, ws, weight=p.weight)
    p.w = w
    p.reference()
    want_dx, e_dx, want_dw, e_dw = p.gradients(torch.bfloat16)
    within(loss, p.loss, p.e_loss, "loss")
    within(dx, want_dx, e_dx, "dx")
    within(dw, want_dw, e_dw, "dw")


def test_the_same_bits_in_every_run(env):
    torch, g = env
    p = Problem(torch, 1003, 5001, 264, seed=9)
    first = run(torch, g, p, torch.float32)
    for _ in range(3):
        for a, b in zip(first, run(torch, g, p, torch.float32)):
            assert torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                               b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))


def test_gradient_against_differences(env):
    """The loss along a direction d of 1/16 steps that bf16 holds: (F(x + d) - F(x - d)) / 2 = <dF/dx, d> + third
    order.  With logits changed by at most a, that is under the total weight times a^3 (|F'''| <= 2 a^3 for a softmax);
    the losses' own errors add."""
    torch, g = env
    p = Problem(torch, 64, 600, 128, seed=10)
    _, _, dx, _ = run(torch, g, p, torch.float32)
    p.reference()
    e_dx = p.gradients(torch.float32)[1]
    p.x.copy_(((p.x.float() * 16).round() / 16).clamp(-2, 2))
    _, _, dx, dw = run(torch, g, p, torch.float32)
    p.reference()
    _, e_dx, _, _ = p.gradients(torch.float32)
    step = 2.0 ** -6
    d = torch.where(torch.rand(p.x.shape, generator=p.gen, device="cuda") < 0.5, -step, step)
    x = p.x.clone()
    total, e = [], 0.0
    weight = p.weight.double()
    for sign in (1, -1):
        p.x = (x.float() + sign * d).bfloat16()
        assert torch.equal(p.x.float(), x.float() + sign * d)  # held exactly
        loss = run(torch, g, p, torch.float32)[0]
        p.reference()
        e += (p.e_loss * weight).sum().item() / 2
        total.append((loss.double() * weight).sum().item())
    along = (dx.double() * d.double()).sum().item()
    a = (d.double() @ p.w64.t()).abs().amax().item()
    tol = e + (e_dx * d.double().abs()).sum().item() + weight.sum().item() * 2 * a ** 3
    assert abs((total[0] - total[1]) / 2 - along) <= tol
    assert abs(along) > 0


def test_other_stream_and_captured_graph(env):
    """Two captured calls share a workspace with eager ones of the same inputs and follow inputs written in place."""
    torch, g = env
    p = Problem(torch, 150, 3000, 128, seed=11)
    side = torch.cuda.Stream()
    want = run(torch, g, p, torch.bfloat16)
    for a, b in zip(want, run(torch, g, p, torch.bfloat16, stream=side)):
        assert torch.equal(a, b)
    loss, lse, dx, dw = outputs(torch, p, torch.bfloat16)
    ws = workspace(torch, g, p, torch.bfloat16)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.gar_vocab_loss(p.x, p.w, p.target, loss, lse, ws, weight=p.weight)
            g.gar_vocab_grad(p.x, p.w, p.target, lse, dx, dw, ws, weight=p.weight)
        graphs.append(graph)
    for graph in graphs:
        for t in (loss, lse, dx, dw):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (loss, lse, dx, dw)):
            assert torch.equal(a, b)
    p.x.neg_()
    want = run(torch, g, p, torch.bfloat16)
    graphs[0].replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (loss, lse, dx, dw)):
        assert torch.equal(a, b)
    assert np.isfinite(loss.sum().item())


def test_two_calls_at_once(env):
    """Calls on two streams, each with its workspace, beside 8-bit products on a third."""
    torch, g = env
    problems = [Problem(torch, 700, 9001, 256, seed=20), Problem(torch, 40, 30001, 512, seed=21)]
    want = [run(torch, g, p, torch.float32) for p in problems]
    a, sa = g.fp8_matrix(300, 2048)
    b, sb = g.fp8_matrix(1000, 2048)
    for m, s in ((a, sa), (b, sb)):
        g.gar_fp8_quantize(torch.randn(m.shape, generator=problems[0].gen, device="cuda"), m, s)
    product, other = torch.empty((300, 1000), device="cuda"), torch.empty((300, 1000), device="cuda")
    g.gar_fp8_matmul(a, sa, b, sb, product)
    streams = [torch.cuda.Stream() for _ in range(3)]
    made = [(outputs(torch, p, torch.float32), workspace(torch, g, p, torch.float32)) for p in problems]
    torch.cuda.synchronize()
    for _ in range(10):
        for p, (o, ws), s in zip(problems, made, streams):
            g.gar_vocab_loss(p.x, p.w, p.target, o[0], o[1], ws, weight=p.weight, stream=s)
            g.gar_vocab_grad(p.x, p.w, p.target, o[1], o[2], o[3], ws, weight=p.weight, stream=s)
        g.gar_fp8_matmul(a, sa, b, sb, other, stream=streams[2])
    torch.cuda.synchronize()
    assert g.gar_sync_status() == 0 and torch.equal(product, other)
    for w, (o, _) in zip(want, made):
        assert all(torch.equal(x, y) for x, y in zip(w, o))
