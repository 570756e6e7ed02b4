"""Tokens sorted by expert and back, and the chosen experts' weights, against plain
loops and sums in 64 bits.

Tolerances: positions, sources, offsets and copies are exact.  A combined row is k
products and sums in fp32 (2^-24 each, of the absolute sum) and one rounding to its
type; dweight a sum of `hidden` products (at most hidden roundings of the absolute
sum); a row's gradient one product and one rounding.  A weight is a quotient of
powers within 2^-21 of themselves (and 2^-23 of |z - top| each for the difference)
and of their sum; its gradient three products and k sums of those."""
import numpy as np
import pytest

from helpers import need_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    return need_cuda()


def half(torch, t):
    return torch.finfo(t).eps / 2


def choices(rng, P, tokens, k, experts, none=0.1, twice=False):
    c = np.full((P, tokens, k), -1, np.int32)
    for w in range(P):
        for t in range(tokens):
            if rng.random() >= none:
                c[w, t] = rng.integers(0, experts, k) if twice or k > experts else rng.permutation(experts)[:k]
    if tokens and k > 1:
        c[0, -1, k - 1] = -1     # a choice that lacks
        c[-1, 0, 0] = experts    # and one that is none of the experts
    return c


def sort(c, experts, align, capacity, rows):
    """(position, source, offsets) by a loop over the pairs."""
    of = [[] for _ in range(experts)]
    for i, e in enumerate(c.reshape(-1)):
        if 0 <= e < experts:
            of[e].append(i)
    position, source, offsets = np.full(c.size, -1, np.int32), np.full(rows, -2, np.int32), [0]
    for pairs in of:
        size = capacity if capacity else -(-len(pairs) // align) * align
        kept = pairs[:capacity] if capacity else pairs
        first = offsets[-1]
        source[first:first + size] = -1
        for r, i in enumerate(kept):
            position[i], source[first + r] = first + r, i
        offsets.append(first + size)
    return position.reshape(c.shape), source, np.array(offsets, np.int32)


def sorted_on_gpu(torch, g, c, experts, align=1, capacity=0, extra=0, table=False, stream=None):
    P, tokens, k = c.shape
    rows = g.gar_expert_rows(P, tokens, k, experts, align, capacity) + extra
    choice = [torch.from_numpy(c[w].copy()).cuda() for w in range(P)]
    position = [torch.full((tokens, k), 77, dtype=torch.int32, device="cuda") for _ in range(P)]
    source = torch.full((rows,), 77, dtype=torch.int32, device="cuda")
    offsets = torch.full((experts + 1,), 77, dtype=torch.int32, device="cuda")
    ws = torch.full((g.gar_expert_workspace_bytes(P, tokens, k, experts),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g.gar_expert_sort(g.pointer_table(choice) if table else choice, experts, g.pointer_table(position) if table else position, source,
                      offsets, ws, align=align, capacity=capacity, stream=stream)
    torch.cuda.synchronize()
    return position, source, offsets


SORTS = [(1, 1, 1, 1), (1, 1, 1, 5), (1, 16, 2, 8), (2, 300, 4, 60), (1, 1025, 8, 256), (3, 1000, 3, 1024), (1, 513, 32, 33),
         (64, 40, 2, 16), (8, 4096, 8, 256), (1, 20001, 1, 3)]


@pytest.mark.parametrize("align,capacity", [(1, 0), (128, 0), (7, 0), (1, 3), (1, 1000)])
@pytest.mark.parametrize("P,tokens,k,experts", SORTS)
def test_sort(env, P, tokens, k, experts, align, capacity):
    torch, g = env
    rng = np.random.default_rng([501, P, tokens, k, experts])
    c = choices(rng, P, tokens, k, experts)
    position, source, offsets = sorted_on_gpu(torch, g, c, experts, align, capacity, extra=5)
    want = sort(c, experts, align, capacity, source.numel())
    assert np.array_equal(torch.stack(position).cpu().numpy(), want[0])
    assert np.array_equal(source.cpu().numpy(), want[1])
    assert np.array_equal(offsets.cpu().numpy(), want[2])


def test_sort_of_one_expert_of_none_and_of_repeats(env):
    torch, g = env
    for c in (np.zeros((2, 5000, 2), np.int32), np.full((2, 700, 3), -1, np.int32), np.full((1, 0, 2), 0, np.int32),
              choices(np.random.default_rng(5), 1, 3000, 4, 2, twice=True)):
        position, source, offsets = sorted_on_gpu(torch, g, c, 4, align=8, table=True)
        want = sort(c, 4, 8, 0, source.numel())
        assert np.array_equal(torch.stack(position).cpu().numpy(), want[0])
        assert np.array_equal(source.cpu().numpy(), want[1]) and np.array_equal(offsets.cpu().numpy(), want[2])


class Case:
    def __init__(self, torch, g, P, tokens, k, experts, hidden, dtype, align=1, capacity=0, pad=0, start=0, seed=0):
        rng = np.random.default_rng([502, seed, P, tokens, k, experts, hidden])
        c = choices(rng, P, tokens, k, experts, twice=seed == 9)
        self.position, self.source, self.offsets = sorted_on_gpu(torch, g, c, experts, align, capacity, extra=9)
        self.rows, self.P, self.tokens, self.k, self.hidden = self.source.numel(), P, tokens, k, hidden
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed + hidden)

        def matrix(n):
            return torch.randn((n, hidden + pad + start), generator=gen, device="cuda").to(dtype)[:, start:start + hidden]

        self.x, self.add = ([matrix(tokens) for _ in range(P)] for _ in range(2))
        self.y = matrix(self.rows)
        self.weight = [torch.rand((tokens, k), generator=gen, device="cuda") + 0.1 for _ in range(P)]
        self.empty = lambda n: torch.full((n, hidden + pad + start), 7.0, device="cuda").to(dtype)
        self.view = lambda t: t[:, start:start + hidden]
        self.canary = lambda t: bool((t[:, :start] == 7).all()) and bool((t[:, start + hidden:] == 7).all())
        # pairs that have a row, their workers' tokens and rows
        self.at = torch.stack(self.position).reshape(-1).long()
        self.pairs = torch.nonzero(self.at >= 0)[:, 0]
        self.to = self.at[self.pairs]
        self.whole = lambda ts: torch.stack([t.double() for t in ts]).reshape(P * tokens, -1)


SHAPES = [  # P, tokens, k, experts, hidden, align, capacity, pad, start
    (1, 1, 1, 1, 1, 1, 0, 0, 0), (1, 16, 2, 8, 1024, 1, 0, 0, 0), (2, 33, 4, 6, 1001, 1, 0, 0, 0), (3, 50, 3, 7, 40, 128, 0, 0, 0),
    (1, 130, 8, 16, 2056, 1, 20, 8, 0), (2, 70, 5, 9, 257, 4, 0, 5, 3), (1, 40, 32, 40, 72, 1, 1, 0, 8), (1, 9, 2, 3, 4096, 16, 0, 0, 0),
    (4, 501, 4, 60, 100, 1, 40, 0, 0), (1, 20, 2, 4, 9000, 1, 0, 0, 0)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_gather(env, shape, weighted, dt):
    torch, g = env
    P, tokens, k, experts, hidden, align, capacity, pad, start = shape
    t = torch.float32 if dt == "f32" else torch.bfloat16
    c = Case(torch, g, P, tokens, k, experts, hidden, t, align, capacity, pad, start)
    y = c.empty(c.rows)
    g.gar_expert_gather(c.x, c.position, c.source, c.view(y), weight=c.weight if weighted else None)
    torch.cuda.synchronize()
    assert c.canary(y)
    want = torch.full((c.rows, hidden), 7.0, dtype=torch.float64, device="cuda")  # rows behind the last expert
    want[c.source == -1] = 0.0
    want[c.to] = c.whole(c.x)[c.pairs // k] * (c.whole(c.weight).reshape(-1)[c.pairs][:, None] if weighted else 1.0)
    tol = (half(torch, t) + (2 * U if dt == "bf16" else 0.0)) * want.abs() if weighted else torch.zeros_like(want)
    assert bool(((c.view(y).double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("weighted,added", [(False, "none"), (True, "none"), (True, "add"), (False, "place")])
@pytest.mark.parametrize("shape", SHAPES)
def test_combine(env, shape, weighted, added, dt):
    torch, g = env
    P, tokens, k, experts, hidden, align, capacity, pad, start = shape
    t = torch.float32 if dt == "f32" else torch.bfloat16
    c = Case(torch, g, P, tokens, k, experts, hidden, t, align, capacity, pad, start, seed=1)
    c.y[c.source < 0] = float("nan")  # rows without a pair are not read
    out = [c.empty(tokens) for _ in range(P)]
    if added == "place":
        for o, a in zip(out, c.add):
            c.view(o).copy_(a)
    views = [c.view(o) for o in out]
    g.gar_expert_combine(c.y, c.position, views, weight=c.weight if weighted else None,
                         addend=None if added == "none" else views if added == "place" else c.add)
    torch.cuda.synchronize()
    want = torch.zeros((P * tokens, hidden), dtype=torch.float64, device="cuda")
    terms = c.y[c.to].double() * (c.whole(c.weight).reshape(-1)[c.pairs][:, None] if weighted else 1.0)
    want.index_add_(0, c.pairs // k, terms)
    size = torch.zeros_like(want).index_add_(0, c.pairs // k, terms.abs())
    if added != "none":
        want += c.whole(c.add)
        size += c.whole(c.add).abs()
    got = c.whole(views)
    assert all(c.canary(o) for o in out)
    assert bool(((got - want).abs() <= (k + 2) * U * size + half(torch, t) * want.abs() * 1.01).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("place", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_combine_gradient(env, shape, place, dt):
    torch, g = env
    P, tokens, k, experts, hidden, align, capacity, pad, start = shape
    t = torch.float32 if dt == "f32" else torch.bfloat16
    c = Case(torch, g, P, tokens, k, experts, hidden, t, align, capacity, pad, start, seed=2)
    dy = c.empty(c.rows)
    y = c.y.clone()
    if place:
        c.view(dy).copy_(c.y)
        y = c.view(dy)
    behind = c.view(dy)[c.source == -2].clone()
    dweight = [torch.full((tokens, k), 7.0, device="cuda") for _ in range(P)]
    g.gar_expert_combine_grad(c.x, y, c.position, c.source, c.weight, c.view(dy), dweight)
    torch.cuda.synchronize()
    assert c.canary(dy) and torch.equal(c.view(dy)[c.source == -2], behind)
    dout = c.whole(c.x)[c.pairs // k]
    want = torch.zeros((c.rows, hidden), dtype=torch.float64, device="cuda")
    want[c.to] = dout * c.whole(c.weight).reshape(-1)[c.pairs][:, None]
    on = c.source >= -1
    assert bool(((c.view(dy).double() - want).abs() <= (half(torch, t) + 2 * U) * want.abs())[on].all())
    terms = dout * c.y[c.to].double()
    wd = torch.zeros(P * tokens * k, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(wd)
    wd[c.pairs], size[c.pairs] = terms.sum(1), terms.abs().sum(1)
    got = c.whole(dweight).reshape(-1)
    assert bool(((got - wd).abs() <= (hidden + 2) * U * size).all())
    assert bool((got[c.at < 0] == 0).all())


def test_combine_gradient_against_differences(env):
    """The combined rows are linear in y and in the weights: F = <dout, out> changes by exactly <dy, step> and <dweight,
    step>, up to the roundings of out (fp32)."""
    torch, g = env
    c = Case(torch, g, 2, 60, 3, 8, 96, torch.float32, seed=3)
    dy, dweight = torch.zeros_like(c.y), [torch.empty_like(w) for w in c.weight]
    g.gar_expert_combine_grad(c.x, c.y, c.position, c.source, c.weight, dy, dweight)

    def F(y, weight):
        out = [torch.empty_like(x) for x in c.x]
        g.gar_expert_combine(y, c.position, out, weight=weight)
        torch.cuda.synchronize()
        return sum((o.double() * x.double()).sum().item() for o, x in zip(out, c.x)), \
            sum((o.double() * x.double()).abs().sum().item() for o, x in zip(out, c.x))

    step = (torch.randint(-8, 9, c.y.shape, device="cuda") / 64.0)
    step[c.source < 0] = 0.0
    y1 = c.y + step
    a, s0 = F(c.y, c.weight)
    b, s1 = F(y1, c.weight)
    moved = ((y1.double() - c.y.double()) * dy.double()).sum().item()
    size = ((y1.double() - c.y.double()) * dy.double()).abs().sum().item()
    # an output's rounding is relative to its absolute sum, at most that of k terms of |y| |w|
    bound = sum((torch.stack([c.y.abs().amax() * w.sum(1)[:, None] * x.abs() for w, x in zip(c.weight, c.x)])).double().sum().item() for _ in (0,))
    assert abs((b - a) - moved) <= 12 * U * (2 * bound + s0 + s1) + 4 * U * size
    w1 = [w + 0.25 for w in c.weight]
    b, s1 = F(c.y, w1)
    moved = sum(((p.double() - w.double()) * d.double()).sum().item() for p, w, d in zip(w1, c.weight, dweight))
    size = sum(((p.double() - w.double()).abs() * d.double().abs()).sum().item() for p, w, d in zip(w1, c.weight, dweight))
    assert abs((b - a) - moved) <= 12 * U * (4 * bound + s0 + s1) + 100 * U * (size + bound)


def test_a_position_outside_the_rows_is_none(env):
    torch, g = env
    y = torch.ones((5, 16), device="cuda")
    position = [torch.tensor([[5, 2], [1 << 30, -7], [4, 0]], dtype=torch.int32, device="cuda")]
    source = torch.tensor([5, -1, 1, -2, 4], dtype=torch.int32, device="cuda")
    out = [torch.full((3, 16), 7.0, device="cuda")]
    g.gar_expert_combine(y, position, out)
    to = torch.full((5, 16), 7.0, device="cuda")
    g.gar_expert_gather(out, position, source, to)
    torch.cuda.synchronize()
    assert out[0][:, 0].tolist() == [1.0, 0.0, 2.0]
    assert to[:, 3].tolist() == [2.0, 0.0, 1.0, 7.0, 2.0]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gather_and_its_gradient_are_adjoint(env, dt):
    """<gather(x), d> = <x, combine(d)>, so the one is the gradient of the other."""
    torch, g = env
    t = torch.float32 if dt == "f32" else torch.bfloat16
    c = Case(torch, g, 2, 100, 3, 8, 64, t, align=8, seed=4)
    y = torch.zeros((c.rows, 64), dtype=t, device="cuda")
    g.gar_expert_gather(c.x, c.position, c.source, y)
    dx = [torch.empty_like(x) for x in c.x]
    g.gar_expert_combine(c.y, c.position, dx)
    torch.cuda.synchronize()
    a = (y.double() * c.y.double())
    b = torch.stack([(x.double() * d.double()) for x, d in zip(c.x, dx)])
    assert abs(a.sum().item() - b.sum().item()) <= (half(torch, t) + 4 * U) * (a.abs().sum().item() + b.abs().sum().item())


WEIGHTS = [(1, 1, 1, 1), (1, 300, 60, 4), (2, 77, 9, 9), (3, 65, 257, 8), (1, 40, 1024, 32), (8, 1000, 64, 2), (1, 33, 40, 17)]


def softmax_of_chosen(z, c, d):
    """weight, dz and what its error is measured in, by loops over tokens."""
    w, dz, size = np.zeros(c.shape), np.zeros(z.shape), np.zeros(z.shape)
    for t in range(c.shape[0]):
        on = np.nonzero((c[t] >= 0) & (c[t] < z.shape[1]))[0]
        q = z[t, c[t, on]]
        if not on.size or np.all(q == -np.inf):
            continue
        e = np.exp(q - q.max())
        w[t, on] = e / e.sum()
        mean = (w[t, on] * d[t, on]).sum()
        np.add.at(dz[t], c[t, on], w[t, on] * (d[t, on] - mean))
        np.add.at(size[t], c[t, on], w[t, on] * (np.abs(d[t, on]) + (w[t, on] * np.abs(d[t, on])).sum()))
    return w, dz, size


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("P,tokens,experts,k", WEIGHTS)
def test_weights(env, P, tokens, experts, k, accumulate, dt):
    torch, g = env
    t = torch.float32 if dt == "f32" else torch.bfloat16
    rng = np.random.default_rng([503, P, tokens, experts, k])
    c = choices(rng, P, tokens, k, experts, twice=experts == 9)
    pad = 3 if experts == 60 else 0
    z = [torch.from_numpy(rng.standard_normal((tokens, experts + pad)).astype(np.float32) * 4).cuda().to(t)[:, :experts] for _ in range(P)]
    if tokens > 5:
        z[0][4, :] = float("-inf")
        z[0][5, 0] = float("-inf")
    choice = [torch.from_numpy(a.copy()).cuda() for a in c]
    weight = [torch.full((tokens, k), 7.0, device="cuda") for _ in range(P)]
    d = [torch.from_numpy(rng.standard_normal((tokens, k)).astype(np.float32)).cuda() for _ in range(P)]
    for a, b in zip(d, choice):
        a[b < 0] = float("nan")  # not looked at
    before = [torch.from_numpy(rng.standard_normal((tokens, experts + pad)).astype(np.float32)).cuda().to(t) for _ in range(P)]
    dz = [(b.clone() if accumulate else torch.full_like(b, 7.0)) for b in before]
    g.gar_expert_weights(z, choice, weight)
    g.gar_expert_weights_grad(weight, d, choice, [a[:, :experts] for a in dz], accumulate=accumulate)
    torch.cuda.synchronize()
    for w in range(P):
        zh = z[w].double().cpu().numpy()
        want, want_dz, size = softmax_of_chosen(zh, c[w], d[w].double().cpu().numpy())
        got = weight[w].double().cpu().numpy()
        spread = np.where(np.isfinite(zh), np.abs(zh), 0.0).max(axis=1, keepdims=True) * 2
        rel = 2.0 ** -20 + 2 * k * U + 4 * U * spread
        assert np.all(np.abs(got - want) <= rel * want)
        if accumulate:
            want_dz = want_dz + before[w][:, :experts].double().cpu().numpy()
        tol = (2 * rel + (k + 6) * U) * size + half(torch, t) * np.abs(want_dz) * 1.01
        assert np.all(np.abs(dz[w][:, :experts].double().cpu().numpy() - want_dz) <= tol)
        edge = before[w][:, experts:] if accumulate else torch.full_like(before[w][:, experts:], 7.0)
        assert torch.equal(dz[w][:, experts:], edge)


def test_weights_gradient_against_differences(env):
    """F = sum d weight along a direction: |F'''| <= 6 |d| a^3 for logits changed by at most a."""
    torch, g = env
    rng = np.random.default_rng(504)
    c = choices(rng, 1, 50, 4, 12, none=0.0)
    z = torch.from_numpy(np.rint(rng.standard_normal((50, 12)) * 64).astype(np.float32) / 64).cuda()
    d = torch.from_numpy(rng.standard_normal((50, 4)).astype(np.float32)).cuda()
    choice = [torch.from_numpy(c[0].copy()).cuda()]
    d[choice[0] < 0] = 0.0
    d[choice[0] >= 12] = 0.0
    weight, dz = torch.empty((50, 4), device="cuda"), torch.empty((50, 12), device="cuda")
    g.gar_expert_weights([z], choice, [weight])
    g.gar_expert_weights_grad([weight], [d], choice, [dz])
    step = 2.0 ** -7
    way = torch.where(torch.rand(z.shape, device="cuda") < 0.5, -step, step)
    total = []
    for sign in (1, -1):
        w = torch.empty((50, 4), device="cuda")
        g.gar_expert_weights([z + sign * way], choice, [w])
        total.append((w.double() * d.double()).sum().item())
    along = (dz.double() * way.double()).sum().item()
    assert abs((total[0] - total[1]) / 2 - along) <= d.double().abs().sum().item() * (step ** 3 + 2.0 ** -18)


def test_a_nan_logit_stays_with_its_token(env):
    torch, g = env
    z = torch.zeros((3, 6), device="cuda")
    z[1, 2] = float("nan")
    choice = [torch.tensor([[0, 2], [2, 1], [5, 2]], dtype=torch.int32, device="cuda")]
    weight = [torch.empty((3, 2), device="cuda")]
    g.gar_expert_weights([z], choice, weight)
    torch.cuda.synchronize()
    assert weight[0][0].tolist() == [0.5, 0.5] and weight[0][2].tolist() == [0.5, 0.5] and bool(weight[0][1].isnan().all())


def test_rows_past_2_31_elements(env):
    torch, g = env
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    hidden, tokens = 1 << 16, 20000  # 40000 rows of 2^16: 2.6e9 elements
    x = torch.arange(tokens, device="cuda", dtype=torch.float32).remainder(251).bfloat16()[:, None].expand(tokens, hidden).contiguous()
    choice = torch.stack([torch.arange(tokens, device="cuda") % 2, 1 - torch.arange(tokens, device="cuda") % 2], 1).int().contiguous()
    position, source, offsets = sorted_on_gpu(torch, g, choice[None].cpu().numpy(), 2)
    y = torch.empty((source.numel(), hidden), dtype=torch.bfloat16, device="cuda")
    g.gar_expert_gather([x], position, source, y)
    torch.cuda.synchronize()
    assert torch.equal(y[:, 0], x[source.long() // 2, 0]) and torch.equal(y[:, -1], x[source.long() // 2, -1])
    out = torch.empty_like(x)
    g.gar_expert_combine(y, position, [out])
    torch.cuda.synchronize()
    assert torch.equal(out[:, ::4096], (2 * x[:, ::4096].float()).bfloat16())


def test_other_stream_and_captured_graph(env):
    """The chain from choices to gradients captured twice over one workspace, replayed, and on another stream."""
    torch, g = env
    c = Case(torch, g, 2, 3000, 4, 16, 64, torch.bfloat16, align=8, seed=6)
    rng = np.random.default_rng(7)
    choice = [torch.from_numpy(a.copy()).cuda() for a in choices(rng, 2, 3000, 4, 16)]
    ws = torch.empty(g.gar_expert_workspace_bytes(2, 3000, 4, 16), dtype=torch.uint8, device="cuda")

    def outputs():
        return ([torch.zeros_like(p) for p in c.position], torch.zeros_like(c.source), torch.zeros_like(c.offsets),
                torch.zeros((c.rows, 64), dtype=torch.bfloat16, device="cuda"), [torch.zeros_like(x) for x in c.x],
                torch.zeros((c.rows, 64), dtype=torch.bfloat16, device="cuda"), [torch.zeros_like(w) for w in c.weight])

    def chain(o, stream=None):
        g.gar_expert_sort(choice, 16, o[0], o[1], o[2], ws, align=8, stream=stream)
        g.gar_expert_gather(c.x, o[0], o[1], o[3], stream=stream)
        g.gar_expert_combine(o[3], o[0], o[4], weight=c.weight, addend=c.add, stream=stream)
        g.gar_expert_combine_grad(c.add, o[3], o[0], o[1], c.weight, o[5], o[6], stream=stream)

    def same(a, b):
        flat = lambda o: [t for x in o for t in (x if isinstance(x, list) else [x])]  # noqa: E731
        return all(torch.equal(p, q) for p, q in zip(flat(a), flat(b)))

    want, other = outputs(), outputs()
    torch.cuda.synchronize()
    chain(want)
    torch.cuda.synchronize()
    chain(other, torch.cuda.Stream())
    torch.cuda.synchronize()
    assert same(want, other)
    graphs = []
    for _ in range(2):
        o, graph = outputs(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain(o)
        graphs.append((graph, o))
    for graph, o in graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert all(same(want, o) for _, o in graphs)
    for a in choice:
        a.copy_(a.flip(0))
    want = outputs()
    chain(want)
    for graph, o in graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert all(same(want, o) for _, o in graphs)
