"""Global gradient norm and clipping against sums in 64 bits.

Tolerances: four squares added by fma and two pairwise sums round in fp32 (6 2^-24 of
the sum of squares, half of that in the norm), the norm once more: 4 2^-24.  A clipped value is
the product with c = max_norm / norm (one quotient, the norm's error) and one rounding
to its type."""
import math

import numpy as np
import pytest

from helpers import need_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    return need_cuda()


def make(torch, sizes, P, dtypes, seed=0, scale=0.01, start=0, gap=0):
    """P lists of tensors, views into one buffer per worker and type: `start` elements in, `gap` apart."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    out = []
    for _ in range(P):
        flat = {d: torch.randn((start + sum(n + gap for n, t in zip(sizes, dtypes) if t == d) + 8,), generator=gen, device="cuda").mul(scale).to(d)
                for d in set(dtypes)}
        at = {d: start for d in flat}
        row = []
        for n, d in zip(sizes, dtypes):
            row.append(flat[d][at[d]:at[d] + n])
            at[d] += n + gap
        out.append(row)
    return out


def norms(grads):
    return [math.sqrt(sum((t.double() ** 2).sum().item() for t in row)) for row in grads]


def space(torch, g, tables):
    return torch.full((g.gar_grad_workspace_bytes(tables),), 255, dtype=torch.uint8, device="cuda")


def check(torch, g, grads, max_norm, shared=False, place=False, out=None, stream=None):
    P = len(grads)
    before = [[t.clone() for t in row] for row in grads]
    want = norms(grads)[:1 if shared else P]
    out = grads if place else out or [[torch.full_like(t, 7.0) for t in row] for row in grads]
    tables = g.grad_tables(grads, None if place else out)
    norm = torch.full((len(want),), 7.0, device="cuda")
    ws = space(torch, g, tables)
    torch.cuda.synchronize()
    g.gar_grad_clip(tables, max_norm, norm, ws, shared=shared, stream=stream)
    torch.cuda.synchronize()
    for a, b in zip(norm.tolist(), want):
        assert abs(a - b) <= 4 * U * b, (a, b)
    for w in range(P):
        n = want[0 if shared else w]
        c = max_norm / n if n > max_norm else 1.0
        for a, b in zip(out[w], before[w]):
            if c == 1.0:
                assert torch.equal(a, b)
                continue
            ref = b.double() * c
            assert bool(((a.double() - ref).abs() <= (torch.finfo(a.dtype).eps / 2 * 1.01 + 7 * U) * ref.abs() + 1e-44).all())
            if not place:
                assert torch.equal(grads[w][0], before[w][0])
    assert g.gar_sync_status() == 0
    return norm, out


SIZES = [[1], [0, 5, 0], [3, 1, 2, 7, 4], [8191, 8192, 8193], [1, 100000, 17, 65536, 0, 300007], [16384 * 3 + 5], [37] * 100, [1000] * 700]


@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("P,shared", [(1, False), (3, False), (3, True)])
@pytest.mark.parametrize("sizes", range(len(SIZES)))
def test_against_64_bits(env, sizes, P, shared, kind):
    torch, g = env
    sizes = SIZES[sizes]
    types = [torch.bfloat16 if kind == "bf16" or (kind == "mixed" and i % 3) else torch.float32 for i in range(len(sizes))]
    grads = make(torch, sizes, P, types, seed=len(sizes), start=sum(sizes) % 5, gap=len(sizes) % 2)
    top = max(norms(grads))
    check(torch, g, grads, 0.3 * top, shared)
    check(torch, g, grads, 2.0 * top, shared)
    check(torch, g, grads, 0.3 * top, shared, place=True)


def test_many_workers(env):
    torch, g = env
    grads = make(torch, [100, 9, 4000] * 10, 64, [torch.float32] * 30)
    check(torch, g, grads, 0.1)
    check(torch, g, grads, 0.1, shared=True, place=True)


def test_outputs_that_start_elsewhere(env):
    """Inputs and outputs without a 16-byte line in common, and canaries around the outputs."""
    torch, g = env
    sizes = [5, 8200, 33, 40000]
    for d in (torch.float32, torch.bfloat16):
        grads = make(torch, sizes, 2, [d] * 4, start=1, gap=3)
        flat = [torch.full((sum(sizes) + 40,), 7.0, device="cuda").to(d) for _ in range(2)]
        at = np.cumsum([0] + [n + 4 for n in sizes]) + 3 - 1
        out = [[f[int(a):int(a) + n] for a, n in zip(at, sizes)] for f in flat]
        check(torch, g, grads, 0.5, out=out)
        for f in flat:
            for a, n in zip(at, sizes):
                f[int(a):int(a) + n] = 7.0
            assert bool((f == 7).all())


def test_norm_alone_and_long_lists(env):
    torch, g = env
    grads = make(torch, [50 + i for i in range(900)], 2, [torch.float32, torch.bfloat16] * 450)
    tables = g.grad_tables(grads)
    norm = torch.full((2,), 7.0, device="cuda")
    g.gar_grad_norm(tables, norm, space(torch, g, tables))
    torch.cuda.synchronize()
    for a, b in zip(norm.tolist(), norms(grads)):
        assert abs(a - b) <= 4 * U * b
    check(torch, g, grads, 0.4 * norms(grads)[0])


@pytest.mark.parametrize("scale", [1e25, 3e37, 1e-25, 1e-38])
def test_no_square_overflows_or_vanishes(env, scale):
    torch, g = env
    grads = make(torch, [70, 3], 1, [torch.float32] * 2)
    for t in grads[0]:
        t.copy_(torch.randn(t.shape, device="cuda").clamp(-2, 2) * scale)
    check(torch, g, grads, 0.25 * norms(grads)[0])


def test_zeros_and_no_tensors(env):
    torch, g = env
    grads = [[torch.zeros(5000, device="cuda"), torch.zeros(3, device="cuda")]]
    norm, out = check(torch, g, grads, 1.0)
    check(torch, g, grads, 0.0)
    assert norm.item() == 0.0
    empty = [[torch.zeros(0, device="cuda")]]
    tables, norm = g.grad_tables(empty), torch.full((1,), 7.0, device="cuda")
    g.gar_grad_clip(tables, 1.0, norm, space(torch, g, tables))
    torch.cuda.synchronize()
    assert norm.item() == 0.0
    tables, norm = g.grad_tables([[], []]), torch.full((2,), 7.0, device="cuda")
    g.gar_grad_clip(tables, 1.0, norm, space(torch, g, tables))
    torch.cuda.synchronize()
    assert norm.tolist() == [0.0, 0.0]


def test_max_norm_zero_and_infinite(env):
    torch, g = env
    grads = make(torch, [1000, 70], 1, [torch.float32, torch.bfloat16])
    check(torch, g, grads, math.inf)
    _, out = check(torch, g, grads, 0.0)
    assert all(bool((t == 0).all()) for t in out[0])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("place", [False, True])
def test_a_norm_that_is_not_finite(env, bad, place):
    """Only the worker whose gradients hold it keeps them; the others are clipped."""
    torch, g = env
    grads = make(torch, [3000, 21], 3, [torch.float32, torch.bfloat16])
    want = norms(grads)
    grads[1][1][20] = bad
    before = [[t.clone() for t in row] for row in grads]
    out = grads if place else [[torch.zeros_like(t) for t in row] for row in grads]
    tables, norm = g.grad_tables(grads, None if place else out), torch.empty(3, device="cuda")
    g.gar_grad_clip(tables, 0.1, norm, space(torch, g, tables))
    assert g.gar_sync_status() == g.GAR_STATUS_NONFINITE
    assert g.gar_sync_status() == 0
    n = norm.tolist()
    assert (math.isnan(n[1]) if math.isnan(bad) else n[1] == math.inf) and abs(n[2] - want[2]) <= 4 * U * want[2]
    same = lambda a, b: bool(((a == b) | (a.isnan() & b.isnan())).all())  # noqa: E731
    assert all(same(a, b) for a, b in zip(out[1], before[1]))
    assert not same(out[0][0], before[0][0])


def test_the_same_bits_in_every_run_streams_and_graphs(env):
    torch, g = env
    grads = make(torch, [100003, 5, 70000], 2, [torch.float32, torch.bfloat16, torch.float32])
    first = check(torch, g, grads, 0.5)
    again = check(torch, g, grads, 0.5, stream=torch.cuda.Stream())
    assert torch.equal(first[0], again[0]) and all(torch.equal(a, b) for p, q in zip(first[1], again[1]) for a, b in zip(p, q))
    out = [[torch.zeros_like(t) for t in row] for row in grads]
    tables, norm = g.grad_tables(grads, out), torch.zeros(2, device="cuda")
    ws = space(torch, g, tables)
    graphs = []
    for _ in range(2):  # two graphs over one workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.gar_grad_clip(tables, 0.5, norm, ws)
        graphs.append(graph)
    for graph in graphs:
        norm.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, first[0]) and all(torch.equal(a, b) for p, q in zip(first[1], out) for a, b in zip(p, q))
    for row in grads:
        for t in row:
            t.mul_(2.0)
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, 2 * first[0])


def test_more_than_2_31_elements(env):
    torch, g = env
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")
    n = (1 << 31) + 70001
    t = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    t[-1] = 8.0
    tables, norm = g.grad_tables([[t]]), torch.zeros(1, device="cuda")
    want = math.sqrt((n - 1) * 2.0 ** -20 + 64)
    g.gar_grad_clip(tables, want / 2, norm, space(torch, g, tables))
    torch.cuda.synchronize()
    assert abs(norm.item() - want) <= 4 * U * want
    assert t[-1].item() == 4.0 and t[0].item() == 2.0 ** -11 and bool((t[1 << 31:-1] == 2.0 ** -11).all())
