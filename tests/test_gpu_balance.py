"""Router choices, counts, balance loss and gradient against the plain 64-bit
form (worker_ref).  Choices and counts have to be equal.  A probability is
within about 2^-20 of itself, a centred count exact to fp32 and d_t a mean of
them: dz is within 2^-18 of coef p max |c - mean|, the loss within 2^-18."""
import numpy as np
import pytest

import worker_ref as ref
from helpers import need_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return need_cuda()


def logits(P, T, E, seed):
    g = np.random.default_rng([501, seed, P, T, E])
    return [(g.standard_normal((T, E)) + 0.5 * g.standard_normal((1, E))).astype(np.float32) for _ in range(P)]


def run(torch, g, zt, k, alpha, valid=None, place=False, grad=True, stream=None):
    P, (T, E) = len(zt), zt[0].shape
    choice = [torch.full((T, k), 99, dtype=torch.int32, device="cuda") for _ in range(P)]
    counts = torch.full((P, E), 99, dtype=torch.int32, device="cuda")
    loss = torch.full((1,), 99.0, device="cuda")
    dz = (zt if place else [torch.full_like(z, 99.0) for z in zt]) if grad else None
    ws = torch.full((g.gar_balance_workspace_bytes(P),), 0xAB, dtype=torch.uint8, device="cuda")
    g.gar_balance_loss(zt, k, alpha, choice, counts, loss, ws, dz=dz, valid=valid, stream=stream)
    torch.cuda.synchronize()
    return choice, counts, loss, dz


def check(torch, g, zt, k, alpha=0.01, valid=None, place=False):
    host = [z.float().cpu().numpy() for z in zt]
    vh = None if valid is None else [v.cpu().numpy() for v in valid]
    want = ref.balance(host, k, alpha, vh)
    choice, counts, loss, dz = run(torch, g, zt, k, alpha, valid, place)
    for w in range(len(zt)):
        np.testing.assert_array_equal(choice[w].cpu().numpy(), want[0][w])
    np.testing.assert_array_equal(counts.cpu().numpy(), np.stack(want[1]))
    assert abs(loss.item() - want[2]) <= 2.0 ** -18 * abs(want[2])
    for w in range(len(zt)):
        got, ref_dz, size = dz[w].float().cpu().numpy().astype(np.float64), want[3][w], want[4][w]
        tol = 2.0 ** -18 * size + 1e-40 + (2.0 ** -8 * np.abs(ref_dz) if dz[w].dtype == torch.bfloat16 else 0.0)
        assert (np.abs(got - ref_dz) <= tol).all(), np.abs(got - ref_dz).max()


def device(torch, zs, dtype):
    return [torch.from_numpy(z).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32) for z in zs]


SHAPES = [(1, 1, 1, 1), (1, 1, 4, 2), (2, 3, 8, 8), (1, 64, 8, 2), (1, 33, 9, 3), (3, 100, 31, 7), (4, 17, 33, 1), (2, 1000, 60, 4),
          (1, 300, 64, 32), (2, 257, 100, 8), (1, 200, 128, 2), (2, 150, 129, 8), (8, 40, 256, 8), (1, 600, 256, 32),
          (2, 100, 257, 3), (1, 90, 512, 8), (1, 70, 700, 32), (1, 50, 1024, 5), (64, 5, 16, 2)]


@pytest.mark.parametrize("P,T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shapes(env, P, T, E, k, dtype):
    torch, g = env
    check(torch, g, device(torch, logits(P, T, E, 1), dtype), k)


# enough tokens that each lane takes 32 logits, at every number of lanes
@pytest.mark.parametrize("P,T,E,k", [(1, 160000, 16, 3), (2, 42000, 31, 4), (1, 45000, 60, 6), (2, 11000, 128, 8),
                                     (1, 11000, 250, 8), (1, 10500, 256, 2), (2, 2600, 500, 9)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_tokens(env, P, T, E, k, dtype):
    torch, g = env
    zt = device(torch, logits(P, T, E, 2), dtype)
    choice, counts, loss, dz = run(torch, g, zt, k, 0.5)
    z = torch.stack([a.double() for a in zt])
    best = torch.sort(z, dim=2, descending=True, stable=True).indices[:, :, :k]
    assert all(torch.equal(c.long(), b) for c, b in zip(choice, best))
    want_counts = torch.stack([torch.bincount(b.flatten(), minlength=E) for b in best])
    assert torch.equal(counts.long(), want_counts)
    p, total, n = torch.softmax(z, 2), want_counts.sum(0).double(), P * T
    assert abs(loss.item() - 0.5 * E * (total * p.sum((0, 1))).sum().item() / (k * n * n)) <= 2.0 ** -18 * loss.item()
    coef = 0.5 * E / (k * n * n)
    want = coef * p * (total - (p * total).sum(2, keepdim=True))
    tol = 2.0 ** -18 * coef * p * (total - total.mean()).abs().max() + 1e-40
    for w in range(P):
        t = tol[w] + (2.0 ** -8 * want[w].abs() if dtype == "bf16" else 0.0)
        assert bool(((dz[w].double() - want[w]).abs() <= t).all())


@pytest.mark.parametrize("E,k", [(7, 3), (64, 4), (200, 8), (600, 8)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
def test_equal_masked_and_odd_logits(env, E, k, dtype, many):
    """Equal logits (all, and many), -inf, the type's lowest value, rows of nothing, NaN, padding tokens."""
    torch, g = env
    T = 40 if not many else 1 + 80 * 1024 * 32 // E
    z = np.tile(logits(1, 40, E, 3)[0], (-(-T // 40), 1))[:T]
    z[0] = 1.25
    z[1] = np.round(z[1])
    z[2] = -np.inf
    z[3, 1:] = -np.inf
    z[4, ::2] = -np.inf
    z[5] = np.finfo(np.float32).min if dtype == "f32" else -3.3895e38
    z[6] = np.where(np.arange(E) % 5 == 0, 2.0, -2.0)
    z[7, E - 1] = 80.0
    z[8, :] = 0.0
    z[8, 2] = -0.0
    z[9] = -np.inf
    zt = device(torch, [z], dtype)
    valid = [torch.ones(T, dtype=torch.uint8, device="cuda")]
    valid[0][11] = 0
    valid[0][0] = 255
    if not many:
        check(torch, g, zt, k, valid=valid)
        check(torch, g, zt, k)
    choice, counts, loss, dz = run(torch, g, zt, k, 0.01, [v.bool() for v in valid])
    want = ref.balance([zt[0][:40].float().cpu().numpy()], k, 0.01, [valid[0][:40].cpu().numpy()])
    np.testing.assert_array_equal(choice[0][:40].cpu().numpy(), want[0][0])
    assert torch.isfinite(dz[0]).all() and torch.isfinite(loss).all()
    assert (dz[0][2] == 0).all() and (dz[0][11] == 0).all() and (choice[0][11] == -1).all()


@pytest.mark.parametrize("E", [12, 100, 300])
def test_nan_is_not_chosen_and_stays_in_its_token(env, E):
    torch, g = env
    z = logits(1, 30, E, 4)[0]
    z[4, 3] = np.nan
    z[5, :] = np.nan
    zt = device(torch, [z], "f32")
    choice, counts, loss, dz = run(torch, g, zt, 3, 0.01)
    host = np.where(np.isnan(z), -np.inf, z)
    np.testing.assert_array_equal(choice[0].cpu().numpy(), ref.balance([host], 3, 0.01)[0][0])
    nan = torch.isnan(dz[0]).any(1).cpu().numpy()
    assert nan[4] and not nan[[i for i in range(30) if i not in (4, 5)]].any()
    assert torch.isnan(loss).all()


@pytest.mark.parametrize("E,k", [(20, 2), (60, 4), (256, 8)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_in_place_and_pointer_tables(env, E, k, dtype):
    torch, g = env
    zs = device(torch, logits(3, 77, E, 5), dtype)
    wide = [torch.zeros((77, E + 5), device="cuda", dtype=z.dtype) for z in zs]
    for w, z in zip(wide, zs):
        w[:, 3:3 + E] = z
    check(torch, g, [w[:, 3:3 + E] for w in wide], k)
    check(torch, g, [w[:, 3:3 + E] for w in wide], k, place=True)
    assert all((w[:, :3] == 0).all() and (w[:, 3 + E:] == 0).all() for w in wide)
    a = run(torch, g, zs, k, 0.01)
    ws = torch.empty(g.gar_balance_workspace_bytes(3), dtype=torch.uint8, device="cuda")
    choice, dz = [torch.empty_like(c) for c in a[0]], [torch.empty_like(z) for z in zs]
    counts, loss = torch.empty_like(a[1]), torch.empty_like(a[2])
    g.gar_balance_loss(g.pointer_table(zs), k, 0.01, g.pointer_table(choice), counts, loss, ws, dz=g.pointer_table(dz))
    assert torch.equal(counts, a[1]) and torch.equal(loss, a[2]) and all(torch.equal(x, y) for x, y in zip(dz, a[3]))


def test_no_tokens_and_no_gradient(env):
    torch, g = env
    zt = [torch.empty((0, 12), device="cuda") for _ in range(2)]
    choice, counts, loss, dz = run(torch, g, zt, 2, 0.01)
    assert (counts == 0).all() and loss.item() == 0.0
    zt = device(torch, logits(2, 50, 12, 6), "f32")
    valid = [torch.zeros(50, dtype=torch.uint8, device="cuda") for _ in range(2)]
    choice, counts, loss, dz = run(torch, g, zt, 2, 0.01, valid)
    assert (counts == 0).all() and loss.item() == 0.0 and all((d == 0).all() for d in dz) and all((c == -1).all() for c in choice)
    a, b = run(torch, g, zt, 2, 0.01, grad=False), run(torch, g, zt, 2, 0.01)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


def test_gradient_against_differences(env):
    """Central differences of the 64-bit loss; no choice changes over the step."""
    torch, g = env
    zs = logits(2, 40, 12, 7)
    zt = device(torch, zs, "f32")
    _, _, _, dz = run(torch, g, zt, 3, 1.0)
    base = ref.balance(zs, 3, 1.0)
    h = 1e-5
    rng = np.random.default_rng(8)
    for w, t, e in [(0, 0, 0), (1, 39, 11), (0, 17, 5)] + [(int(rng.integers(2)), int(rng.integers(40)), int(rng.integers(12))) for _ in range(5)]:
        out = []
        for s in (h, -h):
            moved = [z.astype(np.float64).copy() for z in zs]
            moved[w][t, e] += s
            got = ref.balance(moved, 3, 1.0)
            assert all((a == b).all() for a, b in zip(got[0], base[0]))
            out.append(got[2])
        diff = (out[0] - out[1]) / (2 * h)
        assert abs(diff - dz[w][t, e].item()) <= 1e-8 + 1e-4 * abs(diff)


def test_repeatable_streams_and_graphs(env):
    torch, g = env
    for P, T, E, k in ((1, 50, 8, 2), (4, 2000, 60, 4), (2, 30000, 64, 4)):
        zt = device(torch, logits(P, T, E, 9), "f32")
        a = run(torch, g, zt, k, 0.01)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        b = run(torch, g, zt, k, 0.01, stream=side)
        choice = [torch.empty_like(c) for c in a[0]]
        counts, loss, dz = torch.empty_like(a[1]), torch.empty_like(a[2]), [torch.empty_like(z) for z in zt]
        ws = torch.empty(g.gar_balance_workspace_bytes(P), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.gar_balance_loss(zt, k, 0.01, choice, counts, loss, ws, dz=dz)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        for c in (b, (choice, counts, loss, dz)):
            assert all(torch.equal(x, y) for x, y in zip(a[0], c[0])) and torch.equal(a[1], c[1])
            assert torch.equal(a[2], c[2]) and all(torch.equal(x, y) for x, y in zip(a[3], c[3]))


def test_back_to_back_calls_on_one_workspace(env):
    """Calls of different sizes in a row: the counts of one are not seen by the next."""
    torch, g = env
    ws = torch.empty(g.gar_balance_workspace_bytes(1), dtype=torch.uint8, device="cuda")
    sets = [device(torch, logits(1, T, E, 10), "f32") for T, E in ((3000, 64), (5000, 32), (3000, 64))]
    outs = []
    for zt in sets * 3:
        T, E = zt[0].shape
        o = ([torch.empty((T, 2), dtype=torch.int32, device="cuda")], torch.empty((1, E), dtype=torch.int32, device="cuda"),
             torch.empty(1, device="cuda"))
        g.gar_balance_loss(zt, 2, 0.01, *o, ws)
        outs.append(o)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        T, E = sets[i % 3][0].shape
        assert o[1].sum().item() == 2 * T
        assert torch.equal(o[1], outs[i % 3][1]) and torch.equal(o[2], outs[i % 3][2])


# rows that start on 2, 4, 8 and 16 bytes (of z and of dz apart), their neighbours untouched; few tokens and many
@pytest.mark.parametrize("E,T", [(13, 90), (60, 700), (60, 45000), (131, 300), (131, 22000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_at_every_alignment(env, E, T, dtype):
    torch, g = env
    zs = device(torch, logits(1, T, E, 9), dtype)
    base, k = None, 3
    for lead, pad, dlead, dpad in ((0, 0, 0, 0), (0, 1, 1, 0), (2, 2, 0, 4), (4, 4, 2, 2), (8, 8, 8, 8), (1, 8, 8, 1)):
        ld, dld = (E + 7) // 8 * 8 + pad + 8, (E + 7) // 8 * 8 + dpad + 8
        z = torch.zeros((T, ld), device="cuda", dtype=zs[0].dtype)
        z[:, lead:lead + E] = zs[0]
        dz = torch.full((T, dld), 5.0, device="cuda", dtype=z.dtype)
        choice = torch.full((T, k), 99, dtype=torch.int32, device="cuda")
        counts, loss = torch.zeros((1, E), dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda")
        ws = torch.zeros(g.gar_balance_workspace_bytes(1), dtype=torch.uint8, device="cuda")
        g.gar_balance_loss([z[:, lead:lead + E]], k, 0.5, [choice], counts, loss, ws, dz=[dz[:, dlead:dlead + E]])
        torch.cuda.synchronize()
        got = choice, counts, dz[:, dlead:dlead + E].contiguous()
        if base is None:
            base = got
            if T <= 700:
                check(torch, g, zs, k)
        for a, b in zip(got, base):  # the same values, whatever the pieces they were read in
            assert torch.equal(a, b)
        assert (dz[:, :dlead] == 5.0).all() and (dz[:, dlead + E:] == 5.0).all()


# the calls' one, two and three launches; in place (as a step that keeps one buffer of logits) and not
@pytest.mark.parametrize("P,T,E", [(2, 300, 12), (2, 3000, 60), (1, 41000, 64), (2, 12000, 128), (1, 9000, 300)])
@pytest.mark.parametrize("place", [False, True])
def test_logits_rewritten_before_each_call(env, P, T, E, place):
    """One buffer of logits, rewritten by the 8-bit product directly before each of a hundred calls without a wait of the
    host: every call sees the new ones, as calls with the host waiting in between do."""
    torch, g = env
    gen = torch.Generator(device="cuda").manual_seed(77)
    H, n, k = 128, 4, 4

    def codes(rows):
        q, s = g.fp8_matrix(rows, H)
        g.gar_fp8_quantize(torch.randn((rows, H), generator=gen, device="cuda"), q, s)
        return q, s

    router, xs = codes(E), [[codes(T) for _ in range(P)] for _ in range(n)]
    z = [torch.empty((T, E), device="cuda") for _ in range(P)]
    ws = torch.empty(g.gar_balance_workspace_bytes(P), dtype=torch.uint8, device="cuda")

    def outputs():
        return ([torch.empty((T, k), dtype=torch.int32, device="cuda") for _ in range(P)],
                torch.empty((P, E), dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda"),
                z if place else [torch.empty_like(a) for a in z])

    def step(i, out, wait):
        for w in range(P):
            g.gar_fp8_matmul(*xs[i][w], *router, z[w])
        if wait:
            torch.cuda.synchronize()
        g.gar_balance_loss(z, k, 0.5, *out[:3], ws, dz=out[3])

    want = []
    for i in range(n):
        out = outputs()
        step(i, out, True)
        torch.cuda.synchronize()
        want.append([t.clone() for part in out for t in (part if isinstance(part, list) else [part])])
    outs = [outputs() for _ in range(n)]
    for _ in range(100 // n):
        for i in range(n):
            step(i, outs[i], False)
            if place:
                outs[i] = outs[i][:3] + ([a.clone() for a in z],)  # its gradient, before the next product takes the buffer
        torch.cuda.synchronize()
        for i in range(n):
            got = [t for part in outs[i] for t in (part if isinstance(part, list) else [part])]
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
            outs[i] = outs[i][:3] + (z if place else outs[i][3],)
