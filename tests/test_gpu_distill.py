"""Distillation loss and gradient against the plain 64-bit form (worker_ref).

Tolerances.  A power 2^x is within 2^-21 of itself relative, and its exponent,
formed in fp32, within 2^-22 of the exponent's size: a probability q is within
(2^-20 + 2^-21 |log q|) q.  The loss and the log-sum-exp add the rounding of
the logits' products with 1 / tau.  bf16 gradients are rounded once."""
import numpy as np
import pytest

import worker_ref as ref
from helpers import need_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return need_cuda()


def problem(rows, vocab, k, seed, repeat=False):
    g = np.random.default_rng([401, seed, rows, vocab, k])
    z = (g.standard_normal((rows, vocab)) * 3.0).astype(np.float32)
    if repeat:
        index = g.integers(0, max(1, vocab // 3), (rows, k)).astype(np.int32)
    else:
        index = np.stack([g.permutation(vocab)[:k] if vocab <= 4096 else (g.integers(0, vocab) + np.arange(k) * (vocab // k)) % vocab
                          for _ in range(rows)]).astype(np.int32)
    teacher = (g.standard_normal((rows, k)) * 2.0 + 5.0).astype(np.float32)
    weight = (g.random(rows) + 0.5).astype(np.float32)
    return z, index, teacher, weight


def close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    bad = np.isnan(got) != np.isnan(want)
    fine = np.isfinite(want)
    bad |= ~fine & ~np.isnan(want) & (got != want)
    with np.errstate(invalid="ignore"):
        bad |= fine & ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


def check(torch, g, z, index, teacher, weight, tau, mode, stream=None):
    """z: a CUDA tensor.  mode: fused, split or place (fused, dz over z)."""
    rows, vocab = z.shape
    host = z.float().cpu().numpy()
    want_loss, want_lse, want_dz, q, p = ref.distill(host, index, teacher, tau, np.ones(rows) if weight is None else weight)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    i, t, w = to(index), to(teacher), None if weight is None else to(weight)
    loss, lse = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    dz = z if mode == "place" else torch.full_like(z, 7.0)
    if mode == "split":
        g.gar_distill_loss(z, i, t, tau, loss, lse, weight=w, stream=stream)
        g.gar_distill_grad(z, i, t, tau, lse, dz, weight=w, stream=stream)
    else:
        g.gar_distill_loss(z, i, t, tau, loss, lse, dz=dz, weight=w, stream=stream)
    torch.cuda.synchronize()
    finite = np.where(np.isfinite(host), np.abs(host), 0.0)
    size = finite.max(axis=1) / tau
    with np.errstate(invalid="ignore"):
        close(lse.cpu().numpy(), want_lse, 2.0 ** -20 * (4 + size), "lse")
        close(loss.cpu().numpy(), want_loss, 2.0 ** -19 * (8 + size + np.abs(teacher).max(initial=0, where=np.isfinite(teacher)) / tau), "loss")
        scale = np.abs(np.ones(rows) if weight is None else weight)[:, None] / tau
        rel = 2.0 ** -20 + 2.0 ** -21 * np.where(q > 0, np.abs(np.log(np.where(q > 0, q, 1.0))), 0.0)
        if mode == "split":  # the exponent starts from the saved lse, itself an fp32 number
            rel = rel + 2.0 ** -22 * (np.abs(np.where(np.isfinite(want_lse), want_lse, 0.0)) + size)[:, None]
        mass = np.zeros_like(host, dtype=np.float64)
        for r in range(rows):
            on = (index[r] >= 0) & (index[r] < vocab)
            np.add.at(mass[r], index[r][on], p[r, on])
        tol = scale * (rel * q + 2.0 ** -19 * mass) + 1e-37
        if z.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(want_dz)
        close(dz.float().cpu().numpy(), want_dz, tol, "dz")
    assert g.gar_sync_status() == 0


def device(torch, z, dtype):
    t = torch.from_numpy(z).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


# from single tokens of a tiny vocabulary to rows of several CTAs (the split at 16 KB a row, at 101 KB a CTA)
SHAPES = [(1, 1, 1), (1, 7, 7), (3, 100, 5), (40, 1000, 33), (9, 4095, 64), (5, 4096, 16), (4, 4097, 100), (3, 8191, 1),
          (2, 8193, 128), (400, 8200, 4), (2, 32000, 300), (200, 33333, 20), (3, 50257, 50), (170, 53001, 7),
          (80, 70001, 9), (2, 131072, 64), (40, 131073, 1024), (3, 262144, 32)]


@pytest.mark.parametrize("rows,vocab,k", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mode", ["fused", "split"])
def test_shapes(env, rows, vocab, k, dtype, mode):
    torch, g = env
    z, index, teacher, weight = problem(rows, vocab, k, 1)
    check(torch, g, device(torch, z, dtype), index, teacher, weight, 1.7, mode)


@pytest.mark.parametrize("rows,vocab,k", [(6, 300, 8), (5, 9001, 40), (200, 40000, 8), (100, 90001, 12)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_over_the_logits(env, rows, vocab, k, dtype):
    torch, g = env
    z, index, teacher, weight = problem(rows, vocab, k, 2)
    check(torch, g, device(torch, z, dtype), index, teacher, weight, 0.8, "place")


@pytest.mark.parametrize("vocab", [301, 20001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mode", ["fused", "split"])
def test_rows_at_every_alignment(env, vocab, dtype, mode):
    """z and dz as column ranges of wider matrices, at equal and at different offsets."""
    torch, g = env
    z, index, teacher, weight = problem(9, vocab, 12, 3)
    wide = torch.zeros((9, vocab + 13), device="cuda", dtype=torch.float32 if dtype == "f32" else torch.bfloat16)
    i, t, w = (torch.from_numpy(a).cuda() for a in (index, teacher, weight))
    for off, off2 in ((0, 0), (1, 1), (3, 3), (2, 5), (0, 1)):
        x = wide[:, off:off + vocab]
        x.copy_(device(torch, z, dtype))
        big = torch.full((9, vocab + 9), 5.0, device="cuda", dtype=wide.dtype)
        dz = big[:, off2:off2 + vocab]
        loss, lse = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
        if mode == "split":
            g.gar_distill_loss(x, i, t, 1.1, loss, lse, weight=w)
            g.gar_distill_grad(x, i, t, 1.1, lse, dz, weight=w)
        else:
            g.gar_distill_loss(x, i, t, 1.1, loss, lse, dz=dz, weight=w)
        alone = torch.empty((9, vocab), device="cuda", dtype=wide.dtype)
        loss2, lse2 = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
        g.gar_distill_loss(x.contiguous(), i, t, 1.1, loss2, lse2, dz=alone, weight=w)
        torch.cuda.synchronize()
        tol = 2.0 ** -7 if dtype == "bf16" else 2e-5
        assert torch.allclose(dz.float(), alone.float(), rtol=tol, atol=1e-6)
        assert torch.allclose(loss, loss2, rtol=1e-5, atol=1e-5)
        edge = big.clone()
        edge[:, off2:off2 + vocab] = 5.0
        assert (edge == 5.0).all()


@pytest.mark.parametrize("vocab", [200, 9000, 60001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mode", ["fused", "split"])
def test_repeated_absent_and_empty_entries(env, vocab, dtype, mode):
    torch, g = env
    z, index, teacher, weight = problem(8, vocab, 70, 4, repeat=True)
    index[1, :] = 5                      # one token, many times
    index[2, ::2] = -1                   # absent entries
    index[2, 1::4] = vocab + 3
    index[3, :] = -7                     # none
    teacher[4, 3:] = -np.inf             # cut by the teacher
    teacher[5, :] = -np.inf              # all of them
    weight[6] = 0.0
    z[6] = np.nan                        # a row without weight: whatever it holds
    z[3] = np.inf
    weight[7] = -0.5
    check(torch, g, device(torch, z, dtype), index, teacher, weight, 1.0, mode)


@pytest.mark.parametrize("vocab", [130, 9000, 70000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mode", ["fused", "split"])
def test_masked_student_logits(env, vocab, dtype, mode):
    """-inf at other tokens, at the teacher's, everywhere; the type's lowest value everywhere (tau of 1 and more, so
    that z / tau stays finite); NaN in one row only."""
    torch, g = env
    z, index, teacher, weight = problem(7, vocab, 6, 5)
    z[0, vocab // 2:] = -np.inf
    index[0] = np.arange(6)
    z[1, index[1, 2]] = -np.inf
    z[2] = -np.inf
    z[3] = -3.3895e38 if dtype == "bf16" else np.finfo(np.float32).min
    z[4, vocab // 3] = np.nan
    z[5, :-1] = -np.inf
    zt = device(torch, z, dtype)
    rows = [0, 1, 2, 3, 5, 6]
    rows = rows if mode == "fused" else [0, 1, 2, 5, 6]  # an lse of -3.4e38 leaves no room for log of the sum
    check(torch, g, zt[rows].contiguous(), index[rows], teacher[rows], weight[rows], 1.0 if mode == "split" else 2.0, mode)
    i, t, w = (torch.from_numpy(a).cuda() for a in (index, teacher, weight))
    loss, lse, dz = torch.empty(7, device="cuda"), torch.empty(7, device="cuda"), torch.empty_like(zt)
    g.gar_distill_loss(zt, i, t, 2.0, loss, lse, dz=dz, weight=w)
    assert torch.isnan(loss).tolist() == [False] * 4 + [True] + [False] * 2
    assert torch.isnan(dz).any(1).tolist() == [False] * 4 + [True] + [False] * 2


def test_large_logits_and_temperatures(env):
    torch, g = env
    z, index, teacher, weight = problem(6, 12000, 10, 6)
    for scale, tau in ((1000.0, 1.0), (1.0, 0.01), (1e-3, 50.0), (1e30, 1e30)):
        zt = device(torch, z * np.float32(scale), "f32")
        check(torch, g, zt, index, (teacher * np.float32(min(scale, 10.0))).astype(np.float32), weight, tau, "fused")


@pytest.mark.parametrize("vocab", [100, 9000, 120000])
@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_teacher_logits_masked_by_lowest_values(env, vocab, tau):
    """The lowest fp32, large negative numbers, and a row that has nothing else."""
    torch, g = env
    z, index, teacher, weight = problem(5, vocab, 9, 11)
    teacher[0, 4:] = np.finfo(np.float32).min
    teacher[1, 1:] = -1e30
    teacher[2, :] = np.finfo(np.float32).min
    teacher[3, :3] = 3e38
    teacher[3, 3:6] = np.finfo(np.float32).min
    host = z.astype(np.float64)
    loss, lse = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    dz = torch.empty((5, vocab), device="cuda")
    g.gar_distill_loss(*(torch.from_numpy(a).cuda() for a in (z, index, teacher)), tau, loss, lse, dz=dz,
                       weight=torch.from_numpy(weight).cuda())
    want = ref.distill(host, index, teacher, tau, weight)
    close(loss.cpu().numpy(), want[0], 2.0 ** -19 * (8 + 2 * np.abs(z).max() / tau + 16 / tau), "loss")
    close(dz.cpu().numpy(), want[2], 2.0 ** -18 * weight[:, None] / tau * (want[3] * 40 + 1e-3 * (want[2] < 0) + np.abs(want[2])), "dz")


def test_loss_only_equals_fused_and_no_weights(env):
    torch, g = env
    for vocab in (500, 30000, 120000):
        z, index, teacher, _ = problem(20, vocab, 9, 7)
        check(torch, g, device(torch, z, "bf16"), index, teacher, None, 1.0, "fused")
        zt, i, t = device(torch, z, "bf16"), torch.from_numpy(index).cuda(), torch.from_numpy(teacher).cuda()
        a, b = (torch.empty((2, 20), device="cuda") for _ in range(2))
        g.gar_distill_loss(zt, i, t, 1.0, a[0], a[1])
        g.gar_distill_loss(zt, i, t, 1.0, b[0], b[1], dz=torch.empty_like(zt))
        assert torch.equal(a, b)


@pytest.mark.parametrize("vocab", [37, 10001])
def test_gradient_against_differences(env, vocab):
    """Central differences of the 64-bit loss along single logits and along a random direction."""
    torch, g = env
    z, index, teacher, weight = problem(3, vocab, 5, 8)
    tau = 1.3
    zt = device(torch, z, "f32")
    loss, lse, dz = torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), torch.empty_like(zt)
    g.gar_distill_loss(zt, *(torch.from_numpy(a).cuda() for a in (index, teacher)), tau, loss, lse, dz=dz,
                       weight=torch.from_numpy(weight).cuda())
    got = dz.cpu().numpy().astype(np.float64)
    h = 1e-4

    def total(x):
        return float((ref.distill(x, index, teacher, tau, weight)[0] * weight).sum())

    rng = np.random.default_rng(9)
    spots = [(0, index[0, 0]), (1, index[1, 4]), (2, 0), (0, vocab - 1)]
    directions = [rng.standard_normal(z.shape)]
    for r, v in spots:
        e = np.zeros(z.shape)
        e[r, v] = 1.0
        directions.append(e)
    for e in directions:
        diff = (total(z + h * e) - total(z - h * e)) / (2 * h)
        # h^2 / 6 times a third derivative below 1, and the losses' own rounding over 2 h
        assert abs(diff - (got * e).sum()) <= 1e-6 * (1 + np.abs(e).sum() / vocab) + 1e-5 * abs(diff)


def test_streams_and_graphs(env):
    torch, g = env
    for rows, vocab in ((50, 900), (300, 20000), (20, 110000)):
        z, index, teacher, weight = problem(rows, vocab, 11, 10)
        zt = device(torch, z, "bf16")
        i, t, w = (torch.from_numpy(a).cuda() for a in (index, teacher, weight))
        outs = [(torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda"), torch.zeros_like(zt)) for _ in range(3)]

        def call(o, stream=None):
            g.gar_distill_loss(zt, i, t, 1.0, o[0], o[1], dz=o[2], weight=w, stream=stream)

        call(outs[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        call(outs[1], side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(outs[2])
        graph.replay()
        torch.cuda.synchronize()
        for o in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(outs[0], o))


def test_offsets_beyond_32_bits(env):
    torch, g = env
    rows, vocab = 70000, 32768
    z = torch.randn((rows, vocab), device="cuda", dtype=torch.bfloat16)
    index = torch.randint(0, vocab, (rows, 3), device="cuda", dtype=torch.int32)
    teacher = torch.randn((rows, 3), device="cuda")
    tail = slice(rows - 5, rows)
    host, ih, th = z[tail].float().cpu().numpy(), index[tail].cpu().numpy(), teacher[tail].cpu().numpy()
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    g.gar_distill_loss(z, index, teacher, 1.0, loss, lse, dz=z)
    want = ref.distill(host, ih, th, 1.0, np.ones(5))
    close(loss[tail].cpu().numpy(), want[0], 1e-4, "loss")
    close(z[tail].float().cpu().numpy(), want[2], 2.0 ** -8 * np.abs(want[2]) + 1e-9, "dz")


# rows that fill two stages of eight CTAs, and rows that no eight CTAs hold
@pytest.mark.parametrize("vocab", [151937, 230003, 460001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mode", ["fused", "split", "place"])
def test_very_long_rows(env, vocab, dtype, mode):
    torch, g = env
    z, index, teacher, weight = problem(5, vocab, 37, 12, repeat=True)
    index[1, :] = vocab - 1
    index[2, ::3] = vocab
    weight[3] = 0.0
    z[3] = np.inf
    z[4, : vocab // 2] = -np.inf
    check(torch, g, device(torch, z, dtype), index, teacher, weight, 1.3, mode)


# short rows: each number of vectors a thread holds, one element to each side of it
@pytest.mark.parametrize("vocab", [511, 512, 513, 1023, 1025, 2047, 2049, 4095, 4103, 8185, 8199])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mode", ["fused", "split", "place"])
def test_short_rows_at_every_length(env, vocab, dtype, mode):
    torch, g = env
    z, index, teacher, weight = problem(17, vocab, 19, 13, repeat=True)
    index[1, :] = 0
    index[2, :] = vocab - 1
    check(torch, g, device(torch, z, dtype), index, teacher, weight, 0.9, mode)


# the loss alone takes a row's parts as the call with the gradient does, wherever they run
@pytest.mark.parametrize("rows,vocab,k", [(3, 50001, 9), (400, 50001, 40), (400, 36001, 300), (330, 131072, 64), (170, 151937, 200),
                                          (160, 33000, 1024), (200, 8200, 5)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_loss_alone_is_the_same_bit_for_bit(env, rows, vocab, k, dtype):
    torch, g = env
    gen = torch.Generator(device="cuda").manual_seed(rows + vocab)
    z = (torch.randn((rows, vocab), generator=gen, device="cuda") * 3).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    z[1, : vocab // 2] = float("-inf")
    z[2, 7] = float("inf")
    index = torch.randint(-2, vocab + 2, (rows, k), generator=gen, device="cuda", dtype=torch.int32)
    teacher = torch.randn((rows, k), generator=gen, device="cuda")
    weight = (torch.rand(rows, generator=gen, device="cuda") > 0.1).float()
    got = []
    for dz in (torch.empty_like(z), None):
        loss, lse = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
        g.gar_distill_loss(z, index, teacher, 1.2, loss, lse, dz=dz, weight=weight)
        got.append((loss, lse))
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    assert g.gar_sync_status() == 0


# rows whose stages just fill, or just miss, the shared memory of two CTAs that share an SM
@pytest.mark.parametrize("vocab,dtype", [(16900, "bf16"), (17000, "bf16"), (17100, "bf16"), (8450, "f32"), (8500, "f32"), (8550, "f32")])
def test_rows_at_the_limit_of_two_ctas_an_sm(env, vocab, dtype):
    torch, g = env
    z, index, teacher, weight = problem(310, vocab, 64, 15, repeat=True)
    zt = device(torch, z, dtype)
    check(torch, g, zt, index, teacher, weight, 1.1, "fused")
    check(torch, g, zt, index, teacher, weight, 1.1, "split")
    assert g.gar_sync_status() == 0


@pytest.mark.parametrize("rows,vocab", [(5, 900), (5, 40000), (300, 50001)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_teachers_nan_shows(env, rows, vocab, dtype):
    """A NaN among a row's present entries makes its loss, and its gradient at the entries, NaN; absent ones (an index
    outside the vocabulary) and rows without weight do not see it."""
    torch, g = env
    z, index, teacher, weight = problem(rows, vocab, 8, 16)
    teacher[1, 2] = teacher[2, 3] = teacher[3, 0] = np.nan
    index[2, 3] = -1
    weight[3] = 0.0
    zt = device(torch, z, dtype)
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    loss, lse, dz = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(zt)
    g.gar_distill_loss(zt, to(index), to(teacher), 1.0, loss, lse, dz=dz, weight=to(weight))
    only = torch.arange(rows, device="cuda") == 1
    assert torch.equal(torch.isnan(loss), only) and not torch.isnan(lse).any()
    assert torch.equal(torch.isnan(dz).any(1), only)
    assert torch.isnan(dz[1, torch.from_numpy(index[1].astype(np.int64)).cuda()]).all() and torch.isnan(dz[1]).sum().item() == 8
    assert loss[3].item() == 0.0 and (dz[3] == 0).all()
