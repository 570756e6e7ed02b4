"""Sums of the vocabulary layer longer than an accumulator adds up (8192 terms of a
logit, 32768 of a bf16 result), against 64 bits.

u = 2^-24.  The tensor cores' additions round toward zero, 2 u each, one for a term at
most: an accumulator's sum is within 2 u 8192 (or 32768) of the sum of its terms'
absolute values, the addition of the accumulators within u each.  Where the logits are
multiples of 2^-8 below 2^16 every such addition is exact, however it is cut; then
  lse    300 u and 4 u of itself, as for few terms
  g      of itself lse's error, 2^-22 and 4 u (1 + log2(e) |z - lse|); of the target the same
         of p, or of its loss
  dx, dw g's rounding to bf16 2^-8 (fp32 dw: 2^-16), 2 u a term, the result's half step"""
import pytest

from helpers import need_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LOG2E = 1.4426950408889634


@pytest.fixture(scope="module")
def env():
    return need_cuda()


def of(torch, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def workspace(torch, g, rows, vocab, hidden, dw_type):
    return torch.full((g.gar_vocab_workspace_bytes(rows, vocab, hidden, dw_type),), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("with_loss", [False, True])
@pytest.mark.parametrize("dw_type", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,hidden", [(1, 70, 8200), (300, 1000, 8256), (130, 513, 20001), (33, 300, 65544)])
def test_exact_logits_of_long_rows(env, rows, vocab, hidden, dw_type, with_loss):
    torch, g = env
    gen, t = of(torch, hidden), torch.float32 if dw_type == "f32" else torch.bfloat16
    ld = (hidden + 7) // 8 * 8
    x = (torch.randint(-1, 2, (rows, ld), generator=gen, device="cuda")).bfloat16()[:, :hidden]
    w = (torch.randint(-1, 2, (vocab, ld), generator=gen, device="cuda") / 64).bfloat16()[:, :hidden]
    target = torch.randint(0, vocab, (rows,), generator=gen, device="cuda").int()
    if rows > 5:
        target[5] = -1
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dx, dw = torch.empty((rows, hidden), dtype=torch.bfloat16, device="cuda"), torch.empty((vocab, hidden), dtype=t, device="cuda")
    ws = workspace(torch, g, rows, vocab, hidden, t)
    g.gar_vocab_loss(x, w, target, loss, lse, ws)
    if with_loss:
        g.gar_vocab_grad_with_loss(x, w, target, loss, lse, dx, dw, ws)
    else:
        g.gar_vocab_grad(x, w, target, lse, dx, dw, ws)
    torch.cuda.synchronize()
    assert g.gar_sync_status() == 0
    on = target >= 0
    at = target.long().clamp(min=0)[:, None]
    z = x.double() @ w.double().t()
    want_lse = torch.logsumexp(z, 1)
    want_loss = want_lse - z.gather(1, at)[:, 0]
    e_lse = 300 * U + 4 * U * want_lse.abs()
    for got, want, tol in ((lse, want_lse, e_lse), (loss, want_loss, e_lse + 8 * U * want_loss)):
        assert ((got.double() - want).abs() <= tol)[on].all() and bool((got[~on] == 0).all())
    p = torch.exp(z - want_lse[:, None])
    G = p.scatter_add(1, at, -torch.ones_like(at, dtype=torch.float64)) * on[:, None]
    e_g = p * (e_lse[:, None] + 2 ** -22 + 4 * U * (1 + LOG2E * (z - want_lse[:, None]).abs())) * on[:, None] + 4 * U * G.abs()
    half, part = (U, 2 ** -16) if dw_type == "f32" else (2 ** -8, 2 ** -8)
    X, W = x.double(), w.double()
    want = G @ W
    tol = (1.02 * e_g + (1.02 * 2 ** -8 + 2 * U * (vocab + 80)) * G.abs()) @ W.abs() * 1.01 + 2 ** -8 * want.abs()
    assert ((dx.double() - want).abs() <= tol + 1e-30).all()
    want = G.t() @ X
    tol = (1.02 * e_g + (1.02 * part + 2 * U * (2 * rows + 80)) * G.abs()).t() @ X.abs() * 1.01 + half * want.abs()
    assert ((dw.double() - want).abs() <= tol + 1e-30).all()


def test_logits_of_one_sign(env):
    """2^20 positive products to a logit."""
    torch, g = env
    gen, hidden = of(torch, 1), 1 << 20
    x = (torch.rand((16, hidden), generator=gen, device="cuda") + 0.5).bfloat16()
    w = ((torch.rand((64, hidden), generator=gen, device="cuda") + 0.5) * (40.0 / hidden)).bfloat16()
    target = torch.arange(16, device="cuda").int()
    loss, lse = torch.empty(16, device="cuda"), torch.empty(16, device="cuda")
    g.gar_vocab_loss(x, w, target, loss, lse, workspace(torch, g, 16, 64, hidden, torch.bfloat16))
    torch.cuda.synchronize()
    z = x.double() @ w.double().t()
    want = torch.logsumexp(z, 1)
    ez = (2 * U * 8192 + U * (hidden / 8192 + 1)) * z.amax(1)  # every product is positive
    assert ((lse.double() - want).abs() <= ez + 300 * U + 4 * U * want).all()


@pytest.mark.parametrize("pad,addend", [(0, False), (0, True), (3, False), (3, True)])
@pytest.mark.parametrize("rows", [1 << 22, 98401])
def test_a_bf16_dw_of_many_rows(env, rows, pad, addend):
    """g^T x of one sign for the entries that are no target; rows on 16 bytes and off them, with and without an addend."""
    torch, g = env
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    gen, vocab, hidden = of(torch, 2), 96, 64
    x = (torch.rand((rows, hidden), generator=gen, device="cuda") + 0.5).bfloat16()
    w = (torch.randn((vocab, hidden), generator=gen, device="cuda") * 0.1).bfloat16()
    target = torch.randint(0, 48, (rows,), generator=gen, device="cuda").int()
    weight = torch.full((rows,), 1.0 / rows, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    whole = torch.full((vocab, hidden + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = whole[:, :hidden]
    add = torch.randn((vocab, hidden), generator=gen, device="cuda").mul_(1e-3).bfloat16() if addend else None
    ws = workspace(torch, g, rows, vocab, hidden, torch.bfloat16)
    g.gar_vocab_loss(x, w, target, loss, lse, ws, weight=weight)
    g.gar_vocab_grad(x, w, target, lse, None, dw, ws, weight=weight, addend=add)
    torch.cuda.synchronize()
    assert g.gar_sync_status() == 0 and bool((whole[:, hidden:] == 7).all())
    want, size = (torch.zeros((vocab, hidden), dtype=torch.float64, device="cuda") for _ in range(2))
    for i in range(0, rows, 1 << 18):
        X = x[i:i + (1 << 18)].double()
        G = torch.softmax(X @ w.double().t(), 1)
        G.scatter_add_(1, target[i:i + (1 << 18)].long()[:, None], -torch.ones((len(X), 1), dtype=torch.float64, device="cuda"))
        want += G.t() @ X / rows
        size += G.abs().t() @ X / rows
    if addend:
        want += add.double()
    # of each term: g's rounding, its exponential's error and lse's (below 1e-5), an accumulator's sum, 128 accumulators'
    tol = (2 ** -8 + 1e-5 + 2 * U * 32768 + 128 * U) * size + 2 ** -8 * want.abs()
    assert ((dw.double() - want).abs() <= tol).all()


def test_dx_of_a_long_vocabulary(env):
    """More tiles of dx than CTA pairs, so that whole sums of 200000 terms go to one accumulator."""
    torch, g = env
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    gen, rows, vocab, hidden = of(torch, 3), 512, 200000, 9736
    x = torch.zeros((rows, hidden), dtype=torch.bfloat16, device="cuda")
    x[:, :8] = torch.randn((rows, 8), generator=gen, device="cuda").bfloat16()
    w = torch.empty((vocab, hidden), dtype=torch.bfloat16, device="cuda")
    for part in w.split(20000):
        part.copy_(torch.rand(part.shape, generator=gen, device="cuda") + 0.5)
    target = torch.randint(0, vocab, (rows,), generator=gen, device="cuda").int()
    target[7] = -1
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dx = torch.full((rows, hidden), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = workspace(torch, g, rows, vocab, hidden, torch.bfloat16)
    g.gar_vocab_loss(x, w, target, loss, lse, ws)
    g.gar_vocab_grad(x, w, target, lse, dx, None, ws)
    torch.cuda.synchronize()
    assert g.gar_sync_status() == 0
    G = torch.softmax(x[:, :8].double() @ w[:, :8].double().t(), 1)
    at = target.long().clamp(min=0)[:, None]
    G.scatter_add_(1, at, -torch.ones_like(at, dtype=torch.float64))
    G[7] = 0.0
    some = w[:, ::61].double()
    want, size = G @ some, G.abs() @ some
    tol = (2 ** -8 + 1e-5 + 2 * U * 32768 + 8 * U) * size + 2 ** -8 * want.abs()
    assert ((dx[:, ::61].double() - want).abs() <= tol).all() and bool((dx[7] == 0).all())


@pytest.mark.parametrize("addend", ["none", "given", "in place"])
@pytest.mark.parametrize("hidden,pad", [(64, 0), (61, 0), (64, 3), (72, 8)])
def test_segments_of_an_fp32_dw(env, hidden, pad, addend):
    """More than 4096 rows (two parts of g each): the first segment takes the addend, the later ones what is in dw; rows of
    dw on 16 bytes and off them, a last tile that is not full."""
    torch, g = env
    gen, rows, vocab = of(torch, 5), 9001, 300
    x = torch.randn((rows, (hidden + 7) // 8 * 8), generator=gen, device="cuda").add_(0.25).bfloat16()[:, :hidden]
    w = (torch.randn((vocab, (hidden + 7) // 8 * 8), generator=gen, device="cuda") * 0.2).bfloat16()[:, :hidden]
    target = torch.randint(0, vocab, (rows,), generator=gen, device="cuda").int()
    target[::11] = -1
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    whole = torch.full((vocab, hidden + pad), 7.0, device="cuda")
    dw, add = whole[:, :hidden], None
    before = torch.randn((vocab, hidden), generator=gen, device="cuda")
    if addend == "given":
        add = before.clone()
    elif addend == "in place":
        dw.copy_(before)
        add = dw
    ws = workspace(torch, g, rows, vocab, hidden, torch.float32)
    g.gar_vocab_loss(x, w, target, loss, lse, ws)
    g.gar_vocab_grad(x, w, target, lse, None, dw, ws, addend=add)
    torch.cuda.synchronize()
    assert g.gar_sync_status() == 0 and bool((whole[:, hidden:] == 7).all())
    X, on = x.double(), (target >= 0)[:, None]
    G = torch.softmax(X @ w.double().t(), 1)
    at = target.long().clamp(min=0)[:, None]
    G.scatter_add_(1, at, -torch.ones_like(at, dtype=torch.float64))
    G *= on
    want = G.t() @ X + (before.double() if add is not None else 0.0)
    # of each term: g's parts, its exponential's error and lse's (below 1e-5); a segment's sum; the segments'
    tol = (2 ** -16 + 1e-5 + 2 * U * 8192) * (G.abs().t() @ X.abs()) + 8 * U * (want.abs() + before.double().abs() + 1)
    assert ((dw.double() - want).abs() <= tol).all()
    if addend != "in place":  # and as closely as random signs allow: a segment left out or taken twice shows
        assert (dw.double() - want).norm() <= 1e-4 * (want - (before.double() if add is not None else 0.0)).norm()


@pytest.mark.parametrize("rows", [4096, 16384])
def test_small_terms_behind_a_large_one_of_an_fp32_dw(env, rows):
    """Row 0 with weight 1, all others with 7/8 2^-27, all their logits 0 and their x 1: every term of a dw that is no
    target's is positive, 2^-8 and 7/8 2^-35.  16 of the small ones are below one step of the large one and are lost behind
    it, but in its accumulator alone, 2048 rows: rounding toward zero, no sum of positive terms falls below a part of it.
    So what is missing is at most those 2047 terms; the exponentials' 2^-21 and the additions' 4 u besides."""
    torch, g = env
    x = torch.ones((rows, 64), device="cuda").bfloat16()
    w = torch.zeros((256, 64), device="cuda").bfloat16()
    target = torch.full((rows,), 5, dtype=torch.int32, device="cuda")
    small = 0.875 * 2.0 ** -27
    weight = torch.full((rows,), small, device="cuda")
    weight[0] = 1.0
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw = torch.empty((256, 64), device="cuda")
    ws = workspace(torch, g, rows, 256, 64, torch.float32)
    g.gar_vocab_loss(x, w, target, loss, lse, ws, weight=weight)
    g.gar_vocab_grad(x, w, target, lse, None, dw, ws, weight=weight)
    torch.cuda.synchronize()
    want = (1.0 + (rows - 1) * small) / 256
    got = torch.cat([dw[:5], dw[6:]]).double()
    assert (got - want).abs().max().item() <= (2047 * small + 2.0 ** -21 + 4 * U) / 256
