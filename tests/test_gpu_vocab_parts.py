"""The vocabulary layer's gradient from both parts of g (parts=2): dx and a bf16 dw to
their own rounding.

Tolerances as in test_gpu_vocab.py, with g's 2^-8 replaced by the 2^-16 of two bf16
values: e before the result's rounding.  A value within e of the exact one is rounded to
the same bf16, or both lie within e of the middle between two: either way it ends no more
than 2 e further from the exact value than that one's own bf16."""
import pytest

from helpers import need_cuda
from test_gpu_vocab import U, Problem, outputs, within, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return need_cuda()


def run(torch, g, p, dw_type, parts, addend=None, pad=0):
    loss, lse, dx, dw = outputs(torch, p, dw_type, pad)
    ws, h = workspace(torch, g, p, torch.float32), p.hidden
    g.gar_vocab_loss(p.x, p.w, p.target, loss, lse, ws, weight=p.weight)
    g.gar_vocab_grad_with_loss(p.x, p.w, p.target, loss, lse, dx[:, :h], dw[:, :h], ws, weight=p.weight, addend=addend, parts=parts)
    torch.cuda.synchronize()
    assert g.gar_sync_status() == 0
    assert bool((dx[:, h:] == 7).all()) and bool((dw[:, h:] == 7).all())
    return dx[:, :h], dw[:, :h]


@pytest.mark.parametrize("dw", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,hidden,pad,addend", [(1, 1, 1, 0, False), (3, 257, 64, 3, True), (257, 1000, 1000, 0, False),
                                                          (130, 4099, 264, 0, True), (700, 2049, 100, 0, False), (16, 30001, 136, 0, False),
                                                          (4500, 31000, 40, 0, False), (512, 40000, 2056, 0, False)])
def test_against_64_bits(env, rows, vocab, hidden, pad, addend, dw):
    torch, g = env
    t = torch.float32 if dw == "f32" else torch.bfloat16
    p = Problem(torch, rows, vocab, hidden, seed=31)
    add = (torch.randn((vocab, hidden), generator=p.gen, device="cuda") * 1e-3).to(t) if addend else None
    dx, got = run(torch, g, p, t, 2, add, pad)
    p.reference()
    want, big = p.g @ p.w64, p.g.abs() @ p.w64.abs()
    e = 1.02 * (p.e_g @ p.w64.abs()) + (1.02 * 2.0 ** -16 + 2 * U * (2 * vocab + 80)) * big
    within(dx, want, 2.02 * e + (want.bfloat16().double() - want).abs(), "dx")
    want, big = p.g.t() @ p.x64, p.g.abs().t() @ p.x64.abs()
    e = 1.02 * (p.e_g.t() @ p.x64.abs()) + (1.02 * 2.0 ** -16 + 2 * U * (2 * rows + 80)) * big
    if addend:
        want, e = want + add.double(), e + 2 * U * add.double().abs()
    within(got, want, 2.02 * e + (want.to(t).double() - want).abs(), "dw")


def test_one_part_is_what_is_taken_without_being_asked(env):
    torch, g = env
    p = Problem(torch, 200, 3000, 128, seed=32)
    for a, b in zip(run(torch, g, p, torch.bfloat16, 0), run(torch, g, p, torch.bfloat16, 1)):
        assert torch.equal(a, b)
    two = run(torch, g, p, torch.float32, 0)
    asked = run(torch, g, p, torch.float32, 2)
    assert torch.equal(two[1], asked[1]) and not torch.equal(two[0], asked[0])


def test_the_same_bits_in_every_run_and_in_a_graph(env):
    torch, g = env
    p = Problem(torch, 300, 9001, 200, seed=33)
    want = run(torch, g, p, torch.bfloat16, 2)
    assert all(torch.equal(a, b) for a, b in zip(want, run(torch, g, p, torch.bfloat16, 2)))
    loss, lse, dx, dw = outputs(torch, p, torch.bfloat16)
    ws, graph = workspace(torch, g, p, torch.float32), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gar_vocab_loss(p.x, p.w, p.target, loss, lse, ws, weight=p.weight)
        g.gar_vocab_grad_with_loss(p.x, p.w, p.target, loss, lse, dx, dw, ws, weight=p.weight, parts=2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
