"""A worker step without weights takes 1 / tokens each: captured first and run
eagerly before any replay, it does not depend on what the capture recorded."""
import pytest

from helpers import need_cuda
from test_gpu_language import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return need_cuda()


def captured_then_eager(torch, build, run, results):
    """Of one step that ran eagerly alone, of one that was captured first, and of the capture's replay."""
    plain, fresh = build(), build()
    run(plain)
    torch.cuda.synchronize()
    want = [t.clone() for t in results(plain)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(fresh)
    run(fresh)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results(fresh)))
    for t in results(fresh):
        t.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results(fresh)))


def test_language_step(env):
    torch, g = env
    from gradient_allreduce_homomorphic_gb300.language import LanguageStep

    head, router, experts, hidden, target = make(torch, 2, 200, 64, 1000, 8, 90)
    captured_then_eager(torch, lambda: LanguageStep(head, router, experts, workers=2, tokens=200),
                        lambda s: s.run(5, hidden, target), lambda s: [*s.loss, *s.dx, *s.head_grad, *s.router_grad])
    assert g.gar_sync_status() == 0


def test_student_step(env):
    torch, g = env
    import test_gpu_student
    from gradient_allreduce_homomorphic_gb300.student import StudentStep

    head, router, hidden, index, teacher = test_gpu_student.make(torch, 2, 150, 200, 900, 12, 8, 91)
    captured_then_eager(torch, lambda: StudentStep(head, router, workers=2, tokens=150),
                        lambda s: s.run(5, hidden, index, teacher), lambda s: [*s.loss, *s.dx, *s.head_grad, *s.router_grad])
    assert g.gar_sync_status() == 0
