"""smoke() reaches the worker operators' kernels within its first few hundred device operations, so that a record of its
first launches shows them."""
import pytest

from helpers import need_cuda

pytestmark = pytest.mark.gpu


def test_worker_operators_come_early(monkeypatch):
    torch, _ = need_cuda()
    from torch.utils._python_dispatch import TorchDispatchMode

    import __graft_entry__
    from gradient_allreduce_homomorphic_gb300.student import StudentStep

    class Reached(Exception):
        pass

    class Count(TorchDispatchMode):
        operations = 0

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            self.operations += isinstance(out, torch.Tensor) and out.is_cuda and not func.is_view
            return out

    def run(self, *args, **kwargs):
        raise Reached

    monkeypatch.setattr(StudentStep, "run", run)
    with Count() as count, pytest.raises(Reached):
        __graft_entry__.smoke()
    assert count.operations < 300
