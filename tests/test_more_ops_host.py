"""Argument checks of the vocabulary layer's cross entropy, of the experts'
operators and of norm and clipping (no GPU needed, no kernel launched):
statuses at the C boundary, the binding's own checks of shapes and types."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def gar():
    from gradient_allreduce_homomorphic_gb300 import build

    build.build()
    import gradient_allreduce_homomorphic_gb300 as g

    g.load()
    return g


V = C.c_void_p
A, B, D, S, T, U, W = (V(0x10000 * (i + 1)) for i in range(7))
NULL = V(0)
BIG = 1 << 40


def test_vocab_loss_refusals(gar):
    f = gar.load().gar_vocab_loss

    def call(x=A, ldx=64, w=B, ldw=64, dtype=1, target=D, weight=NULL, rows=5, vocab=100, hidden=50, loss=S, lse=T, ws=U, n=BIG):
        return f(x, ldx, w, ldw, dtype, target, weight, rows, vocab, hidden, loss, lse, ws, n, NULL)

    assert call(dtype=0) == call(dtype=2) == gar.GAR_EDTYPE
    assert call(rows=-1) == call(vocab=0) == call(hidden=0) == call(rows=1 << 31) == call(vocab=1 << 31) == call(
        hidden=(1 << 20) + 1) == gar.GAR_EINVAL
    assert call(x=NULL) == call(w=NULL) == call(target=NULL) == call(loss=NULL) == call(lse=NULL) == call(ws=NULL) == gar.GAR_EINVAL
    assert call(ldx=48) == call(ldw=48) == call(n=16) == gar.GAR_EINVAL
    assert call(x=V(0x10008)) == call(w=V(0x10002)) == call(ldx=60) == call(ldw=57) == gar.GAR_EALIGN
    assert call(target=V(0x10002)) == call(weight=V(0x10001)) == call(loss=V(0x10002)) == call(ws=V(0x10080)) == gar.GAR_EALIGN
    assert call(rows=0) == gar.GAR_OK
    assert "workspace" in gar.gar_last_error()


def test_vocab_grad_refusals(gar):
    f = gar.load().gar_vocab_grad

    def call(x=A, ldx=64, w=B, ldw=64, dtype=1, target=D, weight=NULL, rows=5, vocab=100, hidden=50, lse=T, dx=S, lddx=50,
             add=NULL, ldadd=50, dw=W, lddw=50, dw_type=0, ws=U, n=BIG):
        return f(x, ldx, w, ldw, dtype, target, weight, rows, vocab, hidden, lse, dx, lddx, add, ldadd, dw, lddw, dw_type, ws, n, NULL)

    assert call(dtype=0) == call(dw_type=2) == gar.GAR_EDTYPE
    assert call(rows=-1) == call(vocab=0) == call(hidden=0) == gar.GAR_EINVAL
    assert call(dx=NULL, dw=NULL) == call(dw=NULL, add=S) == call(lse=NULL) == call(ws=NULL) == call(n=100) == gar.GAR_EINVAL
    assert call(lddx=49) == call(lddw=49) == call(add=S, ldadd=49) == call(add=W, ldadd=51) == gar.GAR_EINVAL
    assert call(dx=A) == call(dw=B) == gar.GAR_EINVAL
    assert call(dw=V(0x10002)) == call(dx=V(0x10001)) == call(add=V(0x10002)) == call(lse=V(0x10001)) == call(
        ws=V(0x10010)) == gar.GAR_EALIGN
    assert call(dw_type=1, dw=V(0x10001)) == gar.GAR_EALIGN
    assert call(rows=0, dw=NULL) == call(rows=0, add=W) == gar.GAR_OK


def test_vocab_workspace(gar):
    f = gar.load().gar_vocab_workspace_bytes
    assert f(-1, 5, 5, 0) == f(5, 0, 5, 0) == f(5, 5, 0, 0) == f(5, 5, 5, 2) == 0
    assert f(0, 5, 5, 0) > 0 and f(4096, 131072, 4096, 1) < f(4096, 131072, 4096, 0) + (1 << 29)
    torch = pytest.importorskip("torch")
    assert gar.gar_vocab_workspace_bytes(64, 1000, 64) == f(64, 1000, 64, 1)
    assert gar.gar_vocab_workspace_bytes(64, 1000, 64, torch.float32) == f(64, 1000, 64, 0)
    with pytest.raises(gar.GarError):
        gar.gar_vocab_workspace_bytes(64, 1000, 64, torch.float16)


@pytest.fixture
def binding(gar, monkeypatch):
    """Tensors that pass for device tensors, and calls that go nowhere: their name and arguments."""
    torch = pytest.importorskip("torch")
    made = []
    monkeypatch.setattr(gar, "_call", lambda name, *args: made.append((name, args)))
    monkeypatch.setattr(gar, "_stream", lambda stream: 0)

    class OnDevice(torch.Tensor):
        is_cuda = True

    def tensor(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)

    def refused(fn, *args, **kw):
        with pytest.raises(gar.GarError) as e:
            fn(*args, **kw)
        return e.value.status

    return torch, tensor, made, refused


def test_vocab_binding(gar, binding):
    torch, tensor, made, refused = binding
    bf, i32 = torch.bfloat16, torch.int32
    x, w, target = tensor(6, 64, dtype=bf), tensor(30, 64, dtype=bf), tensor(6, dtype=i32)
    loss, lse, ws = tensor(6), tensor(6), tensor(4096, dtype=torch.uint8)
    gar.gar_vocab_loss(x, w, target, loss, lse, ws, weight=tensor(6))
    gar.gar_vocab_grad(x, w, target, lse, tensor(6, 64, dtype=bf), tensor(30, 64), ws, addend=tensor(30, 70)[:, 3:67])
    assert [n for n, _ in made] == ["gar_vocab_loss", "gar_vocab_grad"]
    args = made[1][1]
    assert args[12] == 64 and args[14] == 70 and args[17] == gar.GAR_F32
    loss_of, grad_of = gar.gar_vocab_loss, gar.gar_vocab_grad
    assert refused(loss_of, x, tensor(30, 64), target, loss, lse, ws) == gar.GAR_EDTYPE
    assert refused(loss_of, x, tensor(30, 56, dtype=bf), target, loss, lse, ws) == gar.GAR_EINVAL
    assert refused(loss_of, x, w, tensor(6), loss, lse, ws) == gar.GAR_EDTYPE
    assert refused(loss_of, x, w, tensor(5, dtype=i32), loss, lse, ws) == gar.GAR_EINVAL
    assert refused(loss_of, x, w, target, tensor(6, 2)[:, 0], lse, ws) == gar.GAR_EINVAL
    assert refused(loss_of, tensor(6, 128, dtype=bf)[:, ::2], w, target, loss, lse, ws) == gar.GAR_EINVAL
    assert refused(loss_of, tensor(6, dtype=bf), w, target, loss, lse, ws) == gar.GAR_EINVAL
    assert refused(loss_of, torch.zeros(6, 64, dtype=bf), w, target, loss, lse, ws) == gar.GAR_EINVAL
    dx, dw = tensor(6, 64, dtype=bf), tensor(30, 64, dtype=bf)
    assert refused(grad_of, x, w, target, lse, tensor(6, 64), dw, ws) == gar.GAR_EDTYPE
    assert refused(grad_of, x, w, target, lse, dx, tensor(30, 64, dtype=torch.float16), ws) == gar.GAR_EDTYPE
    assert refused(grad_of, x, w, target, lse, dx, dw, ws, addend=tensor(30, 64)) == gar.GAR_EDTYPE
    assert refused(grad_of, x, w, target, lse, dx, None, ws, addend=dw) == gar.GAR_EDTYPE
    assert refused(grad_of, x, w, target, lse, dx, tensor(31, 64), ws) == gar.GAR_EINVAL
