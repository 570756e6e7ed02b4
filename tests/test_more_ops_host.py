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


def tables(P, *places):
    return [(V * P)(*[p + 0x100000 * i for i in range(P)]) for p in places]


def test_expert_rows(gar):
    f = gar.load().gar_expert_rows
    assert f(2, 10, 3, 4, 1, 0) == 60 and f(2, 10, 3, 4, 128, 0) == 60 + 4 * 127 and f(2, 10, 3, 4, 1, 9) == 36
    assert f(0, 1, 1, 1, 1, 0) == f(1, -1, 1, 1, 1, 0) == f(1, 1, 33, 1, 1, 0) == f(1, 1, 1, 1025, 1, 0) == f(1, 1, 1, 1, 0, 0) == -1
    assert f(64, 1 << 62, 1, 1, 1, 0) == -1
    with pytest.raises(gar.GarError):
        gar.gar_expert_rows(1, 1, 0, 1)
    assert gar.gar_expert_workspace_bytes(1, 10, 2, 8) > 0 and gar.gar_expert_workspace_bytes(65, 10, 2, 8) == 0


def test_expert_sort_refusals(gar):
    c, p = tables(2, 0x1000000, 0x2000000)

    def call(choice=c, P=2, tokens=10, k=2, experts=4, align=1, capacity=0, position=p, source=S, rows=40, offsets=T, ws=U, n=1 << 20):
        return gar.load().gar_expert_sort(choice, P, tokens, k, experts, align, capacity, position, source, rows, offsets, ws, n, NULL)

    assert call(P=0) == call(P=65) == call(tokens=-1) == call(k=0) == call(k=33) == call(experts=0) == call(
        experts=1025) == gar.GAR_EINVAL
    assert call(align=0) == call(capacity=-1) == call(capacity=8, align=2) == call(rows=39) == call(align=8) == call(
        rows=1 << 31) == gar.GAR_EINVAL
    assert call(tokens=1 << 29, rows=(1 << 31) - 1) == call(tokens=1 << 62) == gar.GAR_EINVAL
    assert call(choice=None) == call(position=None) == call(source=NULL) == call(offsets=NULL) == call(ws=NULL) == call(
        n=10) == gar.GAR_EINVAL
    assert call(choice=(V * 2)(0x1000, None)) == gar.GAR_EINVAL
    assert call(choice=(V * 2)(0x1000, 0x1002)) == call(source=V(0x10001)) == call(ws=V(0x10002)) == gar.GAR_EALIGN


def test_expert_move_refusals(gar):
    x, pos, w, o = tables(2, 0x1000000, 0x2000000, 0x3000000, 0x4000000)
    lib = gar.load()

    def gather(x=x, P=2, tokens=10, hidden=16, ldx=16, dtype=0, k=2, position=pos, source=S, rows=40, weight=w, y=T, ldy=16):
        return lib.gar_expert_gather(x, P, tokens, hidden, ldx, dtype, k, position, source, rows, weight, y, ldy, NULL)

    def combine(y=T, ldy=16, rows=40, P=2, tokens=10, hidden=16, dtype=0, k=2, position=pos, weight=w, add=x, ldadd=16, out=o, ldo=16):
        return lib.gar_expert_combine(y, ldy, rows, P, tokens, hidden, dtype, k, position, weight, add, ldadd, out, ldo, NULL)

    def grad(dout=x, ldd=16, y=T, ldy=16, P=2, tokens=10, hidden=16, dtype=0, k=2, position=pos, source=S, rows=40, weight=w, dy=U,
             lddy=16, dweight=o):
        return lib.gar_expert_combine_grad(dout, ldd, y, ldy, P, tokens, hidden, dtype, k, position, source, rows, weight, dy, lddy,
                                           dweight, NULL)

    bad = (V * 2)(0x1000, None)
    odd = (V * 2)(0x1000, 0x1002)
    for f in (gather, combine, grad):
        assert f(dtype=2) == gar.GAR_EDTYPE
        assert f(P=0) == f(P=65) == f(tokens=-1) == f(hidden=0) == f(k=0) == f(k=33) == f(rows=-1) == f(rows=1 << 31) == gar.GAR_EINVAL
        assert f(position=None) == f(position=bad) == f(weight=bad) == f(tokens=1 << 60) == gar.GAR_EINVAL
        assert f(position=odd) == f(weight=odd) == gar.GAR_EALIGN
    assert gather(ldx=15) == gather(ldy=15) == gather(x=bad) == gather(y=NULL) == gather(source=NULL) == gar.GAR_EINVAL
    assert gather(x=odd) == gather(y=V(0x10002)) == gather(source=V(0x10001)) == gar.GAR_EALIGN
    assert combine(ldy=15) == combine(ldo=15) == combine(ldadd=15) == combine(out=None) == combine(y=NULL) == gar.GAR_EINVAL
    assert combine(add=o, ldadd=17) == combine(add=bad) == gar.GAR_EINVAL
    assert combine(out=odd) == combine(add=odd) == gar.GAR_EALIGN
    assert combine(tokens=0) == gar.GAR_OK
    assert grad(ldd=15) == grad(ldy=15) == grad(lddy=15) == grad(weight=None) == grad(dweight=bad) == grad(dy=NULL) == grad(
        source=NULL) == grad(dy=T, lddy=17) == gar.GAR_EINVAL
    assert grad(dy=V(0x10001)) == grad(dout=odd) == grad(dweight=odd) == gar.GAR_EALIGN
    assert gather(tokens=0, rows=0) == grad(tokens=0, rows=0) == gar.GAR_OK


def test_expert_weights_refusals(gar):
    z, c, w = tables(2, 0x1000000, 0x2000000, 0x3000000)
    lib = gar.load()

    def weights(z=z, P=2, tokens=10, experts=8, ldz=8, dtype=0, k=2, choice=c, weight=w):
        return lib.gar_expert_weights(z, P, tokens, experts, ldz, dtype, k, choice, weight, NULL)

    def grad(weight=w, dweight=w, P=2, tokens=10, experts=8, k=2, choice=c, z=z, ldz=8, dtype=0):
        return lib.gar_expert_weights_grad(weight, dweight, P, tokens, experts, k, choice, z, ldz, dtype, 0, NULL)

    bad, odd = (V * 2)(0x1000, None), (V * 2)(0x1000, 0x1002)
    for f in (weights, grad):
        assert f(dtype=3) == gar.GAR_EDTYPE
        assert f(P=0) == f(experts=0) == f(experts=1025) == f(ldz=7) == f(k=0) == f(k=33) == f(tokens=-1) == gar.GAR_EINVAL
        assert f(z=bad) == f(choice=bad) == f(weight=bad) == f(z=None) == f(choice=None) == f(weight=None) == gar.GAR_EINVAL
        assert f(z=odd) == f(choice=odd) == f(weight=odd) == gar.GAR_EALIGN
        assert f(tokens=0) == gar.GAR_OK
    assert grad(dweight=bad) == gar.GAR_EINVAL


def test_clip_refusals(gar):
    lib = gar.load()
    src, dst = (V * 4)(*range(0x1000, 0x5000, 0x1000)), (V * 4)(*range(0x11000, 0x15000, 0x1000))
    numel, dtype = (C.c_int64 * 2)(10, 20), (C.c_int32 * 2)(0, 1)

    def clip(src=src, dst=dst, P=2, numel=numel, dtype=dtype, count=2, shared=0, top=1.0, norm=S, ws=T, n=1 << 20):
        return lib.gar_grad_clip(src, dst, P, numel, dtype, count, shared, top, norm, ws, n, NULL)

    def norm(src=src, P=2, numel=numel, dtype=dtype, count=2, norm=S, ws=T, n=1 << 20):
        return lib.gar_grad_norm(src, P, numel, dtype, count, norm, ws, n, NULL)

    for f in (clip, norm):
        assert f(P=0) == f(P=65) == f(count=-1) == f(src=None) == f(numel=None) == f(dtype=None) == f(norm=NULL) == f(
            ws=NULL) == f(n=100) == gar.GAR_EINVAL
        assert f(numel=(C.c_int64 * 2)(10, -1)) == f(src=(V * 4)(0x1000, 0x2000, None, 0x4000)) == gar.GAR_EINVAL
        assert f(dtype=(C.c_int32 * 2)(0, 2)) == gar.GAR_EDTYPE
        assert f(src=(V * 4)(0x1000, 0x2000, 0x3002, 0x4000)) == f(norm=V(0x10002)) == f(ws=V(0x10004)) == gar.GAR_EALIGN
    assert clip(top=-1.0) == clip(top=float("nan")) == clip(dst=None) == gar.GAR_EINVAL
    assert clip(dst=(V * 4)(0x1000, 0x2000, 0x3000, 0x4001)) == gar.GAR_EALIGN
    assert lib.gar_grad_workspace_bytes(0, 5) == lib.gar_grad_workspace_bytes(1, -1) == 0


def test_expert_binding(gar, binding):
    torch, tensor, made, refused = binding
    i32 = torch.int32
    choice, position = ([tensor(6, 2, dtype=i32) for _ in range(3)] for _ in range(2))
    source, offsets, ws = tensor(40, dtype=i32), tensor(5, dtype=i32), tensor(64)
    x, weight, out = [tensor(6, 16) for _ in range(3)], [tensor(6, 2) for _ in range(3)], [tensor(6, 16) for _ in range(3)]
    y, dy, dweight = tensor(40, 20)[:, 2:18], tensor(40, 16), [tensor(6, 2) for _ in range(3)]
    z, dz = [tensor(6, 4) for _ in range(3)], [tensor(6, 4, dtype=torch.bfloat16) for _ in range(3)]
    gar.gar_expert_sort(choice, 4, position, source, offsets, ws, align=2)
    gar.gar_expert_gather(x, position, source, y, weight=weight)
    gar.gar_expert_combine(y, position, out, weight=weight, addend=x)
    gar.gar_expert_combine_grad(x, y, position, source, weight, dy, dweight)
    gar.gar_expert_weights(z, choice, weight)
    gar.gar_expert_weights_grad(weight, dweight, choice, dz)
    assert [n for n, _ in made] == ["gar_expert_sort", "gar_expert_gather", "gar_expert_combine", "gar_expert_combine_grad",
                                    "gar_expert_weights", "gar_expert_weights_grad"]
    E, D = gar.GAR_EINVAL, gar.GAR_EDTYPE
    assert refused(gar.gar_expert_sort, choice, 4, position[:2], source, offsets, ws) == E
    assert refused(gar.gar_expert_sort, choice, 5, position, source, offsets, ws) == E
    assert refused(gar.gar_expert_sort, choice, 4, [tensor(6, 4, dtype=i32)[:, ::2] for _ in range(3)], source, offsets, ws) == E
    assert refused(gar.gar_expert_sort, choice, 4, weight, source, offsets, ws) == D
    assert refused(gar.gar_expert_sort, [], 4, [], source, offsets, ws) == E
    assert refused(gar.gar_expert_gather, x, position, source, tensor(39, 16)) == E
    assert refused(gar.gar_expert_gather, x, position, source, tensor(40, 16, dtype=torch.bfloat16)) == D
    assert refused(gar.gar_expert_gather, [tensor(6, 16, dtype=torch.float16)] * 3, position, source, y) == D
    assert refused(gar.gar_expert_gather, x, position, source, y, weight=choice) == D
    assert refused(gar.gar_expert_combine, tensor(40, 15), position, out) == E
    assert refused(gar.gar_expert_combine, y, position, out, addend=x[:2]) == E
    assert refused(gar.gar_expert_combine_grad, x, y, position, source, weight, tensor(40, 16, dtype=torch.bfloat16), dweight) == D
    assert refused(gar.gar_expert_combine_grad, x, y, position, source, weight, dy, [tensor(6, 3) for _ in range(3)]) == E
    assert refused(gar.gar_expert_weights, z, choice, [tensor(5, 2) for _ in range(3)]) == E
    assert refused(gar.gar_expert_weights_grad, weight, dweight, choice, [tensor(7, 4) for _ in range(3)]) == E


def test_clip_binding(gar, binding):
    torch, tensor, made, refused = binding
    grads = [[tensor(10, 3), tensor(7, dtype=torch.bfloat16)] for _ in range(2)]
    out = [[tensor(30), tensor(7, dtype=torch.bfloat16)] for _ in range(2)]
    norm, ws = tensor(2), tensor(1 << 14)
    t = gar.grad_tables(grads, out)
    assert t.P == 2 and t.count == 2 and list(t.numel) == [30, 7] and list(t.dtype) == [0, 1]
    assert gar.grad_tables(t) is t and gar.gar_grad_workspace_bytes(t) == gar.gar_grad_workspace_bytes(grads)
    gar.gar_grad_norm(grads, norm, ws)
    gar.gar_grad_clip(t, 1.0, norm, ws)
    gar.gar_grad_clip(grads, 1.0, tensor(1), ws, out=out, shared=True)
    assert [n for n, _ in made] == ["gar_grad_norm", "gar_grad_clip", "gar_grad_clip"]
    E, D = gar.GAR_EINVAL, gar.GAR_EDTYPE
    assert refused(gar.gar_grad_clip, t, 1.0, tensor(1), ws) == refused(gar.gar_grad_clip, t, 1.0, norm, ws, shared=True) == E
    assert refused(gar.gar_grad_norm, t, tensor(2, dtype=torch.float64), ws) == D
    assert refused(gar.grad_tables, []) == refused(gar.grad_tables, [[tensor(3)], []]) == refused(gar.grad_tables, grads, out[:1]) == E
    assert refused(gar.grad_tables, grads, [[tensor(31), out[0][1]], out[1]]) == E
    assert refused(gar.grad_tables, [[tensor(4, 4)[:, ::2]]]) == E
    assert refused(gar.gar_grad_clip, t, 1.0, norm, ws, out=out) == E
    same = tensor(8)
    assert refused(gar.grad_tables, [[same, same]]) == refused(gar.grad_tables, [[tensor(8)], [tensor(8)]], [[same], [same]]) == E
    gar.grad_tables([[same, same]], [[tensor(8), tensor(8)]])  # read twice, written apart
    assert refused(gar.grad_tables, grads, [[tensor(30, dtype=torch.bfloat16), out[0][1]], out[1]]) == D
    assert refused(gar.grad_tables, [[tensor(3, dtype=torch.float16)]]) == D
    assert refused(gar.grad_tables, [[torch.zeros(3)]]) == E
