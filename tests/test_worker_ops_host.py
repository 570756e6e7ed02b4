"""Argument checks of the operators that a worker runs before its gradients are
averaged (no GPU needed, no kernel launched): statuses at the C boundary, the
binding's own checks of shapes and types."""
import ctypes as C

import numpy as np
import pytest

import worker_ref as ref


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


def test_quantize_refusals(gar):
    f = gar.load().gar_fp8_quantize

    def call(x=A, dtype=0, rows=10, cols=100, ldx=100, fmt=0, square=0, q=B, ldq=112, s=S, qt=D, ldqt=16, st=T):
        return f(x, dtype, rows, cols, ldx, fmt, square, q, ldq, s, qt, ldqt, st, NULL)

    assert call(rows=-1) == call(cols=-1) == call(cols=1 << 31) == gar.GAR_EINVAL
    assert call(dtype=2) == call(fmt=2) == gar.GAR_EDTYPE
    assert call(q=NULL, qt=NULL) == call(x=NULL) == call(ldx=99) == gar.GAR_EINVAL
    assert call(s=NULL) == call(st=NULL) == call(ldq=96) == call(ldqt=0) == gar.GAR_EINVAL
    assert call(ldq=101) == call(q=V(0x10008)) == call(qt=V(0x10001)) == call(s=V(0x10002)) == gar.GAR_EALIGN
    assert call(x=V(0x10002)) == call(x=V(0x10001), dtype=1) == gar.GAR_EALIGN
    assert call(rows=0) == call(cols=0, ldx=0) == gar.GAR_OK
    assert "scales" in gar.gar_last_error() or gar.gar_last_error()


def test_matmul_refusals(gar):
    f = gar.load().gar_fp8_matmul

    def call(a=A, lda=64, sa=S, fa=0, b=B, ldb=64, sb=T, fb=1, M=4, N=5, K=50, c=NULL, ldc=0, d=D, ldd=5, dtype=0):
        return f(a, lda, sa, fa, b, ldb, sb, fb, M, N, K, c, ldc, d, ldd, dtype, NULL)

    assert call(M=-1) == call(N=-1) == call(K=-1) == call(M=1 << 31) == gar.GAR_EINVAL
    assert call(dtype=7) == call(fa=2) == call(fb=-1) == gar.GAR_EDTYPE
    assert call(a=NULL) == call(sb=NULL) == call(lda=48) == call(d=NULL) == call(ldd=4) == gar.GAR_EINVAL
    assert call(c=U, ldc=4) == call(c=D, ldc=6, ldd=5) == gar.GAR_EINVAL
    assert call(a=V(0x10008)) == call(ldb=72) == call(sa=V(0x10001)) == call(d=V(0x10002)) == gar.GAR_EALIGN
    assert call(M=0) == call(N=0) == gar.GAR_OK


def test_distill_refusals(gar):
    lib = gar.load()

    def loss(z=A, dtype=0, rows=3, vocab=10, ldz=10, i=B, t=D, k=2, tau=1.0, w=NULL, loss=S, lse=T, dz=NULL, lddz=0):
        return lib.gar_distill_loss(z, dtype, rows, vocab, ldz, i, t, k, tau, w, loss, lse, dz, lddz, NULL)

    assert loss(rows=-1) == loss(vocab=0) == loss(k=0) == loss(k=1025) == loss(ldz=9) == gar.GAR_EINVAL
    assert loss(tau=0.0) == loss(tau=-1.0) == loss(tau=float("nan")) == loss(tau=float("inf")) == gar.GAR_EINVAL
    assert loss(z=NULL) == loss(i=NULL) == loss(t=NULL) == loss(loss=NULL) == loss(lse=NULL) == gar.GAR_EINVAL
    assert loss(dz=U, lddz=9) == loss(dz=A, lddz=12) == gar.GAR_EINVAL
    assert loss(dtype=3) == gar.GAR_EDTYPE
    assert loss(z=V(0x10002)) == loss(i=V(0x10001)) == loss(w=V(0x10002)) == loss(dz=V(0x10002), lddz=10) == gar.GAR_EALIGN
    assert loss(rows=0) == gar.GAR_OK

    def grad(lse=T, dz=U, lddz=10):
        return lib.gar_distill_grad(A, 0, 3, 10, 10, B, D, 2, 1.0, NULL, lse, dz, lddz, NULL)

    assert grad(lse=NULL) == grad(dz=NULL) == grad(lddz=9) == gar.GAR_EINVAL
    assert grad(lse=V(0x10001)) == gar.GAR_EALIGN


def test_balance_refusals(gar):
    lib = gar.load()
    two = (V * 2)(0x10000, 0x20000)

    def call(z=two, P=2, tokens=3, experts=8, ldz=8, dtype=0, k=2, valid=None, alpha=0.1, choice=two, counts=B, loss=D, dz=None,
             lddz=0, ws=S, nbytes=1 << 16):
        return lib.gar_balance_loss(z, P, tokens, experts, ldz, dtype, k, valid, alpha, choice, counts, loss, dz, lddz, ws, nbytes,
                                    NULL)

    assert call(P=0) == call(P=65) == call(tokens=-1) == call(tokens=1 << 40) == gar.GAR_EINVAL
    assert call(experts=0) == call(experts=1025) == call(k=0) == call(k=9) == call(experts=64, k=33, ldz=64) == gar.GAR_EINVAL
    assert call(alpha=float("nan")) == call(ldz=7) == call(dz=two, lddz=7) == gar.GAR_EINVAL
    assert call(z=None) == call(choice=None) == call(counts=NULL) == call(loss=NULL) == call(ws=NULL) == gar.GAR_EINVAL
    assert call(nbytes=8) == call(z=(V * 2)(0x10000, 0)) == call(valid=(V * 2)(0x10000, 0)) == gar.GAR_EINVAL
    assert call(dz=two, lddz=9) == gar.GAR_EINVAL  # in place with another stride
    assert call(dtype=4) == gar.GAR_EDTYPE
    assert call(counts=V(0x10002)) == call(z=(V * 2)(0x10000, 0x20002)) == call(ws=V(0x10004)) == gar.GAR_EALIGN


def test_sizes(gar):
    assert gar.gar_fp8_scale_bytes(3, 1) == 12 and gar.gar_fp8_scale_bytes(3, 512) == 12
    assert gar.gar_fp8_scale_bytes(3, 513) == 24 and gar.gar_fp8_scale_bytes(0, 5) == 0 and gar.gar_fp8_scale_bytes(-1, 5) == 0
    assert 0 < gar.gar_balance_workspace_bytes(8) <= 1 << 16 and gar.gar_balance_workspace_bytes(0) == 0


def test_binding_checks(gar):
    torch = pytest.importorskip("torch")
    q, s = gar.fp8_matrix(4, 100, device="cpu")
    r, t = gar.fp8_matrix(5, 100, torch.float8_e5m2, device="cpu")
    assert q.shape == (4, 100) and q.stride(0) == 112 and s.shape == (1, 4, 4)
    d = torch.zeros((4, 5))

    def status(f, *a, **k):
        with pytest.raises(gar.GarError) as e:
            f(*a, **k)
        return e.value.status

    x = torch.zeros((4, 100))
    assert status(gar.gar_fp8_quantize, x.double(), q, s) == gar.GAR_EDTYPE
    assert status(gar.gar_fp8_quantize, x, x, s) == gar.GAR_EDTYPE
    assert status(gar.gar_fp8_quantize, x.t(), q, s) == gar.GAR_EINVAL
    assert status(gar.gar_fp8_quantize, x, q, s) == gar.GAR_EINVAL  # not on a CUDA device
    assert status(gar.gar_fp8_matmul, q, s, r, t, d) == gar.GAR_EINVAL
    assert status(gar.gar_fp8_matmul, q, s, r, t, torch.zeros((5, 4))) == gar.GAR_EINVAL
    assert status(gar.gar_fp8_matmul, q, s, x, t, d) == gar.GAR_EDTYPE
    z, i, e, v = torch.zeros((3, 10)), torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2)), torch.zeros(3)
    assert status(gar.gar_distill_loss, z, i, e, 1.0, v, v) == gar.GAR_EINVAL
    assert status(gar.gar_distill_loss, z.half(), i, e, 1.0, v, v) == gar.GAR_EDTYPE
    c = torch.zeros((1, 10), dtype=torch.int32)
    w = torch.zeros(1 << 16, dtype=torch.uint8)
    assert status(gar.gar_balance_loss, [z], 2, 0.1, [i], c, v[:1], w) == gar.GAR_EINVAL
    assert status(gar.gar_balance_loss, [z.half()], 2, 0.1, [i], c, v[:1], w) == gar.GAR_EDTYPE


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_reference_grid_is_the_format(fmt):
    """The plain form's rounding against every code of the format, and midway between neighbours."""
    torch = pytest.importorskip("torch")
    t = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    v = torch.arange(256, dtype=torch.uint8).view(t).double().numpy()
    v = np.unique(v[np.isfinite(v)])
    np.testing.assert_array_equal(ref.round_to_format(v, fmt), v)
    mid = (v[1:] + v[:-1]) / 2
    got = ref.round_to_format(mid, fmt)
    assert all(g in (a, b) for g, a, b in zip(got, v[:-1], v[1:]))
    np.testing.assert_array_equal(got, torch.from_numpy(mid).to(t).double().numpy())
    near = np.nextafter(mid, np.inf)
    np.testing.assert_array_equal(ref.round_to_format(near, fmt), v[1:])


@pytest.fixture
def binding(gar, monkeypatch):
    """gar_balance_loss as it would be called with CUDA tensors, here with the host's: the library is not reached."""
    torch = pytest.importorskip("torch")
    calls = []

    class Cuda(torch.Tensor):
        is_cuda = True

    monkeypatch.setattr(gar, "_call", lambda name, *a: calls.append(name))
    monkeypatch.setattr(gar, "_stream", lambda stream: 0)

    def tensor(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype).as_subclass(Cuda)

    def call(z, choice, k=2, tokens=6, experts=8, table=False, **more):
        wrap = gar.pointer_table if table else list
        P = len(z)
        args = {n: None if v is None else wrap(v) for n, v in more.items()}
        gar.gar_balance_loss(wrap(z), k, 0.1, wrap(choice), tensor(P, experts, dtype=torch.int32), tensor(1), tensor(1 << 15),
                             **args)
        return calls.pop()

    def refused(*a, **more):
        with pytest.raises(gar.GarError) as e:
            call(*a, **more)
        assert not calls
        return e.value.status

    return torch, tensor, call, refused


@pytest.mark.parametrize("table", [False, True])
def test_every_workers_tensor_is_checked(gar, binding, table):
    torch, tensor, call, refused = binding
    i32 = torch.int32
    z, choice = [tensor(6, 8) for _ in range(3)], [tensor(6, 2, dtype=i32) for _ in range(3)]
    dz, valid = [tensor(6, 8) for _ in range(3)], [tensor(6, dtype=torch.uint8) for _ in range(3)]
    assert call(z, choice, table=table, dz=dz, valid=valid) == "gar_balance_loss"
    assert call(z, choice, table=table, valid=[v.bool() for v in valid]) == "gar_balance_loss"
    for bad in (tensor(5, 8), tensor(6, 7), tensor(6, 9)[:, :8], tensor(8, 6).t()):
        assert refused(z[:2] + [bad], choice, table=table) == gar.GAR_EINVAL
        assert refused(z, choice, table=table, dz=[dz[0], bad, dz[2]]) == gar.GAR_EINVAL
    assert refused(z[:2] + [tensor(6, 8, dtype=torch.bfloat16)], choice, table=table) == gar.GAR_EDTYPE
    assert refused(z, choice[:2] + [tensor(5, 2, dtype=i32)], table=table) == gar.GAR_EINVAL
    assert refused(z, choice[:2] + [tensor(6, 2, dtype=torch.int64)], table=table) == gar.GAR_EDTYPE
    assert refused(z, choice, table=table, valid=valid[:2] + [tensor(5, dtype=torch.uint8)]) == gar.GAR_EINVAL
    assert refused(z, choice, table=table, valid=valid[:2] + [tensor(6)]) == gar.GAR_EDTYPE
    assert refused(z, choice[:2], table=table) == gar.GAR_EINVAL


def test_a_table_is_looked_at_once_per_shape_and_type(gar, binding):
    torch, tensor, call, refused = binding
    z, choice = [tensor(6, 8) for _ in range(2)], [tensor(6, 2, dtype=torch.int32) for _ in range(2)]
    tz, tc = gar.pointer_table(z), gar.pointer_table(choice)
    more = (tensor(2, 8, dtype=torch.int32), tensor(1), tensor(1 << 15))
    for _ in range(2):
        gar.gar_balance_loss(tz, 2, 0.1, tc, *more, dz=tz)
    assert tz.checked == {((6, 8), torch.float32): (8, 1)} and tc.checked == {((6, 2), torch.int32): (2, 1)}
    with pytest.raises(gar.GarError):  # another number of choices is another shape
        gar.gar_balance_loss(tz, 3, 0.1, tc, *more, dz=tz)
    with pytest.raises(gar.GarError):
        gar.gar_balance_loss(tz, 2, 0.1, gar.pointer_table([choice[0], None], allow_none=True), *more)


@pytest.mark.parametrize("table", [False, True])
def test_one_token_of_strided_elements(gar, binding, table):
    """A single token's row stride may differ between workers, the stride of its elements may not."""
    torch, tensor, call, refused = binding
    z, choice = [tensor(1, 8) for _ in range(2)], [tensor(1, 2, dtype=torch.int32) for _ in range(2)]
    other = [z[0], tensor(1, 20)[:, 3:11]]
    assert call(other, choice, table=table, dz=other) == "gar_balance_loss"
    for place in (0, 1):
        bad = list(z)
        bad[place] = tensor(1, 16)[:, ::2]
        assert refused(bad, choice, table=table) == gar.GAR_EINVAL
        assert refused(z, choice, table=table, dz=bad) == gar.GAR_EINVAL
        bad = list(choice)
        bad[place] = tensor(1, 4, dtype=torch.int32)[:, ::2]
        assert refused(z, bad, table=table) == gar.GAR_EINVAL


def test_no_workers(gar, binding):
    torch, tensor, call, refused = binding
    assert refused([], []) == refused([], [], table=True) == refused([None], [None]) == gar.GAR_EINVAL
    z, choice = [tensor(6, 8) for _ in range(2)], [tensor(6, 2, dtype=torch.int32) for _ in range(2)]
    for bad in ([None, choice[1]], [choice[0], None]):
        assert refused(z, bad) == gar.GAR_EINVAL


@pytest.mark.parametrize("P", [1, 2, 8, 64])
def test_balance_token_limit(gar, P):
    """P tokens <= 2^26 - 1, also where their product does not fit 64 bits (2^63 and 2^64 at P = 64)."""
    lib = gar.load()
    table = (V * P)(*range(0x10000, 0x10000 * (P + 1), 0x10000))
    for tokens in (1 << 26, ((1 << 26) - 1) // P + 1, 1 << 40, 1 << 57, 1 << 58, 1 << 62, (1 << 63) - 1):
        status = lib.gar_balance_loss(table, P, tokens, 8, 8, 0, 2, None, 0.1, table, B, D, None, 0, V(0x10004), 1 << 16, NULL)
        assert status == gar.GAR_EINVAL, tokens  # (the workspace is misaligned: nothing is launched whatever the count)
    tokens = ((1 << 26) - 1) // P
    assert lib.gar_balance_loss(table, P, tokens, 8, 8, 0, 2, None, 0.1, table, B, D, None, 0, V(0x10004), 1 << 16,
                                NULL) == gar.GAR_EALIGN


@pytest.mark.parametrize("tau", [1e-45, 1e-39, 4e-39])
def test_distill_refuses_a_temperature_without_a_reciprocal(gar, tau):
    """log2(e) / tau would be infinite, and equal logits NaN."""
    lib = gar.load()
    odd = V(0x10002)  # misaligned, so that nothing is launched whatever the temperature
    args = (A, 0, 3, 10, 10, odd, D, 2)
    assert lib.gar_distill_loss(*args, tau, NULL, S, T, NULL, 0, NULL) == gar.GAR_EINVAL
    assert lib.gar_distill_grad(*args, tau, NULL, S, T, 10, NULL) == gar.GAR_EINVAL
    assert lib.gar_distill_loss(*args, 4.5e-39, NULL, S, T, NULL, 0, NULL) == gar.GAR_EALIGN
