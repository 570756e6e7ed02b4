"""Argument checks of gar_vocab_grad_with_loss and the binding's (no GPU needed,
no kernel launched)."""
import pytest

from test_more_ops_host import A, B, BIG, D, NULL, S, T, U, V, W, binding, gar  # noqa: F401


def test_refusals(gar):  # noqa: F811
    f = gar.load().gar_vocab_grad_with_loss

    def call(x=A, rows=5, loss=V(0x80000), lse=T, dx=S, dw=W, ws=U, n=BIG, dtype=1, dw_type=0, parts=0):
        return f(x, 64, B, 64, dtype, D, NULL, rows, 100, 50, loss, lse, dx, 50, NULL, 50, dw, 50, dw_type, parts, ws, n, NULL)

    assert call(loss=NULL) == call(lse=NULL) == call(x=NULL) == call(ws=NULL) == call(n=100) == call(dx=NULL, dw=NULL) == gar.GAR_EINVAL
    assert call(loss=V(0x80002)) == call(lse=V(0x10001)) == gar.GAR_EALIGN
    assert call(dtype=0) == gar.GAR_EDTYPE
    assert call(rows=0, loss=NULL, dw=NULL) == gar.GAR_OK
    assert call(parts=-1) == call(parts=3) == call(parts=1) == gar.GAR_EINVAL
    few = gar.load().gar_vocab_workspace_bytes(5, 100, 50, 1)
    assert few < gar.load().gar_vocab_workspace_bytes(5, 100, 50, 0)
    assert call(dw_type=1, parts=2, n=few) == gar.GAR_EINVAL and "workspace" in gar.gar_last_error()


def test_binding(gar, binding):  # noqa: F811
    torch, tensor, made, refused = binding
    x, w, target = tensor(6, 64, dtype=torch.bfloat16), tensor(30, 64, dtype=torch.bfloat16), tensor(6, dtype=torch.int32)
    lse, loss, ws, dw = tensor(6), tensor(6), tensor(4096, dtype=torch.uint8), tensor(30, 64)
    gar.gar_vocab_grad(x, w, target, lse, None, dw, ws)
    gar.gar_vocab_grad_with_loss(x, w, target, loss, lse, None, dw, ws)
    assert [n for n, _ in made] == ["gar_vocab_grad", "gar_vocab_grad_with_loss"]
    plain, given = made[0][1], made[1][1]
    assert given[:10] == plain[:10] and given[10] == loss.data_ptr() and given[11:19] == plain[10:18]
    assert given[19] == 0 and given[20:] == plain[18:]
    f = gar.gar_vocab_grad_with_loss
    f(x, w, target, loss, lse, None, dw, ws, parts=2)
    assert made[2][1][19] == 2
    assert refused(f, x, w, target, tensor(5), lse, None, dw, ws) == refused(f, x, w, target, loss, tensor(7), None, dw, ws) == gar.GAR_EINVAL
    assert refused(f, x, w, target, tensor(6, dtype=torch.bfloat16), lse, None, dw, ws) == gar.GAR_EDTYPE
