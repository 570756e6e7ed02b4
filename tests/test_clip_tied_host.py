"""A tensor that stands in the gradients' lists more than once: its norm may be
taken, clipping it in place would scale it twice (no GPU needed)."""
from test_more_ops_host import binding, gar  # noqa: F401


def test_tied_tensors(gar, binding):  # noqa: F811
    torch, tensor, made, refused = binding
    same, ws, E = tensor(8), tensor(1 << 14), gar.GAR_EINVAL
    lists = [[same, tensor(3), same]]
    assert gar.gar_grad_workspace_bytes(lists) > 0
    gar.gar_grad_norm(lists, tensor(1), ws)
    tables = gar.grad_tables(lists, norm_only=True)
    gar.gar_grad_norm(tables, tensor(1), ws)
    assert [n for n, _ in made] == ["gar_grad_norm"] * 2
    assert refused(gar.gar_grad_clip, lists, 1.0, tensor(1), ws) == refused(gar.grad_tables, lists) == E
    assert refused(gar.gar_grad_clip, tables, 1.0, tensor(1), ws) == E
    assert refused(gar.grad_tables, lists, lists, norm_only=True) == refused(gar.grad_tables, tables, lists) == E
    gar.gar_grad_clip(lists, 1.0, tensor(1), ws, out=[[tensor(8), tensor(3), tensor(8)]])
    assert refused(gar.gar_grad_norm, [[same, tensor(4, 4)[:, ::2]]], tensor(1), ws) == E
