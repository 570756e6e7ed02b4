"""The norm of lists in which a tensor stands twice."""
import pytest

from helpers import need_cuda

pytestmark = pytest.mark.gpu


def test_a_tied_tensor_counts_twice():
    """fp64 sums of sixteen fp32 squares each: 16 u of the square, half of that and u of the norm (u = 2^-24)."""
    torch, g = need_cuda()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    a, b = torch.randn(5001, generator=gen, device="cuda"), torch.randn(300, generator=gen, device="cuda").bfloat16()
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(g.gar_grad_workspace_bytes([[a, b, a]]), dtype=torch.uint8, device="cuda")
    g.gar_grad_norm([[a, b, a]], norm, ws)
    want = (2 * a.double().square().sum() + b.double().square().sum()).sqrt().item()
    assert abs(norm.item() - want) <= 9 * 2.0 ** -24 * want
