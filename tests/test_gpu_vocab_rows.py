"""dw in rows that start on 16 bytes and end inside 16: nothing is written past a row's
end, whatever lies there."""
import pytest

from helpers import need_cuda
from test_gpu_vocab import Problem, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return need_cuda()


@pytest.mark.parametrize("dw", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,hidden,pad", [(2, 30, 3, 1), (8, 273, 15, 1), (100, 700, 151, 1), (300, 520, 250, 6), (64, 257, 127, 1),
                                                   (9, 300, 129, 7), (5, 40, 1, 15)])
def test_rows_end_inside_16_bytes(env, rows, vocab, hidden, pad, dw):
    """The outputs' margins hold 7 and are looked at by `check`'s run, with every value."""
    torch, g = env
    check(torch, g, Problem(torch, rows, vocab, hidden, seed=40), torch.float32 if dw == "f32" else torch.bfloat16, pad=pad)
