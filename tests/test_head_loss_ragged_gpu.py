"""Log probabilities without logits, and their gradients, where rows end inside 16 bytes of
memory but begin at multiples of them: what lies between a row's end and the next one's
beginning, NaN here, takes no part, and the embedding's last element is its allocation's."""
import numpy as np
import pytest
import torch

from tests import test_head_gpu as hg
from tests import test_head_loss_gpu as lg

pytestmark = pytest.mark.gpu


def ending(view):
    """The same rows where nothing follows the last one."""
    rows, cols = view.shape
    ld = view.stride(0)
    flat = torch.full(((rows - 1) * ld + cols,), float("nan"), device=lg.DEV).to(view.dtype)
    out = flat.as_strided((rows, cols), (ld, 1))
    out.copy_(view)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,width,pad", [
    (1, 90, 131, 5), (20, 300, 129, 7), (40, 700, 130, 6), (130, 515, 300, 4), (300, 1000, 135, 1),
    (257, 258, 513, 7), (300, 130, 100, 4), (50, 8, 150, 2), (50, 9, 150, 2), (600, 7, 140, 4)])
def test_rows_that_end_inside_a_piece(rows, vocab, width, pad, dtype):
    rng = np.random.default_rng(rows + width)
    x, e, t = lg.inputs(rng, rows, vocab, width)
    t[::5] = -1
    a, b = lg.weights(rng, rows, True)
    c = lg.Case(x, e, t, dtype, pad, b, a)
    c.x, c.e = ending(c.x), ending(c.e)
    c.forward().check_forward().backward(pad).check_backward()
    c.backward(pad, dx=False).check_backward(dx=False)
    c.backward(pad, de=False).check_backward(de=False)


def test_pieces_whose_rows_end_inside_16_bytes():
    """The vocabulary in two pieces, the last row of all in the second one."""
    rng = np.random.default_rng(4)
    rows, vocab, width = 17_000, 4400, 130
    x, e, t = lg.inputs(rng, rows, vocab, width)
    t[rng.random(rows) < 0.8] = -1
    a, _ = lg.weights(rng, rows, False)
    c = lg.Case(x, e, t, "bf16", 6, None, a)
    c.x, c.e = ending(c.x), ending(c.e)
    c.forward().backward(6).check_backward()
    assert not hg.host(c.dx)[t < 0].any()
