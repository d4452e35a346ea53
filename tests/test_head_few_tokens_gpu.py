"""Calls of a few tokens over long matrices, as decoding makes them: several turns of rows
with every wave's columns in use, vectors that are loaded again for each chunk of columns,
and each number of row and vector tiles; against binary64.  And layouts in 8 bits of more
tiles than the grid has workgroups."""
import numpy as np
import pytest
import torch

from oracle import head as oh
from tests import test_e4m3_gpu as eg
from tests import test_head_gpu as hg
from tests import test_head_loss_gpu as lg

pytestmark = pytest.mark.gpu

COUNTS = [1, 16, 17, 32]


@pytest.mark.parametrize("rows,cols", [(20_000, 2048), (9000, 5632), (30_011, 2041), (5000, 2304)])
def test_products_in_8_bits(rows, cols):
    rng = np.random.default_rng(rows)
    w, ws, wv = eg.operand(rng, rows, cols, eg.TILE)
    for count in COUNTS:
        x, xs, xv = eg.operand(rng, count, cols, eg.BLOCK)
        for out in ("f32", "bf16"):
            eg.check_product(eg.product(w, ws, x, xs, out), wv, xv, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [2048, 2047, 2304, 4500])
def test_log_probabilities(width, dtype):
    rng = np.random.default_rng(width)
    vocab = 20_000 if width < 4000 else 9000
    x, e, t = lg.inputs(rng, 32, vocab, width)
    t[5::7] = -1
    # (the last rows of the vocabulary, too, are some tokens' targets)
    t[:3] = [vocab - 1, vocab - 2, 0]
    for count in COUNTS:
        lg.Case(x[:count], e, t[:count], dtype).forward().check_forward()


def test_layout_of_more_tiles_than_workgroups():
    """16,407 tiles for 16,384 workgroups, neighbours and those 16,384 apart of different
    magnitude."""
    rng = np.random.default_rng(6)
    rows, cols = 2, 2_100_000
    size = np.repeat(np.exp2(rng.integers(-20, 20, cols // 128 + 1)), 128)[:cols]
    x = (rng.standard_normal((rows, cols)) * size).astype(np.float32)
    eg.check_quantize(x, eg.TILE)
    eg.check_quantize(x, eg.TILE, "bf16")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,count", [(64, 4), (64, 20), (64, 40), (6000, 1200)])
def test_scales_at_the_ends_of_the_range(rows, count, out):
    """Elements of 448 2^119 and of 2^-133, the largest and the smallest that block scales in
    bf16 hold, are exact in every form: one product each, whole in bf16."""
    for code, byte, other in ((0x7E, 246, 27), (0x01, 3, 227), (0x7E, 0, 247)):
        w, x = (np.zeros((n, 128), np.uint8) for n in (rows, count))
        w[:, 7], x[:, 7] = code, 0x38                            # 0x38: 1
        ws = torch.full((eg.groups(eg.TILE, rows), 1), byte, dtype=torch.uint8, device=eg.DEV)
        xs = torch.full((count, 1), other, dtype=torch.uint8, device=eg.DEV)
        dev = lambda v: torch.from_numpy(v).to(eg.DEV).view(torch.float8_e4m3fn)  # noqa: E731
        want = oh.e4m3_value(np.array([code], np.uint8))[0] * 2.0 ** (byte - 127 + other - 127)
        hg.same_bits(eg.product(dev(w), ws, dev(x), xs, out), np.full((count, rows), want), out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_a_short_matrix_times_many_vectors(out):
    rng = np.random.default_rng(7)
    w, ws, wv = eg.operand(rng, 70, 136, eg.TILE)
    x, xs, xv = eg.operand(rng, 200_003, 136, eg.BLOCK)
    eg.check_product(eg.product(w, ws, x, xs, out), wv, xv, out)
