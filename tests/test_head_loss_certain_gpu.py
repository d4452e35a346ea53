"""Gradients where a row gives one token nearly all: relative to that row's own gradient,
whose terms all have the size of 1 - p, whatever form the forward pass took its statistics
in; against binary64."""
import numpy as np
import pytest

from oracle import head as oh
from tests import test_head_gpu as hg
from tests import test_head_loss_gpu as lg

pytestmark = pytest.mark.gpu


def certain(rng, rows, vocab, width):
    """Rows whose largest logit is 3 to 28 above the others."""
    x, e, _ = lg.inputs(rng, rows, vocab, width, lean=0.0)
    t = rng.integers(0, vocab, rows)
    lean = np.linspace(6, 32, rows)[:, None]
    return (0.1 * x + lean * e[t] / (e[t] ** 2).sum(1, keepdims=True)).astype(np.float32), e, t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [5, 16, 20, 32, 33, 128, 150])
@pytest.mark.parametrize("width,entropy", [(128, False), (128, True), (96, False), (200, False),
                                           (200, True), (2048, True), (128, "both"),
                                           (256, "both")])
def test_each_row_keeps_its_digits(width, entropy, rows, dtype):
    rng = np.random.default_rng(rows + width)
    vocab = 300
    x, e, t = certain(rng, rows, vocab, width)
    a, b = lg.weights(rng, rows, entropy)
    if entropy is True:
        a = np.zeros(rows)
    c = lg.Case(x, e, t, dtype, 0, b, a).forward().backward()
    p = np.exp(c.lp[np.arange(rows), t])
    assert (1 - p < 2.0 ** -12).sum() >= rows // 2
    a, b = (None if v is None else v.astype(np.float32).astype(np.float64) for v in (c.a, c.b))
    d = oh.logprobs_backward(c.lp, c.h, t, a, b)
    # A logit's error moves the others' p, and log S and H with them, by twice it and S's own;
    # the largest one's log p is -log S.  Each term of d is a product of such.
    eps = 4 * c.tolerance()[:, None] + 16 * hg.U * (2 + np.abs(c.lp))
    mag = np.abs(oh.logprobs_backward(c.lp, c.h, t, a, None))
    off = mag * eps
    if entropy:
        own = np.abs(b)[:, None] * np.exp(c.lp) * (np.abs(c.lp) + c.h[:, None])
        # (H by itself: its terms' magnitudes are 2 H, and a step of 2^-20)
        off = off + own * (eps * (1 + np.log(vocab)) + 2.0 ** -19)
        mag = mag + own
        # Rows of 128 numbers at most: log2(p) lacks three roundings of m + log S, up to 3 u of
        # it; what of that is taken out of log p + H again has four roundings of its own (the
        # lack, its product, the sum with b H, and of both in the kernel).
        if dtype == "bf16" and width <= 128:
            size = np.abs(b) * (np.abs(c.m) + c.log_s)
            off = off + 12 * hg.U ** 2 * size[:, None] * np.exp(c.lp)
    # (both parts of d may be rounded before they are added)
    off = off + hg.HALF[dtype] * np.abs(d) + 4 * hg.U * mag
    terms = (6 if dtype == "f32" else 1) * max(vocab, rows) + 40
    for other, m, got, name in ((c.ev, d, c.dx, "dx"), (c.xv, d.T, c.de, "dembed")):
        other, o = np.abs(other.astype(np.float64)), off if name == "dx" else off.T
        want = m @ (c.ev if name == "dx" else c.xv).astype(np.float64)
        tol = (o + terms * hg.U * np.abs(m)) @ other + hg.HALF[dtype] * np.abs(want) + 1e-38
        hg.within(hg.host(got), want, tol, name)
