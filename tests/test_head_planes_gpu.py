"""The fp32 products of log probabilities without logits, and of their gradients: results
that are one product each are off by no more than a product of two binary32 numbers may be,
in each form of the product (few tokens; tiles of 128 and 256; operands along and across)."""
import numpy as np
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from tests import head_planes as hp
from tests import test_head_gpu as hg
from tests import test_head_loss_gpu as lg

pytestmark = pytest.mark.gpu

DEV = "cuda"


def dev(v):
    return torch.from_numpy(v).to(DEV)


def forward(x, e, t):
    rows, vocab, width = len(x), len(e), x.shape[1]
    lp, st = torch.empty(rows, device=DEV), torch.empty(rows, 2, device=DEV)
    dh.dl_head_logprobs(x, e, rows, vocab, width, t, lp, stats=st,
                        workspace=lg.workspace(rows, vocab, width, "f32", False))
    return st


@pytest.mark.parametrize("rows", [1, 16, 20, 32, 33, 128, 129, 300])
@pytest.mark.parametrize("vocab,width", [(1000, 200), (70, 39)])
def test_logits(vocab, width, rows):
    rng = np.random.default_rng(rows + width)
    x, e, (a, b) = hp.logits_of_one_product(rng, rows, vocab, width)
    st = forward(dev(x), dev(e), torch.zeros(rows, dtype=torch.int64, device=DEV))
    want = a.astype(np.float64) * b.astype(np.float64)
    hg.within(hg.host(st)[:, 0], want, hp.PRODUCT * np.abs(want), "largest logit")


def gradients(x, e, rng, t):
    rows, vocab, width = len(x), len(e), x.shape[1]
    x, e = dev(x), dev(e)
    t = torch.full((rows,), t, dtype=torch.int64, device=DEV)
    st = forward(x, e, t)
    a = hp.mantissas(rng, rows)
    dx, de = torch.empty_like(x), torch.empty_like(e)
    dh.dl_head_logprobs_backward(x, e, rows, vocab, width, t, st, dev(a), dx=dx, dembed=de,
                                 workspace=lg.workspace(rows, vocab, width, "f32", True))
    log_s = hg.host(st)[:, 1].astype(np.float64)
    assert not hg.host(st)[:, 0].any() and np.abs(log_s / np.log(vocab) - 1).max() < 1e-5
    return -a.astype(np.float64) * np.exp(-log_s), log_s, hg.host(dx), hg.host(de)


SHAPES = [(40, 1000, 200), (300, 1000, 130), (5, 400, 33)]


@pytest.mark.parametrize("rows,vocab,width", SHAPES)
def test_dx(rows, vocab, width):
    """Every logit 0, so that each token but the target (whose row is 0) has the gradient
    -a / vocab, and each element of dx is it times the one element of a column."""
    rng = np.random.default_rng(rows)
    e, at = hp.one_in_each_column(rng, vocab, width, first=1)
    d, log_s, dx, de = gradients(np.zeros((rows, width), np.float32), e, rng, 0)
    want = d[:, None] * e[at, np.arange(width)].astype(np.float64)
    hg.within(dx, want, hp.gradient_error(log_s)[:, None] * np.abs(want), "dx")
    assert not de.any()


@pytest.mark.parametrize("rows,vocab,width", SHAPES)
def test_dembed(rows, vocab, width):
    """The same of an embedding of zeros: each element of dembed is one row's gradient times
    the one element of x in a column."""
    rng = np.random.default_rng(rows + 1)
    x, at = hp.one_in_each_column(rng, rows, width)
    d, log_s, dx, de = gradients(x, np.zeros((vocab, width), np.float32), rng, 0)
    want = d[at] * x[at, np.arange(width)].astype(np.float64)
    tol = hp.gradient_error(log_s)[at] * np.abs(want)
    hg.within(de[1:], np.broadcast_to(want, (vocab - 1, width)), tol, "dembed")
    assert not dx.any()
