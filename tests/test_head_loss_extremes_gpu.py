"""Log probabilities without logits, and their gradients, where logits leave binary32's
range, and over a vocabulary of nearly the length that the call takes."""
import numpy as np
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from tests import test_head_gpu as hg
from tests import test_head_loss_gpu as lg

pytestmark = pytest.mark.gpu

DEV = "cuda"


def forward(x, e, t):
    rows, vocab, width = x.shape[0], e.shape[0], x.shape[1]
    lp, h, st = (torch.full(s, 9.0, device=DEV) for s in ((rows,), (rows,), (rows, 2)))
    need = dh.dl_head_workspace_bytes(rows, vocab, width, x.dtype)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    dh.dl_head_logprobs(x, e, rows, vocab, width, t, lp, entropy=h, stats=st, workspace=ws)
    torch.cuda.synchronize()
    return lp, h, st


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 16, 17, 32, 33, 200])
def test_a_logit_past_the_range_is_nan(rows, dtype):
    """A logit of +infinity from finite inputs: its row's results and gradients are NaN,
    the other rows' are not."""
    rng = np.random.default_rng(rows)
    vocab, width = 500, 40
    x, e, t = lg.inputs(rng, rows, vocab, width)
    x[:, 3], e[:, 3] = 0, 0
    bad = np.arange(0, rows, 5)
    x[bad, 3], e[77, 3] = 2.0 ** 100, 2.0 ** 100
    t[bad] = np.where(bad % 2 == 0, 77, 5)                       # the infinite one, or another
    xd, ed = (torch.from_numpy(v).to(DEV).to(hg.TORCH[dtype]) for v in (x, e))
    td = torch.from_numpy(t).to(DEV)
    lp, h, st = forward(xd, ed, td)
    got = [hg.host(lp), hg.host(h), hg.host(st)[:, 1]]
    for v, name in zip(got, ("logprobs", "entropy", "log S")):
        assert np.isnan(v[bad]).all(), name
        assert np.isfinite(np.delete(v, bad)).all(), name
    a = torch.ones(rows, device=DEV)
    dx = torch.empty_like(xd)
    ws = lg.workspace(rows, vocab, width, dtype, True)
    for b in (None, a):
        dh.dl_head_logprobs_backward(xd, ed, rows, vocab, width, td, st, a, dx=dx,
                                     entropy=None if b is None else h, dentropy=b, workspace=ws)
        got = hg.host(dx)
        assert np.isnan(got[bad]).all()
        # (2^100 is a finite element of every row's sum)
        assert np.isfinite(np.delete(got, bad, 0)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 20, 40])
def test_a_vocabulary_of_nothing_but_nan(rows, dtype):
    x = torch.full((rows, 8), float("nan"), device=DEV).to(hg.TORCH[dtype])
    for vocab in (1, 2):
        e = torch.ones(vocab, 8, device=DEV).to(hg.TORCH[dtype])
        lp, h, st = forward(x, e, torch.zeros(rows, dtype=torch.int64, device=DEV))
        assert torch.isnan(lp).all() and torch.isnan(h).all() and torch.isnan(st[:, 1]).all()


@pytest.mark.parametrize("rows", [1, 20, 33])
@pytest.mark.parametrize("vocab", [1 << 28, 1_036_800, 1_048_577])
def test_sums_over_a_long_vocabulary(vocab, rows):
    """Of up to 2^28 tokens the first are above all others and these are equal: their sum is
    off by no more than the 4e-5 that any vocabulary's may be, and so are log S and what it
    goes into.  (Equal terms below the largest round the same way at each addition.)"""
    tops, other = 1 << 16, -0.75
    e = torch.full((vocab, 1), other, dtype=torch.bfloat16, device=DEV)
    e[:tops] = 0
    x = torch.ones(rows, 1, dtype=torch.bfloat16, device=DEV)
    t = torch.full((rows,), 5, dtype=torch.int64, device=DEV)
    t[1::2] = vocab // 3
    lp, h, st = (hg.host(v).astype(np.float64) for v in forward(x, e, t))
    rest = (vocab - tops) * np.exp(other)
    log_s = np.log(tops + rest)
    # 2 u for the logarithm's last place, u for the subtraction
    off = 4e-5 + 3 * hg.U * log_s
    hg.within(st[:, 1], np.full(rows, log_s), off, "log S")
    want = np.where(np.arange(rows) % 2 == 0, 0.0, other) - log_s
    hg.within(lp, want, off, "logprobs")
    # the entropy's second term is the mean of the distances, whose sum has S's error too
    hg.within(h, np.full(rows, log_s - rest * other / (tops + rest)), 2 * off, "entropy")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 20, 40])
def test_the_widest_rows(rows, dtype):
    rng = np.random.default_rng(rows)
    x, e, t = lg.inputs(rng, rows, 300, dh.DL_MAX_NORM_COLS)
    t[1::5] = -1
    a, b = lg.weights(rng, rows, True)
    lg.Case(x, e, t, dtype, 0, b, a).forward().check_forward().backward().check_backward()


@pytest.mark.parametrize("dtype,width", [("bf16", 24), ("bf16", 136), ("f32", 24)])
@pytest.mark.parametrize("part", [0.01, 0.9])
def test_many_rows(part, width, dtype):
    """More rows than the products' slices and the gradients' walkers take at once, of which
    few or most have a target."""
    rng = np.random.default_rng(width)
    rows, vocab = 300_001, 70
    x, e, t = lg.inputs(rng, rows, vocab, width)
    t[rng.random(rows) > part] = -1
    a, _ = lg.weights(rng, rows, False)
    c = lg.Case(x, e, t, dtype, 0, None, a).forward().check_forward()
    c.backward().check_backward()
    assert not hg.host(c.dx)[t < 0].any()
