"""Gradients of log probabilities where the embedding's rows are of 128 bf16 numbers at
most, at the sizes and rows where that form can go wrong; against binary64, with the
tolerances of the general form (test_head_loss_gpu)."""
import numpy as np
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from checkpoint_averaging_amd import dlmerge as dl
from oracle import head as oh
from tests import test_head_gpu as hg
from tests import test_head_loss_gpu as lg

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("rows,vocab,width", [
    (2, 31, 8), (127, 33, 128), (128, 128, 128), (129, 257, 120), (255, 65, 16),
    (256, 256, 64), (257, 1025, 128), (513, 40, 104), (31, 5000, 128), (1500, 3001, 128)])
@pytest.mark.parametrize("entropy", [False, True])
def test_sizes_about_its_tiles(rows, vocab, width, entropy):
    rng = np.random.default_rng(rows + vocab)
    x, e, t = lg.inputs(rng, rows, vocab, width)
    t[:min(rows, 4)] = np.array([0, vocab - 1, vocab // 2, min(31, vocab - 1)])[:min(rows, 4)]
    a, b = lg.weights(rng, rows, entropy)
    lg.Case(x, e, t, "bf16", 0, b, a).forward().backward().check_backward()


@pytest.mark.parametrize("pad", [8, 24])
def test_rows_apart(pad):
    rng = np.random.default_rng(pad)
    x, e, t = lg.inputs(rng, 200, 700, 96)
    a, _ = lg.weights(rng, 200, False)
    c = lg.Case(x, e, t, "bf16", pad, None, a).forward()
    c.backward(pad).check_backward()
    c.backward(3, dx=False).check_backward(dx=False)
    c.backward(3, de=False).check_backward(de=False)


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("same", [False, True])
def test_certain_tokens_keep_their_digits(same, entropy):
    """Rows that give their targets nearly all: 1 - p is far below p's last place."""
    rng = np.random.default_rng(3)
    rows, vocab, width = 150, 300, 128
    x, e, _ = lg.inputs(rng, rows, vocab, width, lean=0.0)
    t = np.full(rows, 77) if same else rng.integers(0, vocab, rows)
    lean = np.linspace(2, 30, rows)[:, None]
    x = (0.1 * x + lean * e[t] / (e[t] ** 2).sum(1, keepdims=True)).astype(np.float32)
    a, b = lg.weights(rng, rows, entropy)
    c = lg.Case(x, e, t, "bf16", 0, b, a).forward().backward()
    p = np.exp(c.lp[np.arange(rows), t])
    assert (1 - p < 2.0 ** -12).sum() > 20 and (p < 0.9).sum() > 5
    c.check_backward()
    if entropy:
        return
    # one row at a time: relative to that row's own gradient, whose terms all have the size of
    # 1 - p; and a logit's own error moves log(1 - p) by as much
    for r in np.flatnonzero(1 - p < 2.0 ** -12)[::7]:
        d = oh.logprobs_backward(c.lp[r:r + 1], c.h[r:r + 1], t[r:r + 1], c.a[r:r + 1], None)
        mag = np.abs(d) @ np.abs(c.ev.astype(np.float64))
        off = 2 * hg.HALF["bf16"] + 4 * c.err[r] + 2 * hg.sum_error(vocab) + 64 * hg.U
        hg.within(hg.host(c.dx)[r:r + 1], d @ c.ev.astype(np.float64), off * mag + 1e-38, "dx")


@pytest.mark.parametrize("entropy", [False, True])
def test_logits_far_from_zero(entropy):
    """Logits of -300 and less, and of 300: the rows' largest are subtracted before anything
    is raised, also for what lies past the vocabulary's or the tokens' end."""
    rng = np.random.default_rng(8)
    rows, vocab, width = 100, 333, 72
    x, e, t = lg.inputs(rng, rows, vocab, width)
    x[:, 0] = 0
    x[::2, 0], x[1::2, 0] = 300, -300
    e[:, 0] = 1
    a, b = lg.weights(rng, rows, entropy)
    lg.Case(x, e, t, "bf16", 0, b, a).forward().backward().check_backward()


@pytest.mark.parametrize("entropy", [False, True])
def test_masked_tokens_have_no_gradient(entropy):
    """Logits of -infinity: an embedding's row that holds it, where x is positive."""
    rng = np.random.default_rng(9)
    x, e, t = lg.inputs(rng, 70, 200, 64)
    x[:, 5] = np.abs(x[:, 5]) + 0.01
    masked = np.arange(3, 200, 11)
    t = np.where(np.isin(t, masked), 0, t)
    a, b = lg.weights(rng, 70, entropy)
    plain = e.copy()
    e[masked, 5] = -np.inf
    with np.errstate(invalid="ignore"):
        c = lg.Case(x, e, t, "bf16", 0, b, a)
    c.forward().backward(dx=False)
    # p is 0 there, and the others' are those of a vocabulary without them
    keep = np.setdiff1d(np.arange(200), masked)
    at = np.searchsorted(keep, t)
    w = lg.Case(x, plain[keep], at, "bf16", 0, b, a)
    w.err = lg.logit_error(w.xv, w.ev, "bf16")
    w.de = c.de[torch.from_numpy(keep).to(DEV)]
    w.check_backward(dx=False)
    assert not c.de[torch.from_numpy(masked).to(DEV)].any()


def test_nan_stays_in_its_rows():
    rng = np.random.default_rng(10)
    x, e, t = lg.inputs(rng, 90, 400, 128)
    a, _ = lg.weights(rng, 90, False)
    good = lg.Case(x, e, t, "bf16", 0, None, a).forward().backward(de=False)
    x[40, 7] = np.nan
    with np.errstate(invalid="ignore"):
        c = lg.Case(x, e, t, "bf16", 0, None, a)
    c.forward().backward()
    assert torch.isnan(c.dx[40]).all() and torch.isnan(c.de).all()
    keep = torch.arange(90, device=DEV) != 40
    hg.same_bits(hg.bits(c.dx[keep].contiguous()), hg.bits(good.dx[keep].contiguous()), "dx")


def test_vocabulary_in_pieces():
    rng = np.random.default_rng(11)
    rows, vocab, width = 5, (1 << 18) + 300, 8
    x, e, t = lg.inputs(rng, rows, vocab, width)
    t[:3] = vocab - 1, (1 << 18) - 1, 1 << 18
    a, _ = lg.weights(rng, rows, False)
    lg.Case(x, e, t, "bf16", 0, None, a).forward().backward().check_backward()


def test_the_other_form_in_pieces():
    """The general form over several pieces of the vocabulary, in bf16."""
    rng = np.random.default_rng(12)
    rows, vocab, width = 9000, 16_000, 136
    x, e, t = lg.inputs(rng, rows, vocab, width)
    a, b = lg.weights(rng, rows, True)
    lg.Case(x, e, t, "bf16", 0, b, a).forward().backward().check_backward()


def test_both_forms_agree():
    """Rows apart by an odd distance take the general form: the same gradients, but for the
    roundings of each."""
    rng = np.random.default_rng(13)
    x, e, t = lg.inputs(rng, 300, 1200, 128)
    a, b = lg.weights(rng, 300, True)
    lg.Case(x, e, t, "bf16", 0, b, a).forward().backward().check_backward()
    lg.Case(x, e, t, "bf16", 1, b, a).forward().backward().check_backward()


@pytest.mark.parametrize("width", [72, 128])
def test_entropies_alone(width):
    """Rows without a target, and weights of zero for the targets, beside others."""
    rng = np.random.default_rng(width)
    x, e, t = lg.inputs(rng, 140, 900, width)
    a, b = lg.weights(rng, 140, True)
    t[::2] = -1
    a[1::4] = 0
    lg.Case(x, e, t, "bf16", 0, b, a).forward().backward().check_backward()


def test_graphs_replay_it_and_calls_repeat():
    rng = np.random.default_rng(14)
    rows, vocab, width = 300, 2000, 128
    x, e, t = lg.inputs(rng, rows, vocab, width)
    a, _ = lg.weights(rng, rows, False)
    c = lg.Case(x, e, t, "bf16", 0, None, a).forward().backward()
    ws = lg.workspace(rows, vocab, width, "bf16", True)
    dx, de = torch.empty_like(c.dx), torch.empty_like(c.de)
    st, lp = torch.empty_like(c.stats), torch.empty_like(c.logprobs)

    def step():
        dh.dl_head_logprobs(c.x, c.e, rows, vocab, width, c.td, lp, stats=st, workspace=ws)
        dh.dl_head_logprobs_backward(c.x, c.e, rows, vocab, width, c.td, st, c.ad, dx=dx,
                                     dembed=de, workspace=ws)

    step()
    torch.cuda.synchronize()
    hg.same_bits(hg.bits(dx), hg.bits(c.dx), "dx")
    hg.same_bits(hg.bits(de), hg.bits(c.de), "dembed")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(4):
        c.td.copy_(torch.from_numpy(rng.integers(0, vocab, rows)))
        c.td[:90 * k] = -1                                 # 300, 210, 120, 30 targets
        dx.fill_(9)
        de.fill_(9)
        g.replay()
        got = dx.clone(), de.clone()
        ws.fill_(255)
        step()
        torch.cuda.synchronize()
        hg.same_bits(hg.bits(got[0]), hg.bits(dx), f"dx {k}")
        hg.same_bits(hg.bits(got[1]), hg.bits(de), f"dembed {k}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,width", [(1100, 1500, 136), (1100, 1500, 64), (600, 300, 600)])
@pytest.mark.parametrize("some", [1, 40, 270])
def test_few_of_many_rows_have_a_target(rows, vocab, width, dtype, some):
    """The products are cut for the rows that take part, whatever their number."""
    rng = np.random.default_rng(some + width)
    x, e, t = lg.inputs(rng, rows, vocab, width)
    t[rng.permutation(rows)[some:]] = -1
    a, _ = lg.weights(rng, rows, False)
    lg.Case(x, e, t, dtype, 0, None, a).forward().backward().check_backward()


@pytest.mark.parametrize("dtype,width", [("bf16", 64), ("bf16", 264), ("f32", 136)])
def test_rows_4_mb_apart(dtype, width):
    """The embedding and its gradient in rows that go straight to LDS, at offsets past 2^32
    bytes; the inputs too, as far as the calls take them from there."""
    rows, vocab, size = 40, 1100, 4 if dtype == "f32" else 2
    ld = (1 << 22) // size
    rng = np.random.default_rng(width)
    x, e, t = lg.inputs(rng, rows, vocab, width)
    a, _ = lg.weights(rng, rows, False)
    c = lg.Case(x, e, t, dtype, 0, None, a).forward().backward()
    far = torch.empty((vocab + 1) * ld, dtype=hg.TORCH[dtype], device=DEV)
    ev = far.as_strided((vocab, width), (ld, 1))
    ev.copy_(c.e)
    de = far.as_strided((vocab, width), (ld, 1), 4096)
    lp, st, dx = torch.empty_like(c.logprobs), torch.empty_like(c.stats), torch.empty_like(c.dx)
    ws = lg.workspace(rows, vocab, width, dtype, True)
    dh.dl_head_logprobs(c.x, ev, rows, vocab, width, c.td, lp, stats=st, workspace=ws)
    # (dembed's rows lie between embed's: the call sees two spans that overlap, and refuses)
    with pytest.raises(dl.DLError):
        dh.dl_head_logprobs_backward(c.x, ev, rows, vocab, width, c.td, st, c.ad, dx=dx, dembed=de,
                                     workspace=ws)
    dh.dl_head_logprobs_backward(c.x, ev, rows, vocab, width, c.td, st, c.ad, dx=dx, workspace=ws)
    hg.same_bits(hg.bits(lp), hg.bits(c.logprobs), "logprobs")
    hg.same_bits(hg.bits(dx), hg.bits(c.dx), "dx")
    dh.dl_head_logprobs_backward(c.x, c.e, rows, vocab, width, c.td, st, c.ad, dembed=de,
                                 workspace=ws)
    hg.same_bits(hg.bits(de.contiguous()), hg.bits(c.de), "dembed")


@pytest.mark.parametrize("width", [64, 264])
def test_no_rows_at_all(width):
    e = torch.randn(700, width, device=DEV).bfloat16()
    de = torch.full((700, width), 3.0, dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, device=DEV)
    dh.dl_head_logprobs_backward(e[:0], e, 0, 700, width, torch.empty(0, dtype=torch.int64,
                                                                      device=DEV),
                                 none, none, dembed=de)
    torch.cuda.synchronize()
    assert not de.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("rows", [127, 128, 129])
def test_numbers_of_tokens_about_the_general_forms(rows, pad, dtype):
    rng = np.random.default_rng(rows)
    x, e, t = lg.inputs(rng, rows, 900, 200)
    t[::6] = -1
    a, b = lg.weights(rng, rows, True)
    c = lg.Case(x, e, t, dtype, pad, b, a).forward().check_forward()
    c.backward(pad).check_backward()
