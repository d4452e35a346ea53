"""Log probabilities straight from the head's inputs, and their gradients,
against binary64 (oracle/head.py) from the inputs' own values.

Tolerances count roundings: u = 2^-24 is half a step of binary32.  A logit is a
sum of `width` products (six parts each in fp32), so it is off by at most n u of
its magnitudes' sum; what follows moves by at most twice the row's worst such
error, relatively for a probability, and by S's own error (sum_error).
"""
import numpy as np
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from checkpoint_averaging_amd import dlmerge as dl
from oracle import head as oh
from tests import test_head_gpu as hg

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = hg.U


def inputs(rng, rows, vocab, width, lean=8.0):
    """Norm outputs that lean towards one token each by up to `lean` nats."""
    embed = (rng.standard_normal((vocab, width)) / np.sqrt(width)).astype(np.float32)
    peak = rng.integers(0, vocab, rows)
    x = rng.standard_normal((rows, width))
    x += lean * rng.random((rows, 1)) * embed[peak] / (embed[peak] ** 2).sum(1, keepdims=True)
    t = np.where(rng.random(rows) < 0.6, peak, rng.integers(0, vocab, rows))
    return x.astype(np.float32), embed, t


def framed(x, pad, dtype, fill=float("nan")):
    view, values, frame = hg.padded(np.asarray(x, np.float32), pad, dtype, fill)
    return view, values, frame


def workspace(rows, vocab, width, dtype, backward):
    need = dh.dl_head_workspace_bytes(rows, vocab, width, hg.TORCH[dtype], backward)
    return torch.full((max(need, 256),), 255, dtype=torch.uint8, device=DEV)


def logit_error(xv, ev, dtype):
    """Each row's worst error of a logit."""
    terms = xv.shape[1] * (6 if dtype == "f32" else 1) + 4
    mag = np.abs(xv.astype(np.float64)) @ np.abs(ev.astype(np.float64)).T
    return terms * U * mag.max(axis=1)


class Case:
    def __init__(self, x, embed, t, dtype, pad=0, b=None, a=None):
        self.dtype, self.rows, self.vocab, self.width = dtype, len(x), len(embed), x.shape[1]
        self.x, self.xv, _ = framed(x, pad, dtype)
        self.e, self.ev, _ = framed(embed, pad, dtype)
        self.t = np.asarray(t, np.int64)
        self.td = torch.from_numpy(self.t).to(DEV)
        z = self.xv.astype(np.float64) @ self.ev.astype(np.float64).T
        self.lp, self.h, self.m, self.log_s = oh.log_softmax(z)
        self.err = logit_error(self.xv, self.ev, dtype)
        self.a, self.b = a, b

    def forward(self, entropy=True):
        f = lambda *s: torch.full(s, 9.0, device=DEV)  # noqa: E731
        self.logprobs, self.stats = f(self.rows), f(self.rows, 2)
        self.entropy = f(self.rows) if entropy else None
        dh.dl_head_logprobs(self.x, self.e, self.rows, self.vocab, self.width, self.td,
                            self.logprobs, entropy=self.entropy, stats=self.stats,
                            workspace=workspace(self.rows, self.vocab, self.width, self.dtype,
                                                False))
        torch.cuda.synchronize()
        return self

    def tolerance(self):
        return 2 * self.err + hg.sum_error(self.vocab)

    def check_forward(self):
        rows, t = np.arange(self.rows), self.t
        want = np.where(t < 0, 0.0, self.lp[rows, np.clip(t, 0, self.vocab - 1)])
        want = np.where(t >= self.vocab, np.nan, want)
        tol = self.tolerance() + 4 * U * (np.abs(np.nan_to_num(want)) + np.abs(self.m))
        hg.within(hg.host(self.logprobs), want, tol, "logprobs")
        hg.within(hg.host(self.stats)[:, 0], self.m, self.err + U * np.abs(self.m), "m")
        hg.within(hg.host(self.stats)[:, 1], self.log_s, self.tolerance() + 2 * U * self.log_s,
                  "log S")
        if self.entropy is not None:
            # dH/dl = -p (log p + H), whose magnitudes sum to at most 2 H
            tol = 4 * self.tolerance() * (1 + np.log(self.vocab))
            hg.within(hg.host(self.entropy), self.h, tol, "entropy")
        return self

    def backward(self, pad=0, dx=True, de=True):
        def new(n):
            frame = torch.full((n, self.width + pad), 7.0, device=DEV).to(hg.TORCH[self.dtype])
            return frame, frame[:, :self.width]
        (self.fx, self.dx), (self.fe, self.de) = new(self.rows), new(self.vocab)
        dev = lambda v: None if v is None else torch.from_numpy(v.astype(np.float32)).to(DEV)  # noqa: E731
        self.ad, self.bd = dev(self.a), dev(self.b)
        dh.dl_head_logprobs_backward(
            self.x, self.e, self.rows, self.vocab, self.width, self.td, self.stats, self.ad,
            dx=self.dx if dx else None, dembed=self.de if de else None,
            entropy=self.entropy if self.b is not None else None, dentropy=self.bd,
            workspace=workspace(self.rows, self.vocab, self.width, self.dtype, True))
        torch.cuda.synchronize()
        for frame in (self.fx, self.fe):
            assert torch.all(frame[:, self.width:] == 7), "a gap between rows was written"
        return self

    def check_backward(self, dx=True, de=True):
        half = hg.HALF[self.dtype]
        act = (self.t >= 0) if self.b is None else np.ones(self.rows, bool)
        lp, h, t = self.lp[act], self.h[act], self.t[act]
        a = np.where(t < 0, 0, self.a[act].astype(np.float32).astype(np.float64))
        b = np.zeros(len(a)) if self.b is None else self.b[act].astype(np.float32).astype(np.float64)
        d = oh.logprobs_backward(lp, h, t, a, None if self.b is None else b)
        p, tol = np.exp(lp), self.tolerance()[act][:, None]
        eps = tol + 8 * U * (2 + np.abs(lp))
        off = p * eps * (np.abs(a)[:, None] + np.abs(b)[:, None] *
                         (np.abs(lp + h[:, None]) + 1 + 4 * (1 + np.log(self.vocab))))
        off = off + half * np.abs(d)
        xv, ev = self.xv[act].astype(np.float64), self.ev.astype(np.float64)
        terms = 6 if self.dtype == "f32" else 1
        if dx:
            want = np.zeros(self.xv.shape)
            want[act] = d @ ev
            tol = np.zeros(self.xv.shape)
            tol[act] = (off + (terms * self.vocab + 40) * U * np.abs(d)) @ np.abs(ev)
            hg.within(hg.host(self.dx), want, tol + half * np.abs(want) + 1e-38, "dx")
        if de:
            want = d.T @ xv
            tol = (off + (terms * len(a) + 40) * U * np.abs(d)).T @ np.abs(xv)
            hg.within(hg.host(self.de), want, tol + half * np.abs(want) + 1e-38, "dembed")
        return self


SHAPES = [(1, 1, 1), (1, 300, 64), (3, 5, 7), (12, 1000, 96), (16, 4099, 128), (17, 130, 200),
          (33, 1000, 130), (64, 513, 33), (100, 2500, 256), (257, 777, 65), (300, 4000, 72),
          (700, 300, 512)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,width", SHAPES)
def test_logprobs(rows, vocab, width, dtype):
    rng = np.random.default_rng(rows * 7 + vocab)
    x, e, t = inputs(rng, rows, vocab, width)
    t[::5] = -1
    Case(x, e, t, dtype).forward().check_forward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_logprobs_of_rows_apart(pad, dtype):
    rng = np.random.default_rng(pad)
    x, e, t = inputs(rng, 40, 900, 136)
    Case(x, e, t, dtype, pad).forward(entropy=False).check_forward()


@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_nearly_certain_token_keeps_its_digits(dtype, rows):
    """log p of some -1e-5 to -1e-16: relative to itself."""
    rng = np.random.default_rng(3)
    vocab, width = 700, 64
    e = (rng.standard_normal((vocab, width)) / 8).astype(np.float32)
    t = rng.integers(0, vocab, rows)
    x = (np.linspace(20, 40, rows)[:, None] * e[t] / (e[t] ** 2).sum(1, keepdims=True))
    c = Case(x, e, t, dtype).forward()
    want = c.lp[np.arange(rows), t]
    assert (want > -1e-4).all()
    hg.within(hg.host(c.logprobs), want, np.abs(want) * (c.tolerance() + 8 * U), "logprobs")
    hg.within(hg.host(c.entropy), c.h, np.abs(c.h) * (2 * c.tolerance() + 2.0 ** -20), "entropy")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [5, 100])
def test_targets_outside_and_rows_of_nan(rows, dtype):
    rng = np.random.default_rng(11)
    x, e, t = inputs(rng, rows, 600, 96)
    t[0], t[1], t[2] = 600, -5, 1 << 40
    x[4] = np.nan
    t[4] = 3
    c = Case(x, e, t, dtype)
    c.err = np.nan_to_num(c.err, nan=np.nanmax(c.err))
    c.forward()
    got = hg.host(c.logprobs)
    assert np.isnan(got[[0, 2, 4]]).all() and got[1] == 0
    assert np.isnan(hg.host(c.entropy)[4])
    keep = [i for i in range(rows) if i not in (0, 2, 4)]
    tol = c.tolerance() + 4 * U * (np.abs(np.nan_to_num(c.m)) + 30)
    want = np.where(t < 0, 0, c.lp[np.arange(rows), np.clip(t, 0, 599)])
    hg.within(got[keep], want[keep], tol[keep], "the other rows")


def test_without_optional_outputs():
    rng = np.random.default_rng(1)
    x, e, t = inputs(rng, 20, 500, 64)
    c = Case(x, e, t, "bf16").forward()
    ws = workspace(20, 500, 64, "bf16", False)
    only = torch.empty(20, 2, device=DEV)
    dh.dl_head_logprobs(c.x, c.e, 20, 500, 64, stats=only, workspace=ws)
    hg.same_bits(hg.bits(only), hg.bits(c.stats), "stats alone")
    h = torch.empty(20, device=DEV)
    dh.dl_head_logprobs(c.x, c.e, 20, 500, 64, entropy=h, workspace=ws)
    hg.same_bits(hg.bits(h), hg.bits(c.entropy), "entropy alone")
    dh.dl_head_logprobs(c.x, c.e, 0, 500, 64, stats=only, workspace=ws)


def weights(rng, rows, entropy):
    a = rng.standard_normal(rows)
    return a, (rng.standard_normal(rows) if entropy else None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("rows,vocab,width", SHAPES)
def test_gradients(rows, vocab, width, dtype, entropy):
    rng = np.random.default_rng(rows + vocab * 3)
    x, e, t = inputs(rng, rows, vocab, width)
    t[1::4] = -1
    a, b = weights(rng, rows, entropy)
    Case(x, e, t, dtype, 0, b, a).forward().backward().check_backward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 5, 8])
def test_gradients_of_rows_apart(pad, dtype):
    rng = np.random.default_rng(pad + 50)
    x, e, t = inputs(rng, 50, 900, 120)
    a, b = weights(rng, 50, True)
    c = Case(x, e, t, dtype, pad, b, a).forward()
    c.backward(pad).check_backward()
    c.backward(pad, dx=False).check_backward(dx=False)
    assert torch.all(c.fx == 7)
    c.backward(pad, de=False).check_backward(de=False)
    assert torch.all(c.fe == 7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_without_a_target_have_no_part(dtype):
    """Whatever they hold; none left at all gives zeros."""
    rng = np.random.default_rng(5)
    x, e, t = inputs(rng, 90, 400, 72)
    t[::3] = -1
    a, _ = weights(rng, 90, False)
    c = Case(x, e, t, dtype, 0, None, a).forward()
    c.x[::3] = float("nan")
    c.stats[::3] = float("nan")
    c.a = c.a.copy()
    c.a[::3] = np.nan
    c.backward()
    c.a[::3] = 0
    c.check_backward()
    c.td.fill_(-1)
    c.backward()
    assert not c.dx.any() and not c.de.any()


def test_no_rows_give_a_zero_gradient_of_the_embedding():
    e = torch.randn(300, 70, device=DEV)
    de = torch.full((300, 70), 3.0, device=DEV)
    none = torch.empty(0, device=DEV)
    x = torch.empty(0, 70, device=DEV)
    dh.dl_head_logprobs_backward(x, e, 0, 300, 70, none.long(), none, none, dx=x, dembed=de)
    torch.cuda.synchronize()
    assert not de.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_target_past_the_vocabulary_gives_nan(dtype):
    rng = np.random.default_rng(6)
    x, e, t = inputs(rng, 20, 300, 64)
    t[7] = 300
    a, _ = weights(rng, 20, False)
    c = Case(x, e, t, dtype, 0, None, a).forward().backward()
    got = hg.host(c.dx)
    assert np.isnan(got[7]).all() and not np.isnan(np.delete(got, 7, 0)).any()
    assert np.isnan(hg.host(c.de)).all()


def test_gradient_against_differences():
    """fp32; along the gradient's own direction, in binary64."""
    rng = np.random.default_rng(8)
    rows, vocab, width = 30, 500, 48
    x, e, t = inputs(rng, rows, vocab, width)
    t[::6] = -1
    a, b = weights(rng, rows, True)
    c = Case(x, e, t, "f32", 0, b, a).forward().backward()
    a, b = (v.astype(np.float32).astype(np.float64) for v in (a, b))

    def loss(x, e):
        lp, h, _, _ = oh.log_softmax(x @ e.T)
        own = np.where(t >= 0, lp[np.arange(rows), np.maximum(t, 0)], 0)
        return float((a * own).sum() + (b * h).sum())

    x0, e0 = c.xv.astype(np.float64), c.ev.astype(np.float64)
    gx, ge = hg.host(c.dx).astype(np.float64), hg.host(c.de).astype(np.float64)
    step = 1e-4 / max(np.abs(gx).max(), np.abs(ge).max())
    slope = (loss(x0 + step * gx, e0 + step * ge) - loss(x0 - step * gx, e0 - step * ge)) / (2 * step)
    # third-order terms of a step of 1e-4 an element, logits moving by up to some 1e-2: 1e-4
    assert abs(slope / ((gx ** 2).sum() + (ge ** 2).sum()) - 1) < 1e-3


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pieces_of_the_vocabulary(dtype):
    """Enough rows that the gradient takes the vocabulary in several pieces."""
    rng = np.random.default_rng(12)
    rows, vocab, width = (9000, 20_000, 32) if dtype == "bf16" else (5000, 20_000, 32)
    x, e, t = inputs(rng, rows, vocab, width)
    t[::2] = -1
    a, _ = weights(rng, rows, False)
    c = Case(x, e, t, dtype, 0, None, a).forward().check_forward()
    c.backward().check_backward()


def test_rows_far_apart():
    """Offsets past 2^31 and 2^32 elements into the embedding and its gradient."""
    rows, vocab, width, ld = 40, 600, 64, 8_000_000
    rng = np.random.default_rng(2)
    x, e, t = inputs(rng, rows, vocab, width)
    a, _ = weights(rng, rows, False)
    c = Case(x, e, t, "bf16", 0, None, a).forward().backward()
    far = torch.empty(vocab * ld, dtype=torch.bfloat16, device=DEV)
    ev = far.as_strided((vocab, width), (ld, 1))
    ev.copy_(c.e)
    lp = torch.empty(rows, device=DEV)
    dh.dl_head_logprobs(c.x, ev, rows, vocab, width, c.td, lp,
                        workspace=workspace(rows, vocab, width, "bf16", False))
    hg.same_bits(hg.bits(lp), hg.bits(c.logprobs), "logprobs")
    de = far.as_strided((vocab, width), (ld, 1), 1000)
    dx = torch.empty_like(c.x)
    dh.dl_head_logprobs_backward(c.x, c.e, rows, vocab, width, c.td, c.stats, c.ad, dx=dx,
                                 dembed=de, workspace=workspace(rows, vocab, width, "bf16", True))
    hg.same_bits(hg.bits(de.contiguous()), hg.bits(c.de), "dembed")
    hg.same_bits(hg.bits(dx), hg.bits(c.dx), "dx")


def test_calls_give_the_same_bits_and_graphs_replay_them():
    """A forward and backward pass captured once and replayed on new inputs, with eager
    calls and synchronisations between the replays."""
    rng = np.random.default_rng(9)
    rows, vocab, width = 300, 3000, 96
    x, e, t = inputs(rng, rows, vocab, width)
    t[::3] = -1
    a, b = weights(rng, rows, True)
    c = Case(x, e, t, "bf16", 0, b, a)
    ws = [workspace(rows, vocab, width, "bf16", True) for _ in range(2)]
    c.ad, c.bd = (torch.from_numpy(v.astype(np.float32)).to(DEV) for v in (a, b))

    def step(w):
        out = dict(lp=torch.empty(rows, device=DEV), h=torch.empty(rows, device=DEV),
                   st=torch.empty(rows, 2, device=DEV), dx=torch.empty_like(c.x),
                   de=torch.empty_like(c.e))
        dh.dl_head_logprobs(c.x, c.e, rows, vocab, width, c.td, out["lp"], entropy=out["h"],
                            stats=out["st"], workspace=w)
        dh.dl_head_logprobs_backward(c.x, c.e, rows, vocab, width, c.td, out["st"], c.ad,
                                     dx=out["dx"], dembed=out["de"], entropy=out["h"],
                                     dentropy=c.bd, workspace=w)
        return out

    step(ws[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = step(ws[0])
    for k in range(4):
        x2, e2, t2 = inputs(np.random.default_rng(100 + k), rows, vocab, width)
        c.x.copy_(torch.from_numpy(x2))
        c.e.copy_(torch.from_numpy(e2))
        c.td.copy_(torch.from_numpy(t2))
        g.replay()
        eager = step(ws[1])
        torch.cuda.synchronize()
        for name in kept:
            hg.same_bits(hg.bits(kept[name]), hg.bits(eager[name]), name)


def test_two_streams_at_once():
    rng = np.random.default_rng(10)
    sides = []
    for k in range(2):
        x, e, t = inputs(rng, 200 + 100 * k, 2000, 128)
        a, _ = weights(rng, 200 + 100 * k, False)
        sides.append(Case(x, e, t, "bf16", 0, None, a).forward().backward())
    streams = [torch.cuda.Stream() for _ in sides]
    for _ in range(4):
        got = []
        for c, s in zip(sides, streams):
            with torch.cuda.stream(s):
                ws = workspace(c.rows, c.vocab, c.width, "bf16", True)
                lp, st = torch.empty(c.rows, device=DEV), torch.empty(c.rows, 2, device=DEV)
                dx, de = torch.empty_like(c.x), torch.empty_like(c.e)
                dh.dl_head_logprobs(c.x, c.e, c.rows, c.vocab, c.width, c.td, lp, stats=st,
                                    workspace=ws)
                dh.dl_head_logprobs_backward(c.x, c.e, c.rows, c.vocab, c.width, c.td, st, c.ad,
                                             dx=dx, dembed=de, workspace=ws)
                got.append((lp, dx, de, ws))
        torch.cuda.synchronize()
        for c, (lp, dx, de, _) in zip(sides, got):
            assert torch.equal(lp, c.logprobs) and torch.equal(dx, c.dx) and torch.equal(de, c.de)


def test_refusals_on_the_device():
    x, e = torch.ones(4, 64, device=DEV), torch.ones(50, 64, device=DEV)
    st, t = torch.empty(4, 2, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    a = torch.ones(4, device=DEV)
    ws = workspace(4, 50, 64, "f32", True)

    def refused(fn, *args, **kw):
        with pytest.raises(dl.DLError) as ei:
            fn(*args, **kw)
        assert ei.value.status == dl.DL_E_INVAL

    refused(dh.dl_head_logprobs, x, e, 4, 50, 64, stats=st, workspace=ws, workspace_bytes=8)
    refused(dh.dl_head_logprobs, x.data_ptr(), 1 << 40, 4, 50, 64, stats=st, workspace=ws,
            dtype=dl.DL_F32)
    refused(dh.dl_head_logprobs, x, e, 4, 50, 64, stats=ws.view(torch.float32)[:8], workspace=ws)
    refused(dh.dl_head_logprobs_backward, x, e, 4, 50, 64, t, st, a, dx=x, workspace=ws)
    refused(dh.dl_head_logprobs_backward, x, e, 4, 50, 64, t, st, a, dembed=e, workspace=ws)
    with pytest.raises(TypeError):
        dh.dl_head_logprobs(x, e.bfloat16(), 4, 50, 64, stats=st, workspace=ws)
    with pytest.raises(ValueError):
        dh.dl_head_logprobs(x, e[:40], 4, 50, 64, stats=st, workspace=ws)
