"""Log probabilities, their gradients and the 8-bit head as they are used: over a
merge round's candidates, in training steps, captured into a graph, on several
streams.  Stages are checked against the oracle from the stage before, so that each
tolerance is its own."""
import numpy as np
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from checkpoint_averaging_amd import dlmerge as dl
from checkpoint_averaging_amd import synth
from checkpoint_averaging_amd.head import Head, LossHead
from oracle import head as oh
from tests import test_head_gpu as hg
from tests import test_head_loss_gpu as lg
from tests import test_head_path_gpu as hp

pytestmark = pytest.mark.gpu

DEV = "cuda"
WIDTH, VOCAB, LAYOUT = hp.WIDTH, hp.VOCAB, hp.LAYOUT


def f64(t):
    return hg.host(t).astype(np.float64)


def normed(s, weight, dtype):
    inv = oh.norm_inv(s, 1e-5).astype(np.float32)
    return oh.round_to(oh.norm_values(s, inv, weight), dtype).astype(np.float64)


@pytest.mark.parametrize("rows", [1, 32, 33, 300])
def test_candidates_of_a_round_score_without_logits(rows):
    """Both candidates' log probabilities agree with the head's that keeps its logits, to
    what the two products' roundings allow, and with binary64."""
    global_, ema = hp.merged()
    x, r, t = hp.stream(rows, rows)
    t[::5] = -1
    for flat in (global_, ema):
        loss, head = LossHead.of(LAYOUT, flat, 300), Head(LAYOUT, flat, 300)
        a, b = loss.score(x, r, t), head.score(x, r, t)
        # the same norm's output: both products are off by at most this much
        s = oh.round_to(hg.host(x) + hg.host(r), "bf16")
        h = normed(s, hg.host(head.weight), "f32")
        embed = f64(head.embed)
        # (and inv's last place moves h, hence the logits, by 6 u of their magnitudes)
        err = (6 * WIDTH + 16) * hg.U * (np.abs(h) @ np.abs(embed).T).max(axis=1)
        lp, H, m, log_s = oh.log_softmax(h @ embed.T)
        tn = t.cpu().numpy()
        want = np.where(tn < 0, 0.0, lp[np.arange(rows), np.clip(tn, 0, VOCAB - 1)])
        tol = 2 * err + hg.sum_error(VOCAB) + 4 * hg.U * (np.abs(want) + np.abs(m))
        hg.within(hg.host(a.logprobs), want, tol, "logprobs")
        hg.within(hg.host(a.logprobs), f64(b.logprobs), 2 * tol, "the head's with logits")
        tol = 4 * (2 * err + hg.sum_error(VOCAB)) * (1 + np.log(VOCAB))
        hg.within(hg.host(a.entropy), H, tol, "entropy")
        hg.within(hg.host(a.stats)[:, 0], m, err + hg.U * np.abs(m), "largest logit")
        assert loss.score(x, r).logprobs is None


@pytest.mark.parametrize("rows", [1, 32, 33, 100])
def test_head_published_in_8_bits(rows):
    global_, _ = hp.merged()
    x, r, t = hp.stream(rows, rows)
    s = oh.round_to(hg.host(x) + hg.host(r), "bf16")
    head = Head(LAYOUT, global_, max_rows=100)
    weight, embed = hg.host(head.weight), hg.host(head.embed)
    head.publish()
    head.publish(bits=8)
    a = head.answer(x, r, t, top_k=20)
    codes, e, values = oh.e4m3_quantize(embed, 128)
    hg.same_bits(head._codes.view(torch.uint8).cpu().numpy(), codes, "published codes")
    hg.same_bits(head._code_scales.cpu().numpy(), e, "published scales")
    xe = head._h8_scales128[:rows].cpu().numpy()
    h8 = oh.e4m3_value(head._h8[:rows].view(torch.uint8).cpu().numpy()) * oh.tile_spread(
        xe, (rows, WIDTH), 1)
    h = normed(s, weight, "f32")
    hg.within(h8, h, 2.0 ** -4 * np.abs(h) * 1.001 + 2.0 ** -10 * oh.tile_spread(xe, h.shape, 1),
              "norm in 8 bits")
    hg.within(hg.host(a.logits), h8.astype(np.float64) @ values.astype(np.float64).T,
              (WIDTH + 2) * hg.U * (np.abs(h8.astype(np.float64)) @
                                    np.abs(values.astype(np.float64)).T), "published logits")
    hp.check_answer(a, t, 20)
    head.publish()
    four = head.answer(x, r, t).logits.clone()
    head.publish(bits=8)
    assert not torch.equal(four, head.answer(x, r, t).logits)


def loss_of(s, weight, embed, t, a, b, w):
    """sum(a log p) + sum(b H) + sum(w s) in 64 bits, of the stream's sums s."""
    h = s / np.sqrt((s * s).mean(axis=1, keepdims=True) + 1e-5) * weight
    lp, H, _, _ = oh.log_softmax(h @ embed.T)
    on = t >= 0
    return ((a * lp[np.arange(len(t)), np.clip(t, 0, None)])[on].sum() + (b * H).sum() +
            (w * s).sum())


@pytest.mark.parametrize("rows", [40, 300])
@pytest.mark.parametrize("entropy", [False, True])
def test_training_step_against_differences(rows, entropy):
    """Norm, log probabilities and gradients of both; each derivative in a random direction
    is the difference quotient of the loss in 64 bits."""
    rng = np.random.default_rng(rows)
    weight = torch.from_numpy(1 + 0.1 * rng.standard_normal(WIDTH).astype(np.float32)).to(DEV)
    embed = torch.from_numpy(rng.standard_normal((VOCAB, WIDTH)).astype(np.float32) /
                             np.sqrt(WIDTH).astype(np.float32)).to(DEV)
    head = LossHead(weight, embed, 300)
    x, r, t = hp.stream(rows, 8, "f32")
    t[::7] = -1
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV)  # noqa: E731
    gl, gh, ds = f(rows), f(rows), f(rows, WIDTH)
    sm, dx = torch.empty_like(x), torch.full_like(x, 9.0)
    dembed, dweight = torch.full_like(embed, 9.0), torch.full_like(weight, 9.0)
    head.score(x, r, t, sum_=sm)
    head.backward(sm, t, gl, dx, dembed, dweight, dentropy=gh if entropy else None, dsum=ds)
    tn = t.cpu().numpy()
    s, w, e = f64(sm), f64(weight), f64(embed)
    args = (f64(gl), f64(gh) if entropy else np.zeros(rows), f64(ds))
    for k in range(3):
        d = [rng.standard_normal(v.shape) for v in (s, w, e)]
        step = 1e-6
        up = loss_of(s + step * d[0], w + step * d[1], e + step * d[2], tn, *args)
        down = loss_of(s - step * d[0], w - step * d[1], e - step * d[2], tn, *args)
        terms = [f64(g) * v for g, v in zip((dx, dweight, dembed), d)]
        got = sum(v.sum() for v in terms)
        # Differences: third derivatives are of the order of the gradients, so step^2 of
        # them is nothing; the loss's terms (a log probability is no more than 30 here), each
        # off by some 2^-53, over the step.  Gradients: sums of six parts a product over
        # VOCAB terms, whose magnitudes come to no more than 30 of the sum's, with errors u
        # in both directions: sqrt(6000) * 30 u = 1.4e-4 of an element, and elements' own
        # errors add up as the terms' root of squares.
        size = np.sqrt(sum((v * v).sum() for v in terms))
        loss = 30 * np.abs(args[0]).sum() + 7 * np.abs(args[1]).sum() + np.abs(args[2] * s).sum()
        assert abs(got - (up - down) / (2 * step)) <= 2e-4 * size + 8 * 2.0 ** -53 * loss / step, k


def test_training_in_bf16_against_64_bits():
    """The stages of a step in bf16: each against binary64 from the one before."""
    rng = np.random.default_rng(11)
    rows = 70
    weight = torch.from_numpy(1 + 0.1 * rng.standard_normal(WIDTH).astype(np.float32)).to(DEV)
    embed = torch.from_numpy(rng.standard_normal((VOCAB, WIDTH)) / np.sqrt(WIDTH)).to(DEV)
    head = LossHead(weight, embed.bfloat16(), 128)
    x, r, t = hp.stream(rows, 3)
    t[::7] = -1
    sm, dx = torch.empty_like(x), torch.full_like(x, 9.0)
    dembed = torch.full((VOCAB, WIDTH), 9.0, dtype=torch.bfloat16, device=DEV)
    dweight = torch.full((WIDTH,), 9.0, device=DEV)
    gl = torch.full((rows,), -1 / 60, device=DEV)
    a = head.score(x, r, t, sum_=sm)
    head.backward(sm, t, gl, dx, dembed, dweight)
    h, ev = f64(head._h[:rows]), f64(head.embed)
    want = normed(oh.round_to(hg.host(x) + hg.host(r), "bf16"), hg.host(weight), "bf16")
    # (inv's last place may turn a rounding over: a step of bf16)
    hg.within(hg.host(head._h[:rows]), want, 2.0 ** -7 * np.abs(want), "norm")
    c = lg.Case(hg.host(head._h[:rows]), hg.host(head.embed), t.cpu().numpy(), "bf16")
    assert np.array_equal(c.xv, hg.host(head._h[:rows]))
    c.logprobs, c.stats, c.entropy = a.logprobs, a.stats, a.entropy
    c.check_forward()
    # the gradients: a's dlogits in units of 1/60, rounded to 8 bits, products, and 8 bits again
    p = np.exp(c.lp)
    d = -p.copy()
    tn = t.cpu().numpy()
    d[np.arange(rows), np.clip(tn, 0, None)] += 1
    d = np.where((tn >= 0)[:, None], -d / 60, 0.0)
    off = 2.0 ** -8 * np.abs(d) + (2 * c.err + hg.sum_error(VOCAB))[:, None] * np.abs(d) * 2
    # (both terms of a target's 1 - p)
    off += (2 * c.err[:, None] + 4 * hg.U) * p / 60
    want, tol = d @ ev, off @ np.abs(ev) + VOCAB * hg.U * (np.abs(d) @ np.abs(ev))
    hg.within(hg.host(head._dh[:rows]), want, tol + 2.0 ** -8 * np.abs(want) + 2.0 ** -126, "dh")
    want, tol = d.T @ h, off.T @ np.abs(h) + rows * hg.U * (np.abs(d).T @ np.abs(h))
    hg.within(hg.host(dembed), want, tol + 2.0 ** -8 * np.abs(want) + 2.0 ** -126, "dembed")


def test_captured_step_replays():
    """A training step captured once and replayed on new inputs in the same buffers, with
    eager work and synchronisations in between, equals the eager step bit for bit; so does
    a captured answer in 8 bits.  Numbers of targets differ from replay to replay."""
    global_, _ = hp.merged()
    rows = 150
    loss, other = LossHead.of(LAYOUT, global_, 200), LossHead.of(LAYOUT, global_, 200)
    head, plain = Head(LAYOUT, global_, 200), Head(LAYOUT, global_, 200)
    head.publish(8)
    plain.publish(8)
    x, r, t = hp.stream(rows, 1, "f32")
    gl = torch.full((rows,), -0.05, device=DEV)

    def outs():
        return [torch.empty(rows, WIDTH, device=DEV), torch.empty(rows, WIDTH, device=DEV),
                torch.empty(VOCAB, WIDTH, device=DEV), torch.empty(WIDTH, device=DEV)]

    def step(on, o):
        a = on.score(x, r, t, sum_=o[0])
        on.backward(o[0], t, gl, o[1], o[2], o[3])
        return a

    mine, want = outs(), outs()
    step(loss, mine)
    head.answer(x, r, t)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = step(loss, mine)
        eight = head.answer(x, r, t)
    for k in range(4):
        x2, r2, t2 = hp.stream(rows, 50 + k, "f32")
        t2[:40 * k] = -1                                  # 150, 110, 70, 30 targets
        x.copy_(x2)
        r.copy_(r2)
        t.copy_(t2)
        gl.fill_(-0.01 * (k + 1))
        for v in mine:
            v.fill_(9.0)
        g.replay()
        b = step(other, want)
        c = plain.answer(x, r, t)
        torch.cuda.synchronize()
        for u, v, name in zip((*a, *mine, *eight[:3]), (*b, *want, *c[:3]),
                              ("logprobs", "entropy", "stats", "sum", "dx", "dembed", "dweight",
                               "8-bit logits", "8-bit logprobs", "8-bit entropy")):
            hg.same_bits(hg.bits(u), hg.bits(v), f"{name} {k}")


def test_heads_on_two_streams_at_once():
    global_, ema = hp.merged()
    heads = [LossHead.of(LAYOUT, f, 400) for f in (global_, ema)]
    x, r, t = hp.stream(400, 2, "f32")
    gl = torch.full((400,), 0.1, device=DEV)

    def step(h):
        o = [torch.empty(400, WIDTH, device=DEV), torch.empty(400, WIDTH, device=DEV),
             torch.empty(VOCAB, WIDTH, device=DEV), torch.empty(WIDTH, device=DEV)]
        a = h.score(x, r, t, sum_=o[0])
        h.backward(o[0], t, gl, o[1], o[2], o[3])
        return [*a, *o]

    want = [[v.clone() for v in step(h)] for h in heads]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in heads]
    for _ in range(5):
        got = []
        for h, s in zip(heads, streams):
            with torch.cuda.stream(s):
                got.append(step(h))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for u, v in zip(g, w):
                assert torch.equal(u, v)


def test_published_matrix_is_scored_before_it_is_served():
    """Quantise a candidate's embedding with its values, score the values without logits,
    and serve the codes: the served logits are the scored ones but for the tokens' own
    codes."""
    global_, _ = hp.merged()
    head = Head(LAYOUT, global_, 64)
    values = torch.empty_like(head.embed)
    codes = torch.empty(VOCAB, WIDTH, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty((VOCAB + 127) // 128, 1, dtype=torch.uint8, device=DEV)
    dh.dl_e4m3_quantize(head.embed, VOCAB, WIDTH, codes, scales, dh.DL_SCALE_TILE128, values=values)
    rng = np.random.default_rng(1)
    tokens = torch.from_numpy(hg.stream_values(rng, 64, WIDTH)).to(DEV)
    h8 = torch.empty(64, WIDTH, dtype=torch.float8_e4m3fn, device=DEV)
    hs, hv = torch.empty(64, 1, dtype=torch.uint8, device=DEV), torch.empty(64, WIDTH, device=DEV)
    dh.dl_e4m3_quantize(tokens, 64, WIDTH, h8, hs, dh.DL_SCALE_BLOCK128, values=hv)
    t = torch.arange(64, device=DEV)
    logits = torch.empty(64, VOCAB, device=DEV)
    dh.dl_e4m3_matmul(codes, scales, VOCAB, WIDTH, h8, hs, 64, logits)
    served, scored = torch.empty(64, device=DEV), torch.empty(64, device=DEV)
    dh.dl_logprobs(logits, 64, VOCAB, targets=t, logprobs=served)
    ws = torch.empty(dh.dl_head_workspace_bytes(64, VOCAB, WIDTH, torch.float32),
                     dtype=torch.uint8, device=DEV)
    dh.dl_head_logprobs(hv, values, 64, VOCAB, WIDTH, t, scored, workspace=ws)
    mag = (np.abs(f64(hv)) @ np.abs(f64(values)).T).max(axis=1)
    tol = 2 * (7 * WIDTH + 8) * hg.U * mag + 2 * hg.sum_error(VOCAB) + 8 * hg.U * np.abs(f64(scored))
    hg.within(hg.host(served), f64(scored), tol, "served against scored")
