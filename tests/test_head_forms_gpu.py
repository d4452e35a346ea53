"""The output head where the other tests' sizes do not reach: past each
variant's threshold, several turns of a workgroup, and a Head's calls mixed
with captured ones.  Tolerances are those derived in test_head_gpu."""
import numpy as np
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from checkpoint_averaging_amd import dlmerge as dl
from checkpoint_averaging_amd.head import Head
from oracle import head as oh
from tests import test_head_gpu as hg
from tests import test_head_path_gpu as hp

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_captured_score_replays_after_larger_eager_ones():
    """A score of few rows captured, then eager ones of more (the product needs
    more workspace for these) and tensors that fill what may have been freed:
    the replay gives the eager bits and touches nothing else."""
    global_, _ = hp.merged()
    head, other = Head(hp.LAYOUT, global_, 600), Head(hp.LAYOUT, global_, 20)
    needs = [dl.dl_matmul_workspace_bytes(r, hp.VOCAB, hp.WIDTH) for r in (20, 600)]
    assert needs[0] < needs[1]
    x, r, t = hp.stream(20, 1)
    head.score(x, r, t, top_k=3)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = head.score(x, r, t, top_k=3)
        logits, lps = a.logits.clone(), a.logprobs.clone()
    at = head._product_ws.data_ptr()
    for k in range(4):
        xb, rb, tb = hp.stream(600, 70 + k)
        head.score(xb, rb, tb)
        assert head._product_ws.data_ptr() == at
        others = [torch.full((n,), 7.0, device=DEV) for n in (needs[0] // 4, needs[1] // 4)]
        x2, r2, t2 = hp.stream(20, 50 + k)
        x.copy_(x2)
        r.copy_(r2)
        t.copy_(t2)
        torch.cuda.synchronize()
        g.replay()
        b = other.score(x2, r2, t2, top_k=3)
        torch.cuda.synchronize()
        hg.same_bits(hg.bits(logits), hg.bits(b.logits), "logits")
        hg.same_bits(hg.bits(lps), hg.bits(b.logprobs), "logprobs")
        assert all(bool((o == 7.0).all()) for o in others)


# --------------------------------------------------------------------------
# Norm
# --------------------------------------------------------------------------


@pytest.mark.parametrize("out,kind", hg.OUTS, ids=["f32", "bf16", "e4m3_row", "e4m3_block"])
@pytest.mark.parametrize("rows,cols", [(300, 200), (300, 400), (300, 600), (300, 1000),
                                       (300, 1700), (256, 1000), (257, 2047)])
def test_norm_lanes_and_groups(rows, cols, out, kind):
    """Each number of lanes and groups a row, and both sides of 256 rows."""
    rng = np.random.default_rng([rows, cols, 31])
    x, res = hg.stream_values(rng, rows, cols), hg.stream_values(rng, rows, cols)
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    hg.check_norm(x, res, w, "bf16", out, kind, pad=1)
    hg.check_norm(x, None, w, "f32", out, kind)


@pytest.mark.parametrize("dtype,out,kind", [("bf16", "e4m3", dh.DL_SCALE_BLOCK32),
                                            ("f32", "e4m3", dh.DL_SCALE_ROW),
                                            ("f32", "bf16", dh.DL_SCALE_NONE)])
@pytest.mark.parametrize("rows,cols", [(33_000, 130), (8_300, 513), (2_051, 2_049),
                                       (2_050, 8_193)])
def test_norm_several_turns_of_a_workgroup(rows, cols, dtype, out, kind):
    """More rows than the 2048 workgroups take at once, for 16, 64, 256 and 1024
    lanes a row: what the turns share (sums in LDS, the weight) is used again."""
    rng = np.random.default_rng([rows, cols, 32])
    x, res = hg.stream_values(rng, rows, cols), hg.stream_values(rng, rows, cols)
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    hg.check_norm(x, res, w, dtype, out, kind)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(600, 2050), (530, 8200), (1030, 4100), (514, 16_400)])
def test_norm_backward_several_turns_of_1024_lanes(rows, cols, dtype):
    """More rows than the 512 workgroups of the widest form."""
    hg.check_backward(rows, cols, dtype)


@pytest.mark.parametrize("inplace", ["dy", "dsum"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [8_193, 20_001, 32_768])
def test_norm_backward_in_place_where_the_row_is_read_again(cols, dtype, inplace):
    hg.check_backward(5, cols, dtype, inplace=inplace, pad=1)
    hg.check_backward(520, cols, dtype, inplace=inplace)


# --------------------------------------------------------------------------
# 4-bit product, from 8192 rows on (two tiles of rows a wave) and where a
# workgroup passes over several groups of rows
# --------------------------------------------------------------------------

KIND_IDS = ["bf16", "e4m3_row", "e4m3_block"]


def whole_vectors(rng, count, cols):
    x = rng.integers(-7, 8, (count, cols)).astype(np.float32)
    x[:, ::32] = 7
    return x


@pytest.mark.parametrize("kind", hg.KINDS, ids=KIND_IDS)
@pytest.mark.parametrize("count", [1, 12, 16, 17, 32])
@pytest.mark.parametrize("rows,cols", [(8_192, 32), (8_209, 200)])
def test_matvec_of_many_rows(rows, cols, count, kind):
    rng = np.random.default_rng([rows, cols, count, 33])
    packed, scales = hg.random_w4(rng, rows, cols)
    x = rng.standard_normal((count, cols)).astype(np.float32)
    hg.check_matvec(packed, scales, rows, cols, x, kind, "f32", pad_y=1)
    hg.check_matvec(packed, scales, rows, cols, x, kind, "bf16", pad_x=1, pad_y=3)


@pytest.mark.parametrize("kind", hg.KINDS, ids=KIND_IDS)
@pytest.mark.parametrize("rows,cols,count", [
    (8_191, 2_100, 12), (8_200, 2_100, 12), (8_200, 2_100, 32),     # several chunks of columns
    (16_500, 1_600, 5), (16_500, 1_600, 20),                        # eight waves share the columns
    (66_001, 100, 3), (33_003, 100, 19), (33_003, 500, 32),         # two; four
    (4_500, 1_600, 20)])                                            # one row tile, 17 to 32 vectors
def test_matvec_of_whole_numbers_with_many_scales_is_exact(rows, cols, count, kind):
    """Scales of a half to four, whole numbers up to 7: partial sums are multiples
    of 1/4 below 7 * 24 * 2100 < 2^19, so they fit binary32 in any order, and a
    code, scale byte or vector taken from another row, block, turn or chunk shows.
    (Row scales are 2^-6: sums of multiples of 16 below 2^25.)"""
    rng = np.random.default_rng([rows, cols, count, 34])
    packed, scales = hg.random_w4(rng, rows, cols, 126, 130)
    hg.check_matvec(packed, scales, rows, cols, whole_vectors(rng, count, cols), kind, "f32",
                    exact=True)


@pytest.mark.parametrize("kind", hg.KINDS, ids=KIND_IDS)
@pytest.mark.parametrize("count", [1, 12, 32])
def test_matvec_of_the_embedding_with_many_scales(count, kind):
    """73,760 x 2048 against binary64 on the device; exact as above."""
    rows, cols = 73_760, 2_048
    rng = np.random.default_rng([count, 35])
    packed, scales = hg.random_w4(rng, rows, cols, 126, 130)
    x = whole_vectors(rng, count, cols)
    pt, st = torch.from_numpy(packed).to(DEV), torch.from_numpy(scales).to(DEV)
    if kind == dh.DL_SCALE_NONE:
        xt, xs = torch.from_numpy(x).to(DEV).bfloat16(), None
    else:
        xt, xs, _, _ = hg.e4m3_vectors(x, kind)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV, dtype=torch.float64)
    table = torch.cat([table, -table])
    x64 = torch.from_numpy(x.T.copy()).to(DEV).double()
    for out in ("f32", "bf16"):
        y = torch.full((count, rows), 7.0, device=DEV).to(hg.TORCH[out])
        dh.dl_w4_matvec(pt, st, rows, cols, xt, count, y, x_scales=xs, x_scale_kind=kind)
        for r0 in range(0, rows, 8_000):
            p, e = pt[r0:r0 + 8_000], st[r0:r0 + 8_000]
            codes = torch.stack([p & 15, p >> 4], 2).reshape(p.shape[0], -1).long()
            w = table[codes] * torch.exp2(e.double() - 127).repeat_interleave(32, 1)
            want = (w @ x64).t().float().to(hg.TORCH[out])
            assert torch.equal(y[:, r0:r0 + 8_000], want), (out, r0)


@pytest.mark.parametrize("kind", hg.KINDS[1:], ids=KIND_IDS[1:])
@pytest.mark.parametrize("power", [-80, 100])
def test_matvec_of_vectors_with_far_scales(kind, power):
    """Vectors in 8 bits of 2^-80 and 2^100 times whole numbers: exact."""
    rng = np.random.default_rng([power + 200, 36])
    packed, scales = hg.random_w4(rng, 100, 300, 126, 130)
    x = whole_vectors(rng, 3, 300) * np.float32(2.0 ** power)
    hg.check_matvec(packed, scales, 100, 300, x, kind, "f32", exact=True)


def test_matvec_of_many_rows_touches_only_what_a_special_value_belongs_to():
    rng = np.random.default_rng(37)
    rows, cols = 8_300, 300
    packed, scales = hg.random_w4(rng, rows, cols)
    scales[0], scales[8_299, 9], scales[4_000, 3] = 0, 255, 255
    x = rng.integers(-7, 8, (20, cols)).astype(np.float32)
    x[3, 17], x[18, 299], x[1] = np.inf, np.nan, 0
    hg.check_matvec(packed, scales, rows, cols, x, dh.DL_SCALE_NONE, "f32")


# --------------------------------------------------------------------------
# Log probabilities
# --------------------------------------------------------------------------


def logits_of(rows, vocab, dtype, seed, pad):
    """Logits on the device in rows of vocab + pad, with rows that a mask leaves
    one token or nothing, nearly certain ones, and a NaN and an infinity."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    frame = torch.full((rows, vocab + pad), float("nan"), device=DEV, dtype=hg.TORCH[dtype])
    x = frame[:, :vocab]
    for r in range(0, rows, 512):
        part = 2.5 * torch.randn(min(512, rows - r), vocab, generator=g, device=DEV) - 4
        x[r:r + 512] = part.to(x.dtype)
    x[1, 1:] = float("-inf")
    x[2] = float("-inf")
    x[3] = torch.finfo(x.dtype).min
    x[4, vocab - 1] = 60
    x[5, ::2] = float("-inf")
    x[6, vocab // 2] = float("nan")
    x[7, vocab - 2] = float("inf")
    x[rows - 1, 0] = 40
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,pad", [(50_277, 3), (8_193, 0), (2_048, 1)])
def test_logprobs_of_more_than_the_caches_hold(vocab, pad, dtype):
    """At least 192 MB of logits without alternatives, which are read past the
    caches, and their gradient, against binary64 on the device."""
    rows = (192 << 20) // (vocab * hg.TORCH[dtype].itemsize) + 3
    x = logits_of(rows, vocab, dtype, 41, pad)
    g = torch.Generator(device=DEV).manual_seed(42)
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    t[4], t[5], t[8], t[9], t[rows - 1] = vocab - 1, 1, -1, vocab, 0
    lp, h = torch.full((rows,), 9.0, device=DEV), torch.full((rows,), 9.0, device=DEV)
    st = torch.full((rows, 2), 9.0, device=DEV)
    dh.dl_logprobs(x, rows, vocab, t, lp, h, st)
    gl = torch.randn(rows, generator=g, device=DEV)
    d = torch.full((rows, vocab + pad), 7.0, device=DEV, dtype=x.dtype)
    dh.dl_logprobs_backward(x, rows, vocab, t, st, gl, d[:, :vocab])
    torch.cuda.synchronize()
    if pad:
        assert bool((d[:, vocab:] == 7.0).all())
    step = max(8, (1 << 24) // vocab)
    for r in range(0, rows, step):
        check_logprobs_rows(x[r:r + step], t[r:r + step], lp[r:r + step], h[r:r + step],
                            st[r:r + step], gl[r:r + step], d[r:r + step, :vocab], dtype)


def check_logprobs_rows(x, t, lp, h, st, gl, d, dtype):
    """As check_logprobs and check_logprobs_backward of test_head_gpu."""
    rows, vocab = x.shape
    u, es = hg.U, hg.sum_error(vocab)
    bad = x.isnan().any(1) | (x == float("inf")).any(1)
    none = (x == float("-inf")).all(1)
    v = torch.where((bad | none)[:, None], 0.0, x.double())
    m, at = v.max(1)
    dist = v - m[:, None]
    e = dist.exp()
    log_s = torch.log1p(e.scatter(1, at[:, None], 0.0).sum(1))
    want_lp = dist - log_s[:, None]
    p = want_lp.exp()
    f = torch.where(p > 0, want_lp, 0.0)
    want_h = -(p * f).sum(1)
    d_log = es * log_s.expm1().clamp(max=1) + 3 * u * log_s + vocab * 2.0 ** -126

    def close(got, want, tol, what):
        got = got.double()
        err = torch.where(got == want, 0.0, (got - want).abs())         # (infinite ones too)
        assert not bool(((err > tol) | got.isnan()).any()), (what, float((err / tol).max()))

    inside = (t >= 0) & (t < vocab)
    own = want_lp.gather(1, t.clamp(0, vocab - 1)[:, None])[:, 0]
    own = torch.where(none, float("-inf"), own)
    far = dist.gather(1, t.clamp(0, vocab - 1)[:, None])[:, 0]
    tol = 2 * u * torch.where(torch.isinf(own), 0.0, own.abs() + far.abs()) + 2 * u * log_s + d_log
    assert bool((lp[t < 0] == 0).all()) and bool(lp[t >= vocab].isnan().all())
    assert bool(lp[inside & bad].isnan().all()) and bool(h[bad].isnan().all())
    ok = inside & ~bad
    close(lp[ok], own[ok], tol[ok], "logprobs")
    h_tol = d_log + 3 * es * want_h.abs() + 4 * u * log_s + vocab * 2.0 ** -119
    want_h = torch.where(none, 0.0, want_h)
    close(h[~bad], want_h[~bad], h_tol[~bad], "entropy")
    assert bool((st[~bad & ~none, 0] == m[~bad & ~none].float()).all())
    assert bool((st[none, 0] == float("-inf")).all()) and bool((st[none, 1] == 0).all())
    close(st[~bad & ~none, 1], log_s[~bad & ~none], d_log[~bad & ~none], "log sum")
    # gradient
    nans = bad | (t >= vocab)
    assert bool(d[nans].isnan().all())
    a = torch.where(t < 0, 0.0, gl.double())[:, None]
    p = torch.where(none[:, None], 0.0, p)
    f = torch.where(none[:, None], 0.0, f)
    want = -a * p
    hot = t.clamp(0, vocab - 1)[:, None]
    certain = torch.where(none, 1.0, -own.expm1())
    want.scatter_(1, hot, torch.where(inside, a[:, 0] * certain, want.gather(1, hot)[:, 0])[:, None])
    e_lp = (d_log + 2 * u * log_s)[:, None] + 3 * u * f.abs() + \
        2 * u * torch.where(p > 0, dist.abs(), 0.0)
    e_p = p * (e_lp + 3 * u * f.abs() + 2.0 ** -22)
    tol = a.abs() * (e_p + 3 * u * p)
    extra = a[:, 0].abs() * (e_p.gather(1, hot)[:, 0] + 2.0 ** -21 * certain)
    tol.scatter_add_(1, hot, torch.where(inside, extra, 0.0)[:, None])
    # (exponentials below 2^-126 may be 0)
    tol = tol + 1.001 * hg.HALF[dtype] * want.abs() + 2.0 ** -126 * (1 + a.abs())
    close(d[~nans], want[~nans], tol[~nans], "dlogits")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(256, 24_576), (257, 24_576), (256, 24_575), (86, 24_577),
                                        (37, 65_544)])
def test_logprobs_at_the_edges_of_the_split(rows, vocab, dtype):
    rng = np.random.default_rng([rows, vocab, 43])
    x = hg.logit_values(rng, rows, vocab)
    x[0] = -np.inf
    x[1, rng.random(vocab) < 0.9] = -np.inf
    x[2, vocab - 1] = 60
    t = rng.integers(-1, vocab, rows)
    t[2] = vocab - 1
    hg.check_logprobs(x, t, dtype, 0)
    hg.check_logprobs(x, t, dtype, dh.DL_MAX_TOP, pad=1)


def test_logprobs_gradient_of_an_infinite_loss_weight_stays_in_its_row():
    """A NaN or infinite dlogprobs reaches its own row alone, and none without a target."""
    rng = np.random.default_rng(44)
    x = hg.logit_values(rng, 4, 3000)
    lt, _, _, out = hg.run_logprobs(x, [1, 2, -1, 4], "f32")
    t = torch.tensor([1, 2, -1, 4], device=DEV)
    gl = torch.tensor([1.0, float("nan"), float("nan"), 1.0], device=DEV)
    d, want = torch.empty(4, 3000, device=DEV), torch.empty(4, 3000, device=DEV)
    dh.dl_logprobs_backward(lt, 4, 3000, t, out["stats"], gl, d)
    dh.dl_logprobs_backward(lt, 4, 3000, t, out["stats"], torch.ones(4, device=DEV), want)
    assert bool(d[1].isnan().all()) and bool((d[2] == 0).all())
    assert torch.equal(d[[0, 3]], want[[0, 3]])


@pytest.mark.parametrize("level", [-1.17, -3.3, -6.9])
@pytest.mark.parametrize("rows,vocab,dtype", [(2, 73_760, "bf16"), (260, 150_001, "f32"),
                                              (260, 1 << 20, "bf16"), (1, (1 << 30) + 7, "bf16")])
def test_log_sum_of_many_equal_logits(rows, vocab, dtype, level):
    """Every 101st token at 0 (so every thread meets one early) and all others at
    the same level: S = n0 + (vocab - n0) e^level.  Equal terms added one by one
    round the same way every time, so a chain of additions would show at its full
    length.  A term is off by 2^-22 + 3 u |level| (see sum_error) and each
    addition by one rounding: 16 elements (8 in fp32) in a group, the groups of a
    thread in runs of at most 128, 5 for what is left of a row, one for each
    run, 8 for the threads, 4 for the parts.  Log S adds 3 roundings of its own; the
    entropy is log S and a quotient of two such sums times |level|."""
    group = 16 if dtype == "bf16" else 8
    mine = vocab / (16 if rows <= 256 else 1) / 256                  # a thread's share
    chain = group + min(128, mine / group) + 5 + mine // (128 * group) + 12
    x = torch.full((rows, vocab), level, device=DEV, dtype=hg.TORCH[dtype])
    x[:, ::101] = 0
    n0 = -(-vocab // 101)
    level = float(x[0, 1])
    t = torch.full((rows,), vocab - 1, dtype=torch.int64, device=DEV)
    lp, h, st = (torch.full(n, 9.0, device=DEV) for n in ((rows,), (rows,), (rows, 2)))
    need = dh.dl_logprobs_workspace_bytes(rows, vocab)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    dh.dl_logprobs(x, rows, vocab, t, lp, h, st, workspace=ws)
    rest = (vocab - n0) * np.exp(level)
    log_s = np.log(n0 + rest)
    es = 2.0 ** -22 + 3 * hg.U * abs(level) + chain * hg.U
    hg.within(hg.host(st)[:, 1], np.full(rows, log_s), es + 3 * hg.U * log_s, "log sum")
    hg.within(hg.host(lp), np.full(rows, level - log_s),
              es + 4 * hg.U * log_s + 2 * hg.U * (log_s - level), "logprobs")
    mean = rest * level / (n0 + rest)
    hg.within(hg.host(h), np.full(rows, log_s - mean),
              es + 4 * hg.U * log_s + (2 * es + 4 * hg.U) * abs(mean), "entropy")
    assert bool((st[:, 0] == 0).all())


def split_logprobs(x, t, ws, k, stream=None):
    rows, vocab = x.shape
    out = dict(logprobs=torch.empty(rows, device=DEV), entropy=torch.empty(rows, device=DEV),
               stats=torch.empty(rows, 2, device=DEV),
               top_ids=torch.empty(rows, k, dtype=torch.int64, device=DEV),
               top_logprobs=torch.empty(rows, k, device=DEV))
    dh.dl_logprobs(x, rows, vocab, t, top_k=k, workspace=ws, stream=stream, **out)
    return out


def test_split_rows_in_two_graphs_and_on_two_streams_at_once():
    """Rows in parts, whose results meet in a workspace: one each for two graphs
    that are replayed at the same time, and for two streams given by argument."""
    rows, vocab, k = 9, 60_000, 11
    need = dh.dl_logprobs_workspace_bytes(rows, vocab, k)
    assert need > 0
    g = torch.Generator(device=DEV).manual_seed(51)
    xs = [torch.empty(rows, vocab, device=DEV) for _ in range(2)]
    ts = [torch.randint(0, vocab, (rows,), generator=g, device=DEV) for _ in range(2)]
    wss = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for x in xs:
        x.normal_(generator=g)
    for x, t, ws in zip(xs, ts, wss):
        split_logprobs(x, t, ws, k)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, t, ws in zip(xs, ts, wss):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(split_logprobs(x, t, ws, k))
    for _ in range(4):
        for x in xs:
            x.normal_(generator=g).mul_(3)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        want = [split_logprobs(x, t, torch.empty(need, dtype=torch.uint8, device=DEV), k)
                for x, t in zip(xs, ts)]
        torch.cuda.synchronize()
        got = [split_logprobs(x, t, ws, k, stream=s)
               for x, t, ws, s in zip(xs, ts, wss, streams)]
        torch.cuda.synchronize()
        for a, b, c in zip(outs, want, got):
            for name in a:
                assert torch.equal(a[name], b[name]), name
                assert torch.equal(c[name], b[name]), name


def test_published_in_a_graph_follows_the_candidate():
    """publish() and answer() captured together: each replay lays out the flat
    vector as it is then, and eager work on the same head in between is its own."""
    global_, ema = hp.merged()
    flat = global_.clone()
    head = Head(hp.LAYOUT, flat, 40)
    x, r, t = hp.stream(20, 3)
    head.publish()
    head.answer(x, r, t, top_k=5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        head.publish()
        a = head.answer(x, r, t, top_k=5)
        got = [v.clone() for v in (a.logits, a.logprobs, a.entropy, a.top_ids)]
    for k, source in enumerate((ema, global_, ema, global_)):
        flat.copy_(source)
        head.publish()
        head.answer(*hp.stream(33, 60 + k), top_k=3)
        torch.cuda.synchronize()
        graph.replay()
        other = Head(hp.LAYOUT, source, 20)
        other.publish()
        b = other.answer(x, r, t, top_k=5)
        torch.cuda.synchronize()
        for u, v in zip(got, (b.logits, b.logprobs, b.entropy, b.top_ids)):
            assert torch.equal(u, v)


# --------------------------------------------------------------------------
# The training path through the library's calls alone
# --------------------------------------------------------------------------


def test_gradient_of_the_norms_output_by_the_librarys_product():
    """dlogits . E with the product the framework has: the logits' gradient laid
    out tokens last, then dl_matmul_f32(DL_TN); the norm's backward takes it."""
    rows = 64
    global_, _ = hp.merged()
    head = Head(hp.LAYOUT, global_, rows)
    x, r, t = hp.stream(rows, 9, "f32")
    sm, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(hp.WIDTH, device=DEV)
    a = head.score(x, r, t, sum_=sm)
    d = head.loss_gradient(a, t, torch.full((rows,), -1.0 / rows, device=DEV))
    dt = d.t().contiguous()
    dy = torch.empty(rows, hp.WIDTH, device=DEV)
    dl.dl_matmul_f32(dl.DL_TN, dt, rows, head.embed, hp.WIDTH, rows, hp.WIDTH, hp.VOCAB, dy,
                     hp.WIDTH)
    ws = torch.empty(dh.dl_rmsnorm_workspace_bytes(rows, hp.WIDTH), dtype=torch.uint8, device=DEV)
    head.backward(dy, sm, dx, dw, ws)
    g, e = hg.host(d).astype(np.float64), hg.host(head.embed).astype(np.float64)
    hg.within(hg.host(dy), g @ e, (hp.VOCAB + 2) * hg.U * (np.abs(g) @ np.abs(e)), "dy")
    s, inv, w = hg.host(sm), hg.host(head._inv[:rows]), hg.host(head.weight)
    want_dx, want_dw = oh.norm_backward(hg.host(dy), None, s, inv, w)
    # as check_backward of test_head_gpu
    i = inv.astype(np.float64)[:, None]
    gy, h = np.abs(hg.host(dy).astype(np.float64) * w), np.abs(s.astype(np.float64) * i)
    c = (gy * h).mean(axis=1, keepdims=True)
    tol = i * h * c * (hp.WIDTH + 8) * hg.U + 6 * hg.U * (i * (gy + h * c))
    hg.within(hg.host(dx), want_dx, tol + 1.001 * hg.U * np.abs(want_dx), "dx")
    t_abs = np.abs(hg.host(dy).astype(np.float64)) * h
    hg.within(hg.host(dw), want_dw, (rows + 4) * hg.U * t_abs.sum(axis=0), "dweight")
