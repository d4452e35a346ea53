"""The operators of a merged model's output head, as cases to measure.

A merge leaves several candidates for the next published model (the global,
its EMA, the uniform average, snapshots).  Each is read out through the same
chain: the last residual addition and RMS norm, the product with the tied
embedding held in 4 bits, and the log probabilities of given tokens with
their entropy and top alternatives; training adds the gradients of the loss
and of the norm.  The sizes are those of the two models this repository lays
out (width 2048, feed-forward 5632, vocabulary 73,760; width 128, vocabulary
50,304) and generic ones around them.

``run`` computes a case in plain torch operations, or, with ``own``, through
the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = float(np.float32(1e-5))
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
DTYPES = {"f32": F32, "bf16": BF16, "e4m3": E4M3}
# the magnitudes a 4-bit weight (one sign, two exponent and one mantissa bit) takes
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------


def listed():
    return [
        # one token being decoded: the token's confidence and its 8 alternatives
        dict(name="logprobs one token", op="logprobs", rows=1, vocab=73760, dtype="bf16", top=8,
             banned=0, ld_pad=0),
        # 12 draft positions of a masked-diffusion decoder, tokens beside a neighbour banned
        dict(name="logprobs draft", op="logprobs", rows=12, vocab=73760, dtype="f32", top=20,
             banned=40, ld_pad=0),
        # a probe of 2048 tokens that compares the averages: log probability and entropy
        dict(name="logprobs probe", op="logprobs", rows=2048, vocab=73760, dtype="bf16", top=0,
             banned=0, ld_pad=0),
        # the same probe with five alternatives, an odd vocabulary inside padded rows
        dict(name="logprobs odd vocabulary", op="logprobs", rows=777, vocab=50277, dtype="f32",
             top=5, banned=0, ld_pad=27),
        # the loss of a training step at its masked positions, with the logits' gradient
        dict(name="loss and gradient", op="loss", rows=2048, vocab=73760, dtype="bf16",
             entropy=False, ld_pad=0),
        # a fine-tuning loss with an entropy term on a short odd batch
        dict(name="loss with entropy term", op="loss", rows=333, vocab=50304, dtype="f32",
             entropy=True, ld_pad=0),
        # decoding: the last norm of one token, written in 8 bits with a scale for each 32
        dict(name="norm one token", op="norm", rows=1, cols=2048, dtype="bf16", out="e4m3",
             scale="block", residual=True),
        # scoring: the norm before an 8-bit product, a scale for each row
        dict(name="norm of a probe", op="norm", rows=16384, cols=2048, dtype="bf16", out="e4m3",
             scale="row", residual=True),
        # training: the norm with its backward pass
        dict(name="norm and backward", op="norm_train", rows=8191, cols=2048, dtype="bf16",
             residual=True),
        # decoding one token: the tied embedding's product from 4-bit weights
        dict(name="4-bit head, one vector", op="matvec", rows=73760, cols=2048, count=1,
             x="bf16", scale="none", out="f32"),
        # 12 draft positions in 8 bits through a feed-forward matrix
        dict(name="4-bit product, 12 vectors", op="matvec", rows=2048, cols=5632, count=12,
             x="e4m3", scale="block", out="bf16"),
        # publishing: a merged embedding laid out in 4 bits, and the values it stands for
        dict(name="4-bit embedding", op="quantize", rows=73760, cols=2048, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "loss", "norm", "norm_train", "matvec", "matvec",
                     "quantize"])
    if op in ("logprobs", "loss"):
        vocab = rng.choice([73760, 50304, 50277, _log_int(rng, 300, 150000)])
        rows = min(_log_int(rng, 1, 4096), max(1, 120_000_000 // vocab))
        c = dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice(["bf16", "f32"]),
                 ld_pad=rng.choice([0, 0, rng.randrange(1, 64)]))
        if op == "loss":
            c["entropy"] = rng.random() < 0.5
        else:
            c["top"] = rng.choice([0, 1, 5, 20, 32])
            c["banned"] = rng.choice([0, 0, 7, 64])
        return c
    if op == "norm":
        cols = rng.choice([128, 2048, 5632, _log_int(rng, 64, 8192)])
        out, scale = rng.choice([("f32", "none"), ("bf16", "none"), ("e4m3", "row"),
                                 ("e4m3", "block")])
        return dict(op=op, rows=min(_log_int(rng, 1, 65536), 33_000_000 // cols), cols=cols,
                    dtype=rng.choice(["bf16", "f32"]), out=out, scale=scale,
                    residual=rng.random() < 0.7)
    if op == "norm_train":
        cols = rng.choice([128, 2048, 5632, _log_int(rng, 64, 8192)])
        return dict(op=op, rows=min(_log_int(rng, 1, 32768), 16_000_000 // cols), cols=cols,
                    dtype=rng.choice(["bf16", "f32"]), residual=rng.random() < 0.7)
    if op == "matvec":
        cols = rng.choice([128, 2048, 5632, _log_int(rng, 64, 8192)])
        rows = min(rng.choice([2048, 5632, 73760, 50304, _log_int(rng, 64, 80000)]),
                   150_000_000 // cols)
        x, scale = rng.choice([("bf16", "none"), ("e4m3", "row"), ("e4m3", "block")])
        return dict(op=op, rows=rows, cols=cols, count=rng.choice([1, 1, 2, rng.randrange(3, 33)]),
                    x=x, scale=scale, out=rng.choice(["f32", "bf16"]))
    cols = rng.choice([128, 2048, 5632, _log_int(rng, 64, 8192)])
    return dict(op="quantize", rows=min(_log_int(rng, 16, 80000), 120_000_000 // cols), cols=cols,
                dtype=rng.choice(["f32", "bf16"]))


def _size(name):
    return {"f32": 4, "bf16": 2, "e4m3": 1}[name]


def work(case):
    op = case["op"]
    if op in ("logprobs", "loss"):
        n = case["rows"] * case["vocab"]
        b = n * _size(case["dtype"]) + case["rows"] * 20
        if op == "loss":
            return {"bytes": 2 * n * _size(case["dtype"]) + case["rows"] * 24, "flops": 10 * n}
        return {"bytes": b + case["rows"] * case["top"] * 12, "flops": 5 * n}
    if op == "norm":
        n, e = case["rows"] * case["cols"], _size(case["dtype"])
        moved = n * (e * (3 if case["residual"] else 1) + _size(case["out"]))
        scales = {"none": 0, "row": 4 * case["rows"], "block": case["rows"] * -(-case["cols"] // 32)}
        return {"bytes": moved + scales[case["scale"]] + 4 * case["cols"] + 4 * case["rows"],
                "flops": 5 * n}
    if op == "norm_train":
        n, e = case["rows"] * case["cols"], _size(case["dtype"])
        # forward: x (and the residual) in, the sum and y out; backward: dy, the sum (and its
        # own gradient) in, dx out
        moved = n * e * ((4 if case["residual"] else 2) + (4 if case["residual"] else 3))
        return {"bytes": moved + 12 * case["cols"] + 8 * case["rows"], "flops": 14 * n}
    blocks = case["rows"] * -(-case["cols"] // 32)
    if op == "matvec":
        xb = case["count"] * case["cols"] * _size(case["x"])
        return {"bytes": blocks * 17 + xb + case["count"] * case["rows"] * _size(case["out"]),
                "flops": 2 * case["rows"] * case["cols"] * case["count"]}
    n = case["rows"] * case["cols"]
    return {"bytes": 2 * n * _size(case["dtype"]) + blocks * 17, "flops": 4 * n}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _logits(case, g):
    """Logits of a trained model: mostly a wide bulk, one token well above it in most rows."""
    rows, vocab, ld = case["rows"], case["vocab"], case["vocab"] + case["ld_pad"]
    out = (2.5 * _randn(g, rows, ld) - 4).to(DTYPES[case["dtype"]])[:, :vocab]
    peak = torch.randint(0, vocab, (rows, 1), generator=g, device=DEV)
    out.scatter_(1, peak, (6 + 5 * _randn(g, rows, 1)).to(out.dtype))
    return out, peak[:, 0]


def _targets(rows, vocab, peak, g, some_without):
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    pick = torch.rand(rows, generator=g, device=DEV)
    t = torch.where(pick < 0.6, peak, t)
    return torch.where(pick > 0.9, torch.full_like(t, -1), t) if some_without else t


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op in ("logprobs", "loss"):
        rows, vocab = case["rows"], case["vocab"]
        x, peak = _logits(case, g)
        s["logits"] = x
        s["targets"] = _targets(rows, vocab, peak, g, op == "loss")
        new = lambda *sh, dtype=F32: torch.empty(*sh, dtype=dtype, device=DEV)  # noqa: E731
        s["logprobs"], s["entropy_out"], s["stats"] = new(rows), new(rows), new(rows, 2)
        if op == "loss":
            n = int((s["targets"] >= 0).sum())
            s["dlogprobs"] = torch.full((rows,), -1.0 / max(1, n), device=DEV)
            s["dentropy"] = (torch.full((rows,), -0.01 / max(1, n), device=DEV)
                             if case["entropy"] else None)
            s["dlogits"] = torch.empty(rows, vocab, dtype=x.dtype, device=DEV)
        else:
            if case["banned"]:
                at = torch.randint(0, vocab, (rows, case["banned"]), generator=g, device=DEV)
                x.scatter_(1, at, float("-inf"))
            s["top_ids"] = new(rows, case["top"], dtype=torch.int64)
            s["top_logprobs"] = new(rows, case["top"])
        return s
    if op in ("norm", "norm_train"):
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        # a residual stream: a few channels far larger than the rest
        channel = torch.exp(0.5 * _randn(g, cols))
        s["x"] = (0.5 * _randn(g, rows, cols)).to(dt)
        s["residual"] = (_randn(g, rows, cols) * channel).to(dt) if case["residual"] else None
        s["weight"] = 1 + 0.2 * _randn(g, cols)
        s["sum"] = torch.empty(rows, cols, dtype=dt, device=DEV) if case["residual"] else None
        out = case.get("out", case["dtype"])
        s["y"] = torch.empty(rows, cols, dtype=DTYPES[out], device=DEV)
        kind = case.get("scale", "none")
        s["scales"] = (torch.empty(rows, device=DEV) if kind == "row" else
                       torch.empty(rows, -(-cols // 32), dtype=torch.uint8, device=DEV)
                       if kind == "block" else None)
        s["inv_rms"] = torch.empty(rows, device=DEV)
        if op == "norm_train":
            s["dy"] = (1e-3 * _randn(g, rows, cols)).to(dt)
            s["dsum"] = (1e-3 * _randn(g, rows, cols)).to(dt) if case["residual"] else None
            s["dx"] = torch.empty(rows, cols, dtype=dt, device=DEV)
            s["dweight"] = torch.empty(cols, device=DEV)
        return s
    if op == "matvec":
        rows, cols, count = case["rows"], case["cols"], case["count"]
        # a trained matrix held in 4 bits: codes of two weights a byte (the lower index in the
        # low half), a power-of-two exponent byte for each 32 weights of a row
        s["packed"], s["scales"], _ = _quantize_plain(0.02 * _randn(g, rows, cols))
        x = _randn(g, count, cols) * torch.exp(0.3 * _randn(g, cols))
        s["x_scales"] = None
        if case["x"] == "bf16":
            s["x_in"] = x.to(BF16)
        elif case["scale"] == "row":
            s["x_in"], s["x_scales"] = _e4m3_rows(x)
        else:
            s["x_in"], s["x_scales"] = _e4m3_blocks(x)
        s["y"] = torch.empty(count, rows, dtype=DTYPES[case["out"]], device=DEV)
        return s
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    kb = -(-cols // 32)
    s["w"] = (0.02 * _randn(g, rows, cols) * torch.exp(0.5 * _randn(g, rows, 1))).to(dt)
    s["values"] = torch.empty_like(s["w"])
    s["packed"] = torch.empty(rows, kb * 16, dtype=torch.uint8, device=DEV)
    s["scales"] = torch.empty(rows, kb, dtype=torch.uint8, device=DEV)
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "logprobs":
        return _logprobs_plain(s)
    if op == "loss":
        return _loss_plain(s)
    if op == "norm":
        return _norm_plain(s)
    if op == "norm_train":
        return _norm_train_plain(s)
    if op == "matvec":
        return _matvec_plain(s)
    packed, scales, values = _quantize_plain(s["w"].float())
    return {"packed": packed, "scales": scales, "values": values.to(s["w"].dtype)}


def _run_own(s):
    from checkpoint_averaging_amd import dlhead as dl
    op = s["op"]
    if op in ("logprobs", "loss"):
        rows, vocab = s["rows"], s["vocab"]
        top = s.get("top", 0)
        if "workspace" not in s:
            need = dl.dl_logprobs_workspace_bytes(rows, vocab, top)
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
        if op == "logprobs":
            dl.dl_logprobs(s["logits"], rows, vocab, s["targets"], s["logprobs"],
                           entropy=s["entropy_out"], top_k=top,
                           top_ids=s["top_ids"] if top else None,
                           top_logprobs=s["top_logprobs"] if top else None,
                           workspace=s["workspace"])
            return {"logprobs": s["logprobs"], "entropy": s["entropy_out"],
                    "top_ids": s["top_ids"], "top_logprobs": s["top_logprobs"]}
        entropy = s["entropy_out"] if s["entropy"] else None
        dl.dl_logprobs(s["logits"], rows, vocab, s["targets"], s["logprobs"], entropy=entropy,
                       stats=s["stats"], workspace=s["workspace"])
        dl.dl_logprobs_backward(s["logits"], rows, vocab, s["targets"], s["stats"],
                                s["dlogprobs"], s["dlogits"], entropy=entropy,
                                dentropy=s["dentropy"])
        return {"logprobs": s["logprobs"], "entropy": entropy, "dlogits": s["dlogits"]}
    if op in ("norm", "norm_train"):
        rows, cols = s["rows"], s["cols"]
        kind = {"none": dl.DL_SCALE_NONE, "row": dl.DL_SCALE_ROW,
                "block": dl.DL_SCALE_BLOCK32}[s.get("scale", "none")]
        dl.dl_rmsnorm(s["x"], rows, cols, s["weight"], s["y"], eps=EPS, residual=s["residual"],
                      sum_=s["sum"], scales=s["scales"], scale_kind=kind, inv_rms=s["inv_rms"])
        out = {"sum": s["sum"], "y": s["y"], "scales": s["scales"], "inv_rms": s["inv_rms"]}
        if op == "norm":
            return out
        if "workspace" not in s:
            need = dl.dl_rmsnorm_workspace_bytes(rows, cols)
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        dl.dl_rmsnorm_backward(s["dy"], s["x"] if s["sum"] is None else s["sum"], rows, cols,
                               s["weight"], s["inv_rms"], s["dx"], dsum=s["dsum"],
                               dweight=s["dweight"], workspace=s["workspace"])
        return {**out, "dx": s["dx"], "dweight": s["dweight"]}
    rows, cols = s["rows"], s["cols"]
    if op == "matvec":
        kind = {"none": dl.DL_SCALE_NONE, "row": dl.DL_SCALE_ROW,
                "block": dl.DL_SCALE_BLOCK32}[s["scale"]]
        dl.dl_w4_matvec(s["packed"], s["scales"], rows, cols, s["x_in"], s["count"], s["y"],
                        x_scales=s["x_scales"], x_scale_kind=kind)
        return s["y"]
    dl.dl_w4_quantize(s["w"], rows, cols, s["packed"], s["scales"], values=s["values"])
    return {"packed": s["packed"], "scales": s["scales"], "values": s["values"]}


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------


def _stats_plain(x):
    """Distances from the row's maximum, their exponentials, the sum of these and its logarithm.
    The maximum's own 1 is left out of the sum and comes in by log1p, so that a nearly certain
    token keeps its digits."""
    m, at = x.max(1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    rest = e.scatter(1, at, 0.0).sum(1)
    return d, e, 1 + rest, torch.log1p(rest)


def _entropy_plain(d, e, total, log_total):
    return log_total - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(1) / total


def _of_targets(d, log_total, targets):
    got = d.gather(1, targets.clamp(min=0)[:, None])[:, 0] - log_total
    return torch.where(targets >= 0, got, torch.zeros_like(got))


def _top_plain(x, k):
    """Indices of the k largest of each row, equal values by the lowest index: one 64-bit key
    holds the value's order in its high half and the index, counted down, in the low one."""
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).to(torch.int64)
    key = (order << 32) | (x.shape[1] - 1 - torch.arange(x.shape[1], device=x.device))
    return x.shape[1] - 1 - (torch.topk(key, k, dim=1).values & 0xFFFFFFFF)


def _logprobs_plain(s):
    x = s["logits"].float().contiguous()
    d, e, total, log_total = _stats_plain(x)
    out = {"logprobs": _of_targets(d, log_total, s["targets"]),
           "entropy": _entropy_plain(d, e, total, log_total),
           "top_ids": s["top_ids"], "top_logprobs": s["top_logprobs"]}
    if s["top"]:
        out["top_ids"] = _top_plain(x, s["top"])
        out["top_logprobs"] = d.gather(1, out["top_ids"]) - log_total[:, None]
    return out


def _loss_plain(s):
    x = s["logits"].float()
    d, e, total, log_total = _stats_plain(x)
    logp = d - log_total[:, None]
    p = torch.exp(logp)
    t = s["targets"]
    at = t.clamp(min=0)[:, None]
    gl = torch.where(t >= 0, s["dlogprobs"], torch.zeros_like(s["dlogprobs"]))[:, None]
    entropy = None
    # 1 - p of the given token as -expm1(log p): a nearly certain token keeps its digits
    dx = (-gl * p).scatter(1, at, -gl * torch.expm1(logp.gather(1, at)))
    if s["entropy"]:
        entropy = _entropy_plain(d, e, total, log_total)
        dx = dx - s["dentropy"][:, None] * p * (logp + entropy[:, None])
    return {"logprobs": _of_targets(d, log_total, t), "entropy": entropy,
            "dlogits": dx.to(s["logits"].dtype)}


def _norm_forward(s):
    r = s["x"]
    if s["residual"] is not None:
        r = (r.float() + s["residual"].float()).to(r.dtype)
    r32 = r.float()
    # in 64 bits: what is rounded to 8 bits must not hang on the order of this sum
    inv = (1.0 / torch.sqrt(r32.double().square().mean(1) + EPS)).float()
    return r, r32, inv, (r32 * inv[:, None]) * s["weight"]


def _e4m3_rows(y):
    amax = y.abs().amax(1)
    fine = amax >= 2.0 ** -100
    scale = torch.where(fine, amax / 448, torch.zeros_like(amax))
    back = torch.where(fine, 448 / amax, torch.zeros_like(amax))
    return (y * back[:, None]).to(E4M3), scale


def _blocks_of(y):
    rows, cols = y.shape
    kb = -(-cols // 32)
    if kb * 32 != cols:
        y = torch.nn.functional.pad(y, (0, kb * 32 - cols))
    return y.view(rows, kb, 32)


def _e4m3_blocks(y):
    """The smallest power of two b with amax <= 448 b (448 = 1.75 * 2^8) for each 32 columns."""
    b = _blocks_of(y)
    byte = (((b.abs().amax(2).view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=0)
    back = ((254 - byte) << 23).view(F32)
    q = (b * back[:, :, None]).to(E4M3).view(y.shape[0], -1)[:, :y.shape[1]]
    return q.contiguous(), byte.to(torch.uint8)


def _norm_plain(s):
    r, _, inv, y = _norm_forward(s)
    scales = None
    if s["scale"] == "row":
        y, scales = _e4m3_rows(y)
    elif s["scale"] == "block":
        y, scales = _e4m3_blocks(y)
    else:
        y = y.to(DTYPES[s["out"]])
    return {"sum": r if s["residual"] is not None else None, "y": y, "scales": scales,
            "inv_rms": inv}


def _norm_train_plain(s):
    r, r32, inv, y = _norm_forward(s)
    dy, h = s["dy"].float(), r32 * inv[:, None]
    gw = dy * s["weight"]
    dx = inv[:, None] * (gw - h * (gw * h).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"sum": r if s["residual"] is not None else None, "y": y.to(r.dtype), "scales": None,
            "inv_rms": inv, "dx": dx.to(r.dtype), "dweight": (dy * h).sum(0)}


def _quantize_plain(w):
    """Codes, exponent bytes and the values they stand for: the smallest power of two b with
    amax <= 6 b (6 = 1.5 * 2^2) for each 32 weights, then to the nearest of the eight
    magnitudes, a tie to the one whose last bit is 0."""
    rows, cols = w.shape
    b = _blocks_of(w)
    byte = (((b.abs().amax(2).view(torch.int32) + 0x3FFFFF) >> 23) - 2).clamp(min=0)
    back = ((254 - byte) << 23).view(F32)
    v = b * back[:, :, None]
    a = v.abs()
    # (between two magnitudes: the upper one has an odd code where the bound is included below)
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) +
            (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    table = torch.tensor(E2M1, device=w.device)
    scale = torch.ldexp(torch.ones_like(back), byte - 127)
    values = torch.copysign(table[code.long()], v) * scale[:, :, None]
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).view(rows, -1)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    return packed, byte.to(torch.uint8), values.view(rows, -1)[:, :cols]


def _weights_of(packed, scales, cols, dtype):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=packed.device)
    pairs = torch.stack((packed & 15, packed >> 4), dim=2).view(packed.shape[0], -1)
    b = torch.exp2(scales.to(dtype) - 127)
    w = table[pairs.int()].view(packed.shape[0], -1, 32) * b[:, :, None]
    return w.view(packed.shape[0], -1)[:, :cols]


def _vectors_of(s, dtype):
    x = s["x_in"].to(F32).to(dtype)
    if s["scale"] == "row":
        return x * s["x_scales"].to(dtype)[:, None]
    if s["scale"] == "block":
        b = torch.exp2(s["x_scales"].to(dtype) - 127)
        return x * b.repeat_interleave(32, dim=1)[:, :x.shape[1]]
    return x


def _matvec_plain(s):
    w = _weights_of(s["packed"], s["scales"], s["cols"], F32)
    return torch.matmul(_vectors_of(s, F32), w.t()).to(DTYPES[s["out"]])


# --------------------------------------------------------------------------
# In 64 bits, from the definitions
# --------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("logprobs", "loss"):
        return _exact_logprobs(s)
    if op in ("norm", "norm_train"):
        return _exact_norm(s)
    if op == "matvec":
        w = _exact_weights(s["packed"], s["scales"], s["cols"])
        return torch.matmul(w, _vectors_of(s, torch.float64).t()).t()
    return {"packed": None, "scales": None, "values": _exact_values(s["w"])}


def _exact_logprobs(s):
    """log p = x - log sum exp x by the library's own reduction in 64 bits."""
    x, t = s["logits"].double(), s["targets"]
    lp = x - torch.logsumexp(x, dim=1, keepdim=True)
    p = lp.exp()
    h = torch.special.entr(p).sum(1)
    at = (torch.arange(len(t), device=DEV), t.clamp(min=0))
    out = {"logprobs": lp[at].masked_fill(t < 0, 0.0), "entropy": h}
    if s["op"] == "logprobs":
        top = torch.sort(lp, dim=1, descending=True).values[:, :s["top"]] if s["top"] else None
        return {**out, "top_ids": None, "top_logprobs": top}
    gl = s["dlogprobs"].double().masked_fill(t < 0, 0.0)
    hot = torch.zeros_like(p)
    hot[at] = 1.0
    dx = gl[:, None] * (hot - p)
    if s["entropy"]:
        dx -= s["dentropy"].double()[:, None] * p * (lp + h[:, None])
    return {**out, "entropy": h if s["entropy"] else None, "dlogits": dx}


def _exact_norm(s):
    r = s["x"].double()
    if s["residual"] is not None:  # the sum is kept in the stream's type, and that is what is normed
        r = (r + s["residual"].double()).to(s["x"].dtype).double()
    inv = torch.rsqrt((r * r).sum(1) / s["cols"] + EPS)
    h = r * inv[:, None]
    y = h * s["weight"].double()
    scales, kind = None, s.get("scale", "none")
    if kind == "row":
        scales = y.abs().amax(1) / 448
        y = y / scales[:, None]
    elif kind == "block":
        amax = _blocks_of(y).abs().amax(2)
        b = torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(min=-127))
        y = y / b.repeat_interleave(32, dim=1)[:, :s["cols"]]
    out = {"sum": r if s["residual"] is not None else None, "y": y, "scales": scales,
           "inv_rms": inv}
    if s["op"] == "norm":
        return out
    dy = s["dy"].double()
    g = dy * s["weight"].double()
    dx = inv[:, None] * g - r * (inv ** 3 / s["cols"] * (g * r).sum(1))[:, None]
    if s["dsum"] is not None:
        dx = dx + s["dsum"].double()
    return {**out, "dx": dx, "dweight": torch.einsum("rc,rc->c", dy, h)}


def _exact_weights(packed, scales, cols):
    """Each code decoded from its bits: sign, two exponent bits, one mantissa bit."""
    code = torch.empty(packed.shape[0], 2 * packed.shape[1], dtype=torch.int32, device=DEV)
    code[:, 0::2], code[:, 1::2] = (packed & 15).int(), (packed >> 4).int()
    exp, man = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(exp == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2((exp - 1).double()))
    w = torch.where(code >= 8, -mag, mag)
    return (w * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1))[:, :cols]


def _exact_values(w):
    """The nearest magnitude, a tie to the even code: their spacing is 1/2 up to 2, 1 up to 4
    and 2 up to 6, and the even codes are the even multiples of it."""
    b = torch.exp2(torch.ceil(torch.log2(_blocks_of(w.double()).abs().amax(2) / 6)).clamp(min=-127))
    b = b.repeat_interleave(32, dim=1)[:, :w.shape[1]]
    v = w.double() / b
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    return torch.round(v / step) * step * b
