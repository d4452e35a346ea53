"""The output head's kernels against the oracle (oracle/head.py).

Where the call defines every rounding (the norm's values from its own inverse
root mean square, 8-bit and 4-bit codes, scales) the result is compared bit for
bit.  Elsewhere the tolerance counts roundings: u = 2^-24 is half a step of
binary32, and a sum of n terms in any order is off by at most (n - 1) u of the
sum of magnitudes (to first order).
"""
import numpy as np
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from checkpoint_averaging_amd import dlmerge as dl
from oracle import head as oh

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}       # half a step, relative
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def to_dev(x, dtype):
    """binary32 numpy -> device tensor; the values it holds."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(DEV).to(TORCH[dtype])
    return t, t.float().cpu().numpy()


def host(t):
    return t.float().cpu().numpy() if t.dtype != torch.uint8 else t.cpu().numpy()


def bits(t):
    t = t.cpu()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).numpy()


def padded(x, pad, dtype, fill=float("nan")):
    """A device matrix whose rows are `pad` elements apart beyond their length, and its frame."""
    rows, cols = x.shape
    frame = torch.full((rows, cols + pad), 0.0, device=DEV).to(TORCH[dtype])
    if fill is not None:
        frame.fill_(fill)
    view = frame[:, :cols]
    t, values = to_dev(x, dtype)
    view.copy_(t)
    return view, values, frame


def same_bits(got, want, what):
    a, b = np.asarray(got), np.asarray(want)
    assert a.shape == b.shape, (what, a.shape, b.shape)
    ok = (a == b) | ((a != a) & (b != b))
    every = bool(ok.all())
    assert every, (what, int((~ok).sum()), np.argwhere(~ok)[:4].tolist(),
                      a[~ok][:4].tolist(), b[~ok][:4].tolist())


def within(got, want, tol, what):
    got, want, tol = np.asarray(got, np.float64), np.asarray(want, np.float64), np.asarray(tol)
    tol = np.broadcast_to(tol, want.shape)
    fin = np.isfinite(want)
    nans = np.array_equal(np.isnan(got), np.isnan(want))
    assert nans, (what, "NaN", np.argwhere(np.isnan(got) != np.isnan(want))[:4].tolist())
    infs = np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    assert infs, (what, "infinities")
    err = np.abs(got[fin] - want[fin])
    bad = err > tol[fin]
    any_bad = bool(bad.any())
    assert not any_bad, (what, int(bad.sum()), float((err / np.maximum(tol[fin], 1e-300)).max()))


# --------------------------------------------------------------------------
# Norm
# --------------------------------------------------------------------------


def stream_values(rng, rows, cols):
    return (rng.standard_normal((rows, cols)) *
            np.exp(0.5 * rng.standard_normal(cols))).astype(np.float32)


def check_norm(x, res, weight, dtype, out, kind, eps=1e-5, pad=0, keep_sum=True, inplace=None):
    rows, cols = x.shape
    xt, xv, _ = padded(x, pad, dtype)
    rt = rv = None
    if res is not None:
        rt, rv, _ = padded(res, pad, dtype)
    wt = torch.from_numpy(weight).to(DEV)
    frame = torch.full((rows, cols + pad), 7.0, device=DEV).to(TORCH[out])
    y = frame[:, :cols]
    sframe = torch.full((rows, cols + pad), 7.0, device=DEV).to(TORCH[dtype])
    sm = None
    if res is not None and keep_sum:
        sm = {"x": xt, "residual": rt}.get(inplace, sframe[:, :cols])
    scales = (torch.full((rows,), 9.0, device=DEV) if kind == dh.DL_SCALE_ROW else
              torch.full((rows, -(-cols // 32)), 9, dtype=torch.uint8, device=DEV)
              if kind == dh.DL_SCALE_BLOCK32 else None)
    inv = torch.empty(rows, device=DEV)
    dh.dl_rmsnorm(xt, rows, cols, wt, y, eps=eps, residual=rt, sum_=sm, scales=scales,
                  scale_kind=kind, inv_rms=inv)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore", over="ignore"):
        s = xv if rv is None else oh.round_to(xv + rv, dtype)
    if sm is not None:
        same_bits(host(sm), s, "sum")
    want_inv = oh.norm_inv(s, eps)
    want_inv[want_inv >= 2.0 ** 128] = np.inf                   # rounded to binary32
    got_inv = host(inv)
    # one rounding of a value that is itself off by some 2^-50
    within(got_inv, want_inv, np.abs(want_inv) * U * 1.0001, "inv")
    v = oh.norm_values(s, got_inv, weight)
    if out == "e4m3":
        codes, sc = (oh.e4m3_rows if kind == dh.DL_SCALE_ROW else oh.e4m3_blocks)(v)
        same_bits(bits(y.contiguous()), codes, "codes")
        same_bits(host(scales), sc, "scales")
    else:
        same_bits(host(y), oh.round_to(v, out), "y")
    if pad:
        assert bool((host(frame)[:, cols:] == 7.0).all()), "gap between rows written"
    return s


OUTS = [("f32", dh.DL_SCALE_NONE), ("bf16", dh.DL_SCALE_NONE), ("e4m3", dh.DL_SCALE_ROW),
        ("e4m3", dh.DL_SCALE_BLOCK32)]


@pytest.mark.parametrize("out,kind", OUTS, ids=["f32", "bf16", "e4m3_row", "e4m3_block"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (3, 31), (5, 33), (70, 128), (9, 500),
                                       (300, 2048), (6, 2049), (4, 5632), (3, 8193), (2, 20001),
                                       (2, 32768)])
def test_norm(rows, cols, dtype, out, kind):
    rng = np.random.default_rng([rows, cols])
    x, res = stream_values(rng, rows, cols), stream_values(rng, rows, cols)
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    check_norm(x, res, w, dtype, out, kind)
    check_norm(x, None, w, dtype, out, kind, pad=3)


@pytest.mark.parametrize("inplace", ["x", "residual", None])
def test_norm_sum_in_place(inplace):
    rng = np.random.default_rng(3)
    x, res = stream_values(rng, 37, 777), stream_values(rng, 37, 777)
    w = rng.standard_normal(777).astype(np.float32)
    check_norm(x, res, w, "bf16", "e4m3", dh.DL_SCALE_BLOCK32, pad=5, inplace=inplace)
    check_norm(x, res, w, "bf16", "bf16", dh.DL_SCALE_NONE, keep_sum=False)


@pytest.mark.parametrize("out,kind", OUTS, ids=["f32", "bf16", "e4m3_row", "e4m3_block"])
def test_norm_extreme_rows(out, kind):
    """Zero rows, tiny and huge values, NaN and infinities: those rows alone are touched."""
    rng = np.random.default_rng(11)
    x = stream_values(rng, 10, 96)
    x[0] = 0
    x[1] = 1e-42                                    # subnormal
    x[2, 5] = np.nan
    x[3, 40] = np.inf
    x[4, 95] = -np.inf
    x[5] *= 1e18                                    # squares past binary32
    x[6] *= 1e-30
    x[7, :64] = 0                                   # empty blocks
    w = np.ones(96, np.float32)
    w[90:] = 1e-38
    check_norm(x, None, w, "f32", out, kind)
    check_norm(x, None, w, "f32", out, kind, eps=0.0)


def test_norm_many_rows():
    """More rows than one launch's workgroups hold at once, small rows."""
    rng = np.random.default_rng(1)
    check_norm(stream_values(rng, 40_003, 24), stream_values(rng, 40_003, 24),
               np.ones(24, np.float32), "bf16", "bf16", dh.DL_SCALE_NONE)


def run_backward(dy, ds, s, inv, w, dtype, pad=0, inplace=None, want_dw=True):
    rows, cols = dy.shape
    yt, yv, _ = padded(dy, pad, dtype)
    st, sv, _ = padded(s, pad, dtype)
    dt = dv = None
    if ds is not None:
        dt, dv, _ = padded(ds, pad, dtype)
    frame = torch.full((rows, cols + pad), 7.0, device=DEV).to(TORCH[dtype])
    dx = {"dy": yt, "dsum": dt}.get(inplace, frame[:, :cols])
    dw = torch.full((cols,), 5.0, device=DEV) if want_dw else None
    ws = torch.full((max(4, dh.dl_rmsnorm_workspace_bytes(rows, cols)),), 255, dtype=torch.uint8,
                    device=DEV)
    dh.dl_rmsnorm_backward(yt, st, rows, cols, torch.from_numpy(w).to(DEV),
                           torch.from_numpy(inv).to(DEV), dx, dsum=dt, dweight=dw, workspace=ws)
    torch.cuda.synchronize()
    if pad and inplace is None:
        assert bool((host(frame)[:, cols:] == 7.0).all()), "gap between rows written"
    return host(dx), None if dw is None else host(dw), yv, dv, sv


def check_backward(rows, cols, dtype, with_ds=True, **kw):
    rng = np.random.default_rng([rows, cols, 2])
    s, dy, ds = (stream_values(rng, rows, cols) for _ in range(3))
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    inv = oh.norm_inv(to_dev(s, dtype)[1], 1e-5).astype(np.float32)
    dx, dw, yv, dv, sv = run_backward(dy, ds if with_ds else None, s, inv, w, dtype, **kw)
    want_dx, want_dw = oh.norm_backward(yv, dv, sv, inv, w)
    g, h = np.abs(yv.astype(np.float64) * w), np.abs(sv.astype(np.float64) * inv[:, None])
    i = inv.astype(np.float64)[:, None]
    # c: cols products of two rounded factors, summed in any order; then 5 roundings to dx
    c_abs = (g * h).mean(axis=1, keepdims=True)
    tol = i * h * c_abs * (cols + 8) * U + 6 * U * (i * (g + h * c_abs))
    tol = tol + (0 if dv is None else 2 * U * np.abs(dv)) + 1.001 * HALF[dtype] * np.abs(want_dx)
    within(dx, want_dx, tol, "dx")
    if dw is not None:
        t = np.abs(yv.astype(np.float64)) * h
        within(dw, want_dw, (rows + 4) * U * t.sum(axis=0), "dweight")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (7, 33), (129, 128), (1000, 500),
                                       (513, 2048), (3001, 2048), (65, 2050), (33, 5632), (9, 8200), (5, 32768)])
def test_norm_backward(rows, cols, dtype):
    check_backward(rows, cols, dtype)
    check_backward(rows, cols, dtype, with_ds=False, pad=3)


@pytest.mark.parametrize("inplace", ["dy", "dsum"])
def test_norm_backward_in_place(inplace):
    check_backward(300, 777, "bf16", inplace=inplace, pad=1)
    check_backward(300, 2048, "f32", inplace=inplace)


def test_norm_backward_without_weight_gradient_and_rows():
    check_backward(50, 300, "f32", want_dw=False)
    dw = torch.full((300,), 5.0, device=DEV)
    ws = torch.empty(max(4, dh.dl_rmsnorm_workspace_bytes(0, 300)), dtype=torch.uint8, device=DEV)
    e = torch.empty(0, 300, device=DEV)
    dh.dl_rmsnorm_backward(e, e, 0, 300, torch.ones(300, device=DEV),
                           torch.empty(0, device=DEV), e, dweight=dw, workspace=ws)
    assert bool((dw == 0).all())


def test_norm_gradient_against_differences():
    """dx and dweight against central differences of the forward call itself:
    f = sum(dy * y) + sum(ds * s), in binary32 outputs, step 2^-6.  The
    difference quotient is off by its third-order term (below 2^-12 here: the
    curvature of x/rms over a row of 40 unit values) and by the outputs'
    roundings, 40 values of u each over the step."""
    rng = np.random.default_rng(17)
    rows, cols, step = 2, 40, 2.0 ** -6
    x, dy, ds = (rng.standard_normal((rows, cols)).astype(np.float32) for _ in range(3))
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)

    def f(x, w):
        y, inv = torch.empty(rows, cols, device=DEV), torch.empty(rows, device=DEV)
        xt = torch.from_numpy(x).to(DEV)
        dh.dl_rmsnorm(xt, rows, cols, torch.from_numpy(w).to(DEV), y, inv_rms=inv)
        return float((dy.astype(np.float64) * host(y)).sum() + (ds.astype(np.float64) * x).sum())

    inv = oh.norm_inv(x, 1e-5).astype(np.float32)
    dx, dw, *_ = run_backward(dy, ds, x, inv, w, "f32")
    tol = 2.0 ** -10 + 2 * rows * cols * 4 * 4 * U / step
    for i in [(0, 0), (0, 39), (1, 7), (1, 20)]:
        e = np.zeros_like(x)
        e[i] = step
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * step) - dx[i]) < tol
    for c in (0, 13, 39):
        e = np.zeros_like(w)
        e[c] = step
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * step) - dw[c]) < tol


# --------------------------------------------------------------------------
# 4 bits
# --------------------------------------------------------------------------


def quantize(wt, rows, cols, values=None):
    kb = -(-cols // 32)
    packed = torch.full((rows, kb * 16), 0xEE, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, kb), 0xEE, dtype=torch.uint8, device=DEV)
    dh.dl_w4_quantize(wt, rows, cols, packed, scales, values=values)
    torch.cuda.synchronize()
    return packed, scales


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 31, 0), (5, 32, 1), (7, 33, 0),
                                           (64, 128, 0), (17, 500, 3), (130, 2048, 0),
                                           (2, 5632, 0), (1001, 96, 0)])
def test_quantize(rows, cols, pad, dtype):
    rng = np.random.default_rng([rows, cols, 4])
    w = (0.02 * rng.standard_normal((rows, cols)) *
         np.exp(0.5 * rng.standard_normal((rows, 1)))).astype(np.float32)
    wt, wv, _ = padded(w, pad, dtype)
    frame = torch.full((rows, cols + pad), 7.0, device=DEV).to(TORCH[dtype])
    packed, scales = quantize(wt, rows, cols, frame[:, :cols])
    want_p, want_s, want_v = oh.w4_quantize(wv)
    same_bits(host(scales), want_s, "scales")
    same_bits(host(packed), want_p, "packed")
    same_bits(host(frame)[:, :cols], want_v, "values")
    if pad:
        assert bool((host(frame)[:, cols:] == 7.0).all()), "gap between rows written"
    p2, s2 = quantize(wt, rows, cols)                             # without values
    assert torch.equal(p2, packed) and torch.equal(s2, scales)
    quantize(wt, rows, cols, wt)                                  # values over w itself
    same_bits(host(wt), want_v, "in place")


def test_quantize_ties_and_extremes():
    w = np.zeros((12, 64), np.float32)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32)
    near = np.concatenate([mids, np.nextafter(mids, np.float32(0)),
                           np.nextafter(mids[:-1], np.float32(9))])
    w[0, :len(near)] = near
    w[0, 32:32 + len(near)] = -near
    w[1] = w[0] * 2.0 ** -100
    w[2] = w[0] * 2.0 ** 100
    w[3, 0] = 2.0 ** -149                                         # smallest subnormal
    w[4, :40] = 1e-39
    w[5, 3] = np.nan
    w[6, 33] = np.inf
    w[7, 1] = -np.inf
    w[8, 0] = np.finfo(np.float32).max
    w[9, 0] = np.nextafter(np.float32(6), np.float32(9))
    w[10] = -0.0
    packed, scales = quantize(torch.from_numpy(w).to(DEV), 12, 64,
                              values := torch.empty(12, 64, device=DEV))
    want_p, want_s, want_v = oh.w4_quantize(w)
    same_bits(host(scales), want_s, "scales")
    same_bits(host(packed), want_p, "packed")
    with np.errstate(over="ignore"):                              # 2^128 is infinite
        same_bits(host(values), want_v.astype(np.float32), "values")


def e4m3_vectors(x, kind):
    codes, sc = (oh.e4m3_rows if kind == dh.DL_SCALE_ROW else oh.e4m3_blocks)(x)
    v = oh.e4m3_value(codes)
    if kind == dh.DL_SCALE_ROW:
        values = v * sc.astype(np.float64)[:, None]
    else:
        values = v * np.repeat(oh.scale_value(sc), 32, axis=1)[:, :x.shape[1]]
    return (torch.from_numpy(codes).to(DEV).view(torch.float8_e4m3fn),
            torch.from_numpy(sc).to(DEV), values, v)


def check_matvec(packed, scales, rows, cols, x, kind, out, pad_x=0, pad_y=0, exact=False):
    """x: binary32 vectors, given to the call in bf16 (kind NONE) or 8 bits."""
    count = x.shape[0]
    sc = None
    if kind == dh.DL_SCALE_NONE:
        xt, xv, _ = padded(x, pad_x, "bf16")
        xv = xv.astype(np.float64)
    else:
        q, sc, xv, _ = e4m3_vectors(x, kind)
        frame = torch.full((count, cols + pad_x), 127, dtype=torch.uint8, device=DEV)
        frame[:, :cols] = q.view(torch.uint8)
        xt = frame.view(torch.float8_e4m3fn)[:, :cols]
    frame = torch.full((count, rows + pad_y), 7.0, device=DEV).to(TORCH[out])
    dh.dl_w4_matvec(torch.from_numpy(packed).to(DEV), torch.from_numpy(scales).to(DEV), rows,
                    cols, xt, count, frame[:, :rows], x_scales=sc, x_scale_kind=kind)
    torch.cuda.synchronize()
    w = oh.w4_values(packed, scales, cols)
    w = np.where(np.abs(w) >= 2.0 ** 128, np.copysign(np.inf, w), w)     # past binary32
    with np.errstate(invalid="ignore"):
        want = xv @ w.T
        mag = np.abs(xv) @ np.abs(w).T
    got = host(frame)
    # where the magnitudes' sum passes binary32, a partial sum may be infinite and the total
    # infinite or NaN, by the order of additions: nothing to compare
    past = np.isfinite(mag) & (mag >= 2.0 ** 128)
    got[:, :rows][past] = want[past] = mag[past] = 0
    if exact:
        same_bits(got[:, :rows], oh.round_to(want, out), "y")
    else:
        within(got[:, :rows], want,
               (cols + 2) * U * mag + 1.001 * HALF[out] * np.abs(want) +
               cols * 2.0 ** -126, "y")                      # products below 2^-126 may be 0
    if pad_y:
        assert bool((got[:, rows:] == 7.0).all()), "gap between rows written"


def random_w4(rng, rows, cols, lo=118, hi=124):
    kb = -(-cols // 32)
    packed = rng.integers(0, 256, (rows, kb * 16), dtype=np.uint8)
    scales = rng.integers(lo, hi, (rows, kb), dtype=np.uint8)
    return packed, scales


KINDS = [dh.DL_SCALE_NONE, dh.DL_SCALE_ROW, dh.DL_SCALE_BLOCK32]


@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "e4m3_row", "e4m3_block"])
@pytest.mark.parametrize("rows,cols,count", [(1, 1, 1), (5, 31, 2), (16, 32, 1), (17, 33, 3),
                                             (70, 128, 16), (33, 129, 17), (128, 160, 32),
                                             (2048, 2048, 1), (300, 2048, 12), (64, 5632, 5),
                                             (50, 5632, 32), (1000, 96, 7), (19, 8200, 31)])
def test_matvec(rows, cols, count, kind):
    rng = np.random.default_rng([rows, cols, count])
    packed, scales = random_w4(rng, rows, cols)
    x = rng.standard_normal((count, cols)).astype(np.float32)
    check_matvec(packed, scales, rows, cols, x, kind, "f32")
    check_matvec(packed, scales, rows, cols, x, kind, "bf16", pad_x=1, pad_y=3)


@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "e4m3_row", "e4m3_block"])
@pytest.mark.parametrize("rows,cols,count", [(40, 77, 1), (129, 288, 9), (16, 2048, 16),
                                             (35, 1000, 32), (200, 5632, 2)])
def test_matvec_of_whole_numbers_is_exact(rows, cols, count, kind):
    """Small multiples of a half on both sides: every partial sum is a multiple
    of 1/4 below 2^22 and fits binary32 in any order, so the result is the exact
    one and a misplaced element cannot hide.  (x in 8 bits: whole numbers up to
    7 with amax 7 in every row and block, whose scale is 2^-6, or 2^-6 exactly.)"""
    rng = np.random.default_rng([rows, cols, count, 9])
    packed, scales = random_w4(rng, rows, cols, 127, 128)
    x = rng.integers(-7, 8, (count, cols)).astype(np.float32)
    x[:, ::32] = 7
    check_matvec(packed, scales, rows, cols, x, kind, "f32", exact=True)


def test_matvec_every_code_scale_and_special_value():
    """Scale bytes 0 and 254, NaN blocks, infinite and NaN vector elements: only
    the rows and vectors they belong to are touched."""
    rng = np.random.default_rng(21)
    rows, cols = 40, 320
    packed, scales = random_w4(rng, rows, cols)
    scales[0], scales[1] = 0, 254
    scales[2, 3] = 255
    x = rng.integers(-7, 8, (6, cols)).astype(np.float32)
    x[1], x[2] = 0, x[2] * 2.0 ** -60
    x[3, 17] = np.inf
    x[4, 300] = np.nan
    check_matvec(packed, scales, rows, cols, x, dh.DL_SCALE_NONE, "f32")
    # products of row 1 with whole numbers pass binary32: compared where they fit
    x[3, 17] = x[4, 300] = 1
    scales[1] = 120
    for kind in KINDS:
        check_matvec(packed, scales, rows, cols, x, kind, "f32")


def test_matvec_of_a_vector_that_stands_for_nan():
    """x in 8 bits with a NaN block (or row) scale: NaN for that vector alone."""
    rng = np.random.default_rng(22)
    packed, scales = random_w4(rng, 50, 160)
    x = rng.standard_normal((4, 160)).astype(np.float32)
    x[2, 70] = np.nan
    check_matvec(packed, scales, 50, 160, x, dh.DL_SCALE_ROW, "f32")
    check_matvec(packed, scales, 50, 160, x, dh.DL_SCALE_BLOCK32, "bf16")


def test_matvec_of_small_factors():
    """Factors on one side near 2^-126 and below, large ones on the other, whole
    multiples: results in the normal range are the exact ones."""
    rng = np.random.default_rng(23)
    rows, cols = 48, 160
    packed, scales = random_w4(rng, rows, cols, 1, 4)            # weights of 2^-127 to 6 * 2^-124
    x = (rng.integers(-7, 8, (3, cols)) * 2.0 ** 100).astype(np.float32)
    check_matvec(packed, scales, rows, cols, x, dh.DL_SCALE_NONE, "f32", exact=True)
    packed, scales = random_w4(rng, rows, cols, 220, 223)
    x = (rng.integers(-7, 8, (3, cols)) * 2.0 ** -126).astype(np.float32)
    check_matvec(packed, scales, rows, cols, x, dh.DL_SCALE_NONE, "f32", exact=True)


def test_matvec_of_the_embedding():
    """73,760 x 2048 (byte offsets past 2^26, every row tile), whole numbers."""
    rng = np.random.default_rng(2)
    packed, scales = random_w4(rng, 73760, 2048, 127, 128)
    x = rng.integers(-7, 8, (2, 2048)).astype(np.float32)
    check_matvec(packed, scales, 73760, 2048, x, dh.DL_SCALE_NONE, "f32", exact=True)


# --------------------------------------------------------------------------
# Log probabilities
# --------------------------------------------------------------------------


def logit_values(rng, rows, vocab):
    x = (2.5 * rng.standard_normal((rows, vocab)) - 4).astype(np.float32)
    x[np.arange(rows), rng.integers(0, vocab, rows)] = 6 + 5 * rng.standard_normal(rows)
    return x


def sum_error(vocab):
    """Relative error of S (and of sums of e d): at least 64 lanes share a row,
    so no chain of additions is longer than vocab/64 + 64; each term exp(d) is
    off by 2^-22 + 3 u |d|, and |d| e <= 1/e (e of the sum weighs it at most
    with mean |d| <= log vocab + 40)."""
    return (vocab / 64 + 64) * U + 2.0 ** -22 + 3 * U * (np.log(vocab) + 40)


def run_logprobs(x, targets, dtype, top_k=0, pad=0, want_stats=True):
    rows, vocab = x.shape
    lt, lv, _ = padded(x, pad, dtype)
    t = torch.from_numpy(np.asarray(targets, np.int64)).to(DEV)
    out = dict(logprobs=torch.full((rows,), 9.0, device=DEV),
               entropy=torch.full((rows,), 9.0, device=DEV),
               stats=torch.full((rows, 2), 9.0, device=DEV) if want_stats else None,
               top_ids=torch.full((rows, top_k), -7, dtype=torch.int64, device=DEV) if top_k else None,
               top_logprobs=torch.full((rows, top_k), 9.0, device=DEV) if top_k else None)
    need = dh.dl_logprobs_workspace_bytes(rows, vocab, top_k)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV) if need else None
    dh.dl_logprobs(lt, rows, vocab, t, top_k=top_k, workspace=ws, **out)
    torch.cuda.synchronize()
    return lt, lv, t, out


def check_logprobs(x, targets, dtype, top_k=0, pad=0):
    rows, vocab = x.shape
    targets = np.asarray(targets, np.int64)
    lt, lv, t, out = run_logprobs(x, targets, dtype, top_k, pad)
    lp, h, m, log_s = oh.log_softmax(lv)
    es = sum_error(vocab)
    with np.errstate(invalid="ignore", over="ignore"):
        rest = np.expm1(log_s)
        # error of log S (exponentials below 2^-126 may count as 0)
        d_log = es * np.minimum(1, np.abs(rest)) + 3 * U * np.abs(log_s) + vocab * 2.0 ** -126
        lp_tol = 2 * U * np.abs(np.where(np.isfinite(lp), lp, 0)) + \
            2 * U * np.abs(log_s)[:, None] + d_log[:, None]
    want = np.zeros(rows)
    tol = np.zeros(rows)
    for r, c in enumerate(targets):
        want[r] = 0.0 if c < 0 else np.nan if c >= vocab else lp[r, c]
        if 0 <= c < vocab:
            tol[r] = lp_tol[r, c] + 2 * U * abs(float(lv[r, c]) - m[r]) if np.isfinite(want[r]) else 0
    within(host(out["logprobs"]), want, tol, "logprobs")
    within(host(out["entropy"]), h, d_log + 3 * es * np.abs(h) + 4 * U * np.abs(log_s) +
           vocab * 2.0 ** -119, "entropy")                   # such a term times |d| below 2^7
    st = host(out["stats"])
    finite = np.isfinite(log_s) & ~np.isneginf(m)
    same_bits(st[finite, 0], m[finite].astype(np.float32), "row maximum")
    within(st[finite, 1], log_s[finite], d_log[finite], "log sum")
    nothing = np.isneginf(m)
    assert (st[nothing, 0] == -np.inf).all() and (st[nothing, 1] == 0).all()
    assert np.isnan(st[~finite & ~nothing, 1]).all()
    if top_k:
        ids = oh.top_ids(lv, top_k)
        same_bits(out["top_ids"].cpu().numpy(), ids, "top_ids")
        r = np.arange(rows)[:, None]
        with np.errstate(invalid="ignore"):
            d = np.where(np.isfinite(lp[r, ids]), lv[r, ids] - m[:, None], 0)
        within(host(out["top_logprobs"]), lp[r, ids], lp_tol[r, ids] + 2 * U * np.abs(d),
               "top_logprobs")
    return lt, lv, t, out, lp, h, log_s, d_log


SIZES = [(1, 1), (2, 5), (3, 64), (1, 257), (5, 1000), (300, 513), (2, 8193), (1, 73760),
         (9, 50277), (70, 50304), (3, 200001)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_logprobs(rows, vocab, dtype):
    rng = np.random.default_rng([rows, vocab])
    x = logit_values(rng, rows, vocab)
    t = np.where(rng.random(rows) < 0.5, x.argmax(1), rng.integers(0, vocab, rows))
    check_logprobs(x, t, dtype, 0)
    check_logprobs(x, t, dtype, min(vocab, 1))
    check_logprobs(x, t, dtype, min(vocab, 20), pad=1)
    check_logprobs(x, t, dtype, min(vocab, dh.DL_MAX_TOP), pad=8)


def test_logprobs_of_a_nearly_certain_token_keep_their_digits():
    rng = np.random.default_rng(8)
    x = logit_values(rng, 4, 3000)
    x[:, 77] = [18, 25, 40, 90]
    lt, lv, t, out, lp, h, log_s, _ = check_logprobs(x, [77] * 4, "f32", 3)
    got = host(out["logprobs"]).astype(np.float64)
    assert (np.abs(got[:3] / lp[:3, 77] - 1) < sum_error(3000)).all()
    assert got[3] <= 0 and host(out["entropy"])[3] >= 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 700), (3, 9000), (40, 9000), (1, 73760)])
def test_logprobs_masked_and_special_rows(rows, vocab, dtype):
    """Masked tokens of -infinity and of the type's lowest value, rows that a mask
    leaves nothing or one token of, NaN and +infinity (also where masked)."""
    rng = np.random.default_rng([rows, vocab, 1])
    low = float(torch.finfo(TORCH[dtype]).min)
    base = logit_values(rng, rows, vocab)
    some = rng.random((rows, vocab)) < 0.7
    targets = rng.integers(0, vocab, rows)
    rows_of = [np.where(some, -np.inf, base),
               np.where(some, low, base),
               np.full((rows, vocab), -np.inf),
               np.full((rows, vocab), low),
               np.where(np.arange(vocab) == vocab // 2, 1.5, -np.inf) * np.ones((rows, 1)),
               np.where(np.arange(vocab) == vocab - 1, low, -np.inf) * np.ones((rows, 1)),
               np.where(np.arange(vocab) == 3, np.nan, np.where(some, -np.inf, base)),
               np.where(np.arange(vocab) == vocab - 2, np.inf, base),
               np.full((rows, vocab), np.nan),
               np.where(np.arange(vocab) % 2 == 0, np.nan, np.inf) * np.ones((rows, 1)),
               np.zeros((rows, vocab)), np.full((rows, vocab), -0.0),
               np.where(some, -0.0, 0.0)]
    for i, x in enumerate(rows_of):
        print("special rows", i, flush=True)
        check_logprobs(x.astype(np.float32), targets, dtype, 9)
        check_logprobs(x.astype(np.float32), [vocab // 2] * rows, dtype, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 30])
def test_alternatives_of_ordered_and_tied_rows(rows, dtype):
    """Ascending, descending, few distinct values, the largest ones side by side
    at the row's end: orders in which a running choice has to be given up often."""
    vocab = 40_000
    i = np.arange(vocab)
    for k in (1, 7, 32):
        for x in (i * 1e-3, -i * 1e-3, (i % 7) * 1.0, (i // 1000) * 0.5, -(i // 64) * 0.25,
                  np.where(i >= vocab - 300, 3.0 + (i % 5), 0.0), np.where(i == 39_999, 1.0, 0.0)):
            check_logprobs(np.broadcast_to(x, (rows, vocab)).astype(np.float32), [5] * rows,
                           dtype, k)


def test_logprobs_more_rows_than_a_grid():
    """Rows past the launch limits of both directions, of five logits each."""
    rows, vocab = (1 << 20) + 77, 5
    x = torch.randn(rows, vocab, device=DEV)
    t = torch.randint(0, vocab, (rows,), device=DEV)
    lp, st = torch.empty(rows, device=DEV), torch.empty(rows, 2, device=DEV)
    ids, top = torch.empty(rows, 1, dtype=torch.int64, device=DEV), torch.empty(rows, 1, device=DEV)
    dh.dl_logprobs(x, rows, vocab, t, lp, stats=st, top_k=1, top_ids=ids, top_logprobs=top)
    d = torch.empty_like(x)
    dh.dl_logprobs_backward(x, rows, vocab, t, st, torch.ones(rows, device=DEV), d)
    want = torch.log_softmax(x.double(), 1)
    tol = 16 * U * (1 + x.abs().max().item() + 4)            # a few roundings of small values
    assert (lp - want.gather(1, t[:, None])[:, 0]).abs().max().item() < tol
    assert torch.equal(ids[:, 0], x.argmax(1))
    hot = torch.zeros_like(want).scatter_(1, t[:, None], 1.0)
    assert (d - (hot - want.exp())).abs().max().item() < 2 * tol


def test_logprobs_targets_outside_the_vocabulary():
    rng = np.random.default_rng(4)
    x = logit_values(rng, 6, 300)
    check_logprobs(x, [-1, 300, 299, 0, -(1 << 40), 1 << 40], "f32", 2)


def test_logprobs_without_optional_outputs():
    x = torch.randn(5, 300, device=DEV)
    h = torch.empty(5, device=DEV)
    dh.dl_logprobs(x, 5, 300, entropy=h)
    ids, lps = torch.empty(5, 4, dtype=torch.int64, device=DEV), torch.empty(5, 4, device=DEV)
    dh.dl_logprobs(x, 5, 300, top_k=4, top_ids=ids, top_logprobs=lps)
    lp, want_h, _, _ = oh.log_softmax(host(x))
    within(host(h), want_h, 1e-4, "entropy")
    same_bits(ids.cpu().numpy(), oh.top_ids(host(x), 4), "ids")


def check_logprobs_backward(x, targets, dtype, with_h, pad=0, inplace=False, seed=0):
    rows, vocab = x.shape
    rng = np.random.default_rng([rows, vocab, seed])
    lt, lv, t, out, lp, h, log_s, d_log = check_logprobs(x, targets, dtype, 0, pad)
    gl = rng.standard_normal(rows).astype(np.float32)
    gh = rng.standard_normal(rows).astype(np.float32) if with_h else None
    frame = torch.full((rows, vocab + pad), 7.0, device=DEV).to(TORCH[dtype])
    dst = lt if inplace else frame[:, :vocab]
    dh.dl_logprobs_backward(lt, rows, vocab, t, out["stats"], torch.from_numpy(gl).to(DEV), dst,
                            entropy=out["entropy"] if with_h else None,
                            dentropy=torch.from_numpy(gh).to(DEV) if with_h else None)
    torch.cuda.synchronize()
    want = oh.logprobs_backward(lp, h, np.asarray(targets), gl, gh)
    with np.errstate(invalid="ignore", over="ignore"):
        f = np.where(np.isfinite(lp), lp, 0.0)
        p = np.where(np.isfinite(lp), np.exp(f), 0.0)
        # log p: error of log S, two roundings of its parts; p adds its exponential's own
        e_lp = np.nan_to_num(d_log + 2 * U * np.abs(log_s))[:, None] + 3 * U * np.abs(f) + \
            2 * U * np.abs(np.nan_to_num(lv.astype(np.float64), neginf=0, posinf=0) * (p > 0))
        e_p = p * (e_lp + 3 * U * np.abs(f) + 2.0 ** -22)
        tol = np.abs(gl.astype(np.float64))[:, None] * (e_p + 3 * U * p)
        for r, c in enumerate(targets):
            if 0 <= c < vocab:                 # -expm1(log p)
                tol[r, c] += abs(gl[r]) * (e_lp[r, c] * p[r, c] + 2.0 ** -21 * -np.expm1(f[r, c]))
        if with_h:
            hh = np.nan_to_num(h)[:, None]
            e_h = np.nan_to_num(d_log + 3 * sum_error(vocab) * np.abs(h) +
                                4 * U * np.abs(log_s))[:, None]
            tol += np.abs(gh.astype(np.float64))[:, None] * (
                e_p * np.abs(f + hh) + p * (e_lp + e_h + 4 * U * (np.abs(f) + hh)))
    tol = tol + 1.001 * HALF[dtype] * np.abs(np.nan_to_num(want)) + 2.0 ** -126
    within(host(dst), want, tol, "dlogits")
    if pad and not inplace:
        assert bool((host(frame)[:, vocab:] == 7.0).all()), "gap between rows written"


@pytest.mark.parametrize("with_h", [False, True], ids=["logprob", "with_entropy"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,pad", [(1, 1, 0), (3, 64, 0), (7, 257, 1), (40, 1000, 0),
                                            (2, 73760, 0), (33, 50277, 3), (1, 200001, 0)])
def test_logprobs_backward(rows, vocab, pad, dtype, with_h):
    rng = np.random.default_rng([rows, vocab, 6])
    x = logit_values(rng, rows, vocab)
    t = np.where(rng.random(rows) < 0.6, x.argmax(1), rng.integers(0, vocab, rows))
    t = np.where(rng.random(rows) < 0.2, -1, t)
    check_logprobs_backward(x, t, dtype, with_h, pad)
    check_logprobs_backward(x, t, dtype, with_h, pad, inplace=True)


def test_logprobs_backward_special_rows():
    rng = np.random.default_rng(12)
    x = logit_values(rng, 9, 400)
    x[1, rng.random(400) < 0.8] = -np.inf
    x[2] = -np.inf
    x[3, 7] = np.nan
    x[4, 9] = np.inf
    x[5] = float(np.finfo(np.float32).min)
    x[6, 50] = 60
    t = [3, int(np.argmax(x[1])), 5, 7, 9, 11, 50, 400, -1]
    check_logprobs_backward(x, t, "f32", False)
    check_logprobs_backward(x, t, "f32", True)


def test_logprobs_gradient_against_differences():
    """dlogits against central differences of the forward call: f = sum(g logp) +
    sum(b H) with step 2^-6; the quotient is off by its third-order term
    (below 2^-13 x the gradients' size: third derivatives of log S are below 1/4)
    and by 2 x 4 values' roundings (below 16 u each) over the step."""
    rng = np.random.default_rng(19)
    rows, vocab, step = 2, 30, 2.0 ** -6
    x = rng.standard_normal((rows, vocab)).astype(np.float32)
    t = np.array([4, 17])
    gl, gh = (rng.standard_normal(rows).astype(np.float32) for _ in range(2))

    def f(x):
        _, _, _, out = run_logprobs(x, t, "f32")
        return float((gl.astype(np.float64) * host(out["logprobs"])).sum() +
                     (gh.astype(np.float64) * host(out["entropy"])).sum())

    lt, _, tt, out = run_logprobs(x, t, "f32")
    d = torch.empty(rows, vocab, device=DEV)
    dh.dl_logprobs_backward(lt, rows, vocab, tt, out["stats"], torch.from_numpy(gl).to(DEV), d,
                            entropy=out["entropy"], dentropy=torch.from_numpy(gh).to(DEV))
    d = host(d)
    tol = 2.0 ** -11 + 8 * 16 * U * 4 / step
    for i in [(0, 0), (0, 4), (0, 29), (1, 17), (1, 3)]:
        e = np.zeros_like(x)
        e[i] = step
        assert abs((f(x + e) - f(x - e)) / (2 * step) - d[i]) < tol, i


def test_offsets_past_32_bits():
    """Two rows 2^31 + 8 elements apart: row offsets need 64 bits."""
    ld, vocab = (1 << 31) + 8, 5000
    big = torch.zeros(ld + vocab, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(31)
    x = logit_values(rng, 2, vocab)
    xt, xv = to_dev(x, "bf16")
    big[:vocab], big[ld:] = xt[0], xt[1]
    out = torch.empty(2, device=DEV)
    ids, lps = torch.empty(2, 3, dtype=torch.int64, device=DEV), torch.empty(2, 3, device=DEV)
    t, st = torch.tensor([1, 4999], device=DEV), torch.empty(2, 2, device=DEV)
    need = dh.dl_logprobs_workspace_bytes(2, vocab, 3)
    ws = torch.empty(max(need, 4), dtype=torch.uint8, device=DEV)
    dh.dl_logprobs(big, 2, vocab, t, out, stats=st, top_k=3, top_ids=ids, top_logprobs=lps,
                   workspace=ws, ldl=ld)
    lp = oh.log_softmax(xv)[0]
    within(host(out), lp[[0, 1], [1, 4999]], 1e-4, "logprobs")
    same_bits(ids.cpu().numpy(), oh.top_ids(xv, 3), "ids")
    dh.dl_logprobs_backward(big, 2, vocab, t, st, torch.ones(2, device=DEV), big, ldl=ld, lddl=ld)
    got = host(big[ld:])
    want = -np.exp(lp[1])
    want[4999] = -np.expm1(lp[1, 4999])
    within(got, want, 2.0 ** -8 * 1.01 * np.abs(want) + 1e-6, "dlogits")
    w = torch.ones(vocab, device=DEV)
    big[:vocab], big[ld:] = xt[0], xt[1]
    y = torch.empty(2, vocab, device=DEV)
    dh.dl_rmsnorm(big, 2, vocab, w, y, ldx=ld, y_dtype=dl.DL_F32)
    inv = oh.norm_inv(xv, 1e-5).astype(np.float32)
    within(host(y), xv * inv[:, None], 1e-6 + 3 * U * np.abs(xv), "norm")
