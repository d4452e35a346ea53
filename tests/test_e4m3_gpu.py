"""8-bit matrices with scales for 128 x 128 or 128 elements, and their product,
against the oracle: codes, scales and values bit for bit, products within the
roundings of a binary32 sum (and bf16's of the result)."""
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
TILE, BLOCK = dh.DL_SCALE_TILE128, dh.DL_SCALE_BLOCK128
HIGH = {TILE: 128, BLOCK: 1}


def groups(kind, rows):
    return -(-rows // HIGH[kind])


def quantized(x, kind, dtype="f32", pad=0, inplace=False):
    rows, cols = x.shape
    xt, xv, frame = hg.padded(x, pad, dtype)
    cframe = torch.full((rows, cols + pad), 0x55, dtype=torch.uint8, device=DEV)
    codes = cframe.view(torch.float8_e4m3fn)[:, :cols]
    scales = torch.full((groups(kind, rows), -(-cols // 128)), 9, dtype=torch.uint8, device=DEV)
    vframe = frame if inplace else torch.full((rows, cols + pad), 7.0, device=DEV).to(hg.TORCH[dtype])
    values = xt if inplace else vframe[:, :cols]
    dh.dl_e4m3_quantize(xt, rows, cols, codes, scales, kind, values=values)
    torch.cuda.synchronize()
    assert torch.all(cframe[:, cols:] == 0x55)
    if not inplace:
        assert torch.all(vframe[:, cols:] == 7)
    return xv, codes, scales, values


def check_quantize(x, kind, dtype="f32", pad=0, inplace=False):
    xv, codes, scales, values = quantized(x, kind, dtype, pad, inplace)
    want, e, v = oh.e4m3_quantize(xv, HIGH[kind])
    hg.same_bits(hg.host(scales), e, "scales")
    hg.same_bits(hg.bits(codes.contiguous()), want, "codes")
    with np.errstate(over="ignore"):
        hg.same_bits(hg.host(values), oh.round_to(v.astype(np.float32), dtype), "values")


SHAPES = [(1, 1), (1, 128), (3, 7), (5, 129), (128, 128), (127, 255), (130, 300), (300, 2048),
          (257, 65)]


@pytest.mark.parametrize("kind", [TILE, BLOCK])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(rows, cols, dtype, kind):
    rng = np.random.default_rng(rows * 3 + cols)
    x = hg.stream_values(rng, rows, cols) * np.exp(2 * rng.standard_normal((rows, 1)))
    check_quantize(x.astype(np.float32), kind, dtype)


@pytest.mark.parametrize("kind", [TILE, BLOCK])
@pytest.mark.parametrize("pad,inplace", [(1, False), (16, False), (3, True)])
def test_quantize_rows_apart(kind, pad, inplace):
    rng = np.random.default_rng(pad)
    check_quantize(hg.stream_values(rng, 150, 270), kind, "bf16", pad, inplace)


@pytest.mark.parametrize("kind", [TILE, BLOCK])
def test_quantize_ties_and_extremes(kind):
    """Every code's value and the midpoints between neighbours, at scales from the
    smallest to the largest; zeros, subnormals, infinities and NaN."""
    mags = oh.e4m3_value(np.arange(127))
    mids = (mags[1:] + mags[:-1]) / 2
    row = np.concatenate([mags, -mags, mids, -mids])
    rows = []
    for e in (-127, -126, -100, 0, 7, 100, 119):
        r = np.zeros(4 * 128)
        r[:127], r[128:255], r[256:382], r[384:510] = (row[:127] * 2.0 ** e, row[127:254] * 2.0 ** e,
                                                       row[254:380] * 2.0 ** e, row[380:] * 2.0 ** e)
        r[[127, 255, 383, 511]] = 448 * 2.0 ** e
        rows.append(r)
    rows.append(np.full(512, 3.4e38))
    rows.append(np.full(512, 1e-45))
    rows.append(np.zeros(512))
    x = np.repeat(np.array(rows, np.float32), HIGH[kind], axis=0)
    check_quantize(x, kind)
    for bad in (np.inf, -np.inf, np.nan):
        y = np.ones((130, 300), np.float32)
        y[129, 140] = bad
        check_quantize(y, kind)


def test_quantize_more_blocks_than_a_grid():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((70_000, 600)).astype(np.float32)
    for kind in (TILE, BLOCK):
        _, codes, scales, _ = quantized(x, kind)
        hg.same_bits(hg.host(scales), oh.tile_bytes(x, HIGH[kind]), "scales")
        some = slice(69_888, 70_000)
        want, _, _ = oh.e4m3_quantize(x[some], HIGH[kind])
        hg.same_bits(hg.bits(codes[some].contiguous()), want, "codes")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 7), (3, 128), (5, 300), (2, 2048), (300, 2047),
                                       (7, 5632), (2, 20_000)])
def test_norm_to_blocks_of_128(rows, cols, dtype):
    rng = np.random.default_rng(cols)
    x, r = hg.stream_values(rng, rows, cols), hg.stream_values(rng, rows, cols)
    weight = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    xt, xv = hg.to_dev(x, dtype)
    rt, rv = hg.to_dev(r, dtype)
    y = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.full((rows, -(-cols // 128)), 9, dtype=torch.uint8, device=DEV)
    inv = torch.empty(rows, device=DEV)
    dh.dl_rmsnorm(xt, rows, cols, torch.from_numpy(weight).to(DEV), y, residual=rt, scales=scales,
                  scale_kind=BLOCK, inv_rms=inv)
    torch.cuda.synchronize()
    v = oh.norm_values(oh.round_to(xv + rv, dtype), hg.host(inv), weight)
    codes, e, _ = oh.e4m3_quantize(v, 1)
    hg.same_bits(hg.host(scales), e, "scales")
    hg.same_bits(hg.bits(y), codes, "codes")


# --------------------------------------------------------------------------
# The product
# --------------------------------------------------------------------------


def operand(rng, rows, cols, kind, pad=0, spread=0.5):
    """Codes and scales of random values, and what they stand for."""
    x = (rng.standard_normal((rows, cols)) * np.exp(spread * rng.standard_normal((rows, 1)))
         ).astype(np.float32)
    codes, e, v = oh.e4m3_quantize(x, HIGH[kind])
    frame = torch.full((rows, cols + pad), 0x7F, dtype=torch.uint8, device=DEV)     # NaN codes
    frame[:, :cols] = torch.from_numpy(codes).to(DEV)
    return frame.view(torch.float8_e4m3fn)[:, :cols], torch.from_numpy(e).to(DEV), v


def product(w, ws, x, xs, out, ldy_pad=0):
    rows, cols, count = w.shape[0], w.shape[1], x.shape[0]
    frame = torch.full((count, rows + ldy_pad), 7.0, device=DEV).to(hg.TORCH[out])
    dh.dl_e4m3_matmul(w, ws, rows, cols, x, xs, count, frame[:, :rows])
    torch.cuda.synchronize()
    assert torch.all(frame[:, rows:] == 7)
    return hg.host(frame[:, :rows])


def check_product(got, wv, xv, out):
    want, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    cols = wv.shape[1]
    if out == "f32":
        tol = (cols + 2) * U * mag
    else:
        # each 128 products lose at most 2^-13 of their magnitudes' sum
        tol = (2.0 ** -13 + cols * U) * mag + 2.0 ** -8 * np.abs(want)
    hg.within(got, want, tol, "product")


PRODUCTS = [(1, 1, 1), (5, 7, 3), (128, 128, 16), (130, 129, 17), (300, 300, 1), (1000, 96, 33),
            (2048, 512, 12), (257, 2047, 70), (64, 5632, 2), (700, 260, 500), (4100, 128, 1100),
            (6000, 136, 2049)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,count", PRODUCTS)
def test_product(rows, cols, count, out):
    rng = np.random.default_rng(rows + cols + count)
    w, ws, wv = operand(rng, rows, cols, TILE)
    x, xs, xv = operand(rng, count, cols, BLOCK)
    check_product(product(w, ws, x, xs, out), wv, xv, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("count", [1, 20, 300])
@pytest.mark.parametrize("pad", [1, 2, 16])
def test_product_of_rows_apart(pad, count, out):
    """The gaps hold NaN codes, and y's are left alone."""
    rng = np.random.default_rng(pad)
    w, ws, wv = operand(rng, 500, 330, TILE, pad)
    x, xs, xv = operand(rng, count, 330, BLOCK, pad)
    check_product(product(w, ws, x, xs, out, pad), wv, xv, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,count", [(300, 384, 5), (300, 384, 200), (9000, 384, 1100)])
def test_product_of_whole_numbers_is_exact(rows, cols, count, out):
    """Small integers with scales of one power of two: every sum is exact, whatever the order."""
    rng = np.random.default_rng(rows)
    wi, xi = rng.integers(-2, 3, (rows, cols)), rng.integers(-2, 3, (count, cols))
    if out == "bf16":
        wi, xi = wi * (rng.random((rows, cols)) < 0.1), xi * (rng.random((count, cols)) < 0.1)
    code = lambda v: torch.from_numpy(oh.e4m3_code(v.astype(np.float64))).to(DEV)  # noqa: E731
    ws = torch.full((groups(TILE, rows), -(-cols // 128)), 127, dtype=torch.uint8, device=DEV)
    xs = torch.full((count, -(-cols // 128)), 127 + 3, dtype=torch.uint8, device=DEV)
    got = product(code(wi).view(torch.float8_e4m3fn), ws, code(xi).view(torch.float8_e4m3fn), xs, out)
    want = 8.0 * (xi.astype(np.float64) @ wi.T)
    assert np.abs(want).max() < 256 * 8
    hg.same_bits(got, want if out == "f32" else oh.round_to(want.astype(np.float32), "bf16"), "sum")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("count", [3, 60, 1200])
def test_product_scales_of_each_block(count, out):
    """Blocks of far scales: each row's scale and each block of columns has its own."""
    rng = np.random.default_rng(count)
    rows, cols = 6000 if count > 1000 else 400, 500
    w, ws, _ = operand(rng, rows, cols, TILE)
    x, xs, _ = operand(rng, count, cols, BLOCK)
    ws.copy_(torch.from_numpy(rng.integers(110, 140, ws.shape).astype(np.uint8)))
    xs.copy_(torch.from_numpy(rng.integers(110, 140, xs.shape).astype(np.uint8)))
    wv = oh.e4m3_value(hg.bits(w.contiguous())) * oh.tile_spread(hg.host(ws), w.shape, 128)
    xv = oh.e4m3_value(hg.bits(x.contiguous())) * oh.tile_spread(hg.host(xs), x.shape, 1)
    check_product(product(w, ws, x, xs, out), wv, xv, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("count", [4, 50, 1200])
def test_product_of_what_stands_for_nan(count, out):
    """A NaN code or scale reaches what it belongs to and nothing else."""
    rng = np.random.default_rng(1)
    rows = 6000 if count > 1000 else 300
    w, ws, _ = operand(rng, rows, 256, TILE)
    x, xs, _ = operand(rng, count, 256, BLOCK)
    clean = product(w, ws, x, xs, out)
    bad = ws.clone()
    bad[1, 1] = 255
    got = product(w, bad, x, xs, out)
    assert np.isnan(got[:, 128:256]).all()
    hg.same_bits(np.delete(got, range(128, 256), 1), np.delete(clean, range(128, 256), 1), "others")
    bad = xs.clone()
    bad[2, 0] = 255
    got = product(w, ws, x, bad, out)
    assert np.isnan(got[2]).all()
    hg.same_bits(np.delete(got, 2, 0), np.delete(clean, 2, 0), "others")
    x.view(torch.uint8)[1, 255] = 0x7F
    got = product(w, ws, x, xs, out)
    assert np.isnan(got[1]).all()
    hg.same_bits(np.delete(got, 1, 0), np.delete(clean, 1, 0), "others")


def test_product_of_nothing():
    rng = np.random.default_rng(1)
    w, ws, _ = operand(rng, 10, 128, TILE)
    y = torch.full((3, 10), 5.0, device=DEV)
    x, xs = w[:0], ws[:0]
    dh.dl_e4m3_matmul(w, ws, 10, 128, x, xs, 0, y)
    dh.dl_e4m3_matmul(w[:0], ws[:0], 0, 128, w, torch.zeros(10, 1, dtype=torch.uint8, device=DEV),
                      3, y)
    torch.cuda.synchronize()
    assert torch.all(y == 5)


def test_product_offsets_past_32_bits():
    """Rows of codes far apart, and a result whose last rows begin past 2^32 bytes."""
    rng = np.random.default_rng(2)
    rows, cols, count, ld = 600, 256, 40, 9_000_000
    w, ws, wv = operand(rng, rows, cols, TILE)
    x, xs, xv = operand(rng, count, cols, BLOCK)
    far = torch.empty(rows * ld, dtype=torch.uint8, device=DEV)
    fw = far.as_strided((rows, cols), (ld, 1))
    fw.copy_(w.view(torch.uint8))
    for out in ("f32", "bf16"):
        want = product(w, ws, x, xs, out)
        hg.same_bits(product(fw.view(torch.float8_e4m3fn), ws, x, xs, out), want, "far rows")
    ldy = 40_000_000
    y = torch.empty(count * ldy, device=DEV).as_strided((count, rows), (ldy, 1))
    dh.dl_e4m3_matmul(w, ws, rows, cols, x, xs, count, y)
    hg.same_bits(hg.host(y.contiguous()), product(w, ws, x, xs, "f32"), "far results")


def test_captured_product_replays():
    rng = np.random.default_rng(7)
    for count in (1, 30, 900):
        w, ws, _ = operand(rng, 5000, 400, TILE)
        x, xs, _ = operand(rng, count, 400, BLOCK)
        ys = [torch.empty(count, 5000, dtype=t, device=DEV) for t in (torch.float32, torch.bfloat16)]

        def step(out):
            for y in out:
                dh.dl_e4m3_matmul(w, ws, 5000, 400, x, xs, count, y)

        step(ys)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(ys)
        for _ in range(3):
            x2, xs2, _ = operand(rng, count, 400, BLOCK)
            x.copy_(x2)
            xs.copy_(xs2)
            g.replay()
            again = [torch.empty_like(y) for y in ys]
            step(again)
            torch.cuda.synchronize()
            for a, b in zip(ys, again):
                hg.same_bits(hg.bits(a), hg.bits(b), "replay")


def test_refusals_on_the_device():
    rng = np.random.default_rng(1)
    w, ws, _ = operand(rng, 200, 128, TILE)
    x, xs, _ = operand(rng, 8, 128, BLOCK)
    y = torch.empty(8, 200, device=DEV)
    with pytest.raises(ValueError):
        dh.dl_e4m3_matmul(w, ws[:1], 200, 128, x, xs, 8, y)
    with pytest.raises(TypeError):
        dh.dl_e4m3_matmul(w.view(torch.uint8).float(), ws, 200, 128, x, xs, 8, y)
    with pytest.raises(dl.DLError):
        dh.dl_e4m3_matmul(w, ws, 200, 128, x, xs, 8, w.data_ptr(), y_dtype=dl.DL_BF16)
    with pytest.raises(dl.DLError):
        dh.dl_e4m3_quantize(y, 8, 200, x.data_ptr(), y.data_ptr(), TILE)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("count", [32, 33, 128, 129, 192, 193, 257])
def test_product_about_its_forms(count, out):
    """Counts at which another form is taken, with rows enough for the largest tiles."""
    rng = np.random.default_rng(count)
    w, ws, wv = operand(rng, 33_000, 112, TILE)
    x, xs, xv = operand(rng, count, 112, BLOCK)
    check_product(product(w, ws, x, xs, out), wv, xv, out)


def test_product_straight_to_lds_past_32_bits():
    """Large tiles of rows 4 MB apart: offsets past 2^32 bytes on both sides."""
    rng = np.random.default_rng(3)
    rows, cols, count, ld = 4300, 128, 2100, 1 << 22
    w, ws, _ = operand(rng, rows, cols, TILE)
    x, xs, _ = operand(rng, count, cols, BLOCK)

    def far(t):
        f = torch.empty((len(t) - 1) * ld + cols, dtype=torch.uint8, device=DEV)
        f = f.as_strided((len(t), cols), (ld, 1))
        f.copy_(t.view(torch.uint8))
        return f.view(torch.float8_e4m3fn)

    fw, fx = far(w), far(x)
    for out in ("f32", "bf16"):
        hg.same_bits(product(fw, ws, fx, xs, out), product(w, ws, x, xs, out), "far rows")
