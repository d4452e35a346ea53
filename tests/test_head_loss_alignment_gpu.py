"""Every alignment and distance of rows gives the same results, bit for bit: log
probabilities without logits, their gradients, and 8-bit products.  What lies between rows,
and before the first, is NaN."""
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from tests import test_head_gpu as hg
from tests import test_head_loss_gpu as lg

pytestmark = pytest.mark.gpu

DEV = "cuda"


def placed(v, pad, offset):
    """v in rows `pad` elements further apart, the first `offset` elements into memory."""
    rows, cols = v.shape
    ld = cols + pad
    flat = torch.full((offset + (rows - 1) * ld + cols,), 255, dtype=torch.uint8, device=DEV)
    if v.dtype != torch.uint8:
        flat = torch.full(flat.shape, float("nan"), device=DEV).to(v.dtype)
    out = flat.as_strided((rows, cols), (ld, 1), offset)
    out.copy_(v)
    return out


def head(x, e, t, a, b, pad, offset):
    rows, vocab, width = x.shape[0], e.shape[0], x.shape[1]
    x, e = placed(x, pad, offset), placed(e, pad, offset)
    lp, h, st = (torch.empty(s, device=DEV) for s in ((rows,), (rows,), (rows, 2)))
    dx, de = torch.empty_like(x), placed(e, pad, offset)
    ws = lg.workspace(rows, vocab, width, "bf16" if x.dtype == torch.bfloat16 else "f32", True)
    dh.dl_head_logprobs(x, e, rows, vocab, width, t, lp, entropy=h, stats=st, workspace=ws)
    dh.dl_head_logprobs_backward(x, e, rows, vocab, width, t, st, a, dx=dx, dembed=de,
                                 entropy=None if b is None else h, dentropy=b, workspace=ws)
    torch.cuda.synchronize()
    return dict(logprobs=lp, entropy=h, stats=st, dx=dx, dembed=de)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("rows,vocab,width", [
    (1, 500, 200), (20, 500, 128), (40, 1000, 64), (200, 3000, 200), (300, 1000, 203),
    (300, 5000, 512), (300, 1000, 128), (513, 2001, 72), (1500, 700, 1001)])
def test_log_probabilities_and_gradients(rows, vocab, width, entropy, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows + width)
    new = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, e = new(rows, width).to(hg.TORCH[dtype]), (new(vocab, width) / width ** 0.5).to(hg.TORCH[dtype])
    t = torch.randint(-1, vocab, (rows,), generator=g, device=DEV)
    a, b = new(rows), new(rows) if entropy else None
    whole = -width % 8
    want = head(x, e, t, a, b, whole, 0)
    for pad, offset in ((whole + 8, 8), (1, 0), (whole, 1), (3, 3)):
        got = head(x, e, t, a, b, pad, offset)
        for name in want:
            hg.same_bits(hg.bits(got[name].contiguous()), hg.bits(want[name].contiguous()), name)


@pytest.mark.parametrize("ld", [4_000_000, 5_000_001])
def test_narrow_rows_far_apart(ld):
    """Offsets past 2^31 bytes from the first row, and rows too far apart to go to LDS straight."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    rows, vocab, width = 200, 400, 96
    x = torch.randn(rows, width, generator=g, device=DEV).bfloat16()
    e = (torch.randn(vocab, width, generator=g, device=DEV) / 10).bfloat16()
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    a = torch.randn(rows, generator=g, device=DEV)
    want = head(x, e, t, a, None, 0, 0)
    far = torch.empty((vocab - 1) * ld + width, dtype=torch.bfloat16, device=DEV)
    far = far.as_strided((vocab, width), (ld, 1))
    far.copy_(e)
    dx = torch.empty_like(x)
    dh.dl_head_logprobs_backward(x, far, rows, vocab, width, t, want["stats"], a, dx=dx,
                                 workspace=lg.workspace(rows, vocab, width, "bf16", True))
    hg.same_bits(hg.bits(dx), hg.bits(want["dx"]), "dx")


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,count", [(300, 384, 5), (300, 384, 40), (6000, 400, 1200),
                                             (300, 511, 200), (9000, 300, 20)])
def test_8_bit_products(rows, cols, count, out):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows)
    codes = lambda n: torch.randint(0, 0x7F, (n, cols), dtype=torch.uint8, generator=g,  # noqa: E731
                                    device=DEV)
    w, x, kb = codes(rows), codes(count), -(-cols // 128)
    ws = torch.full((-(-rows // 128), kb), 120, dtype=torch.uint8, device=DEV)
    xs = torch.full((count, kb), 121, dtype=torch.uint8, device=DEV)
    want = None
    for pad, offset in ((-cols % 16, 0), (16 - cols % 16, 16), (1, 0), (0, 1), (3, 3)):
        y = torch.empty(count, rows, dtype=out, device=DEV)
        dh.dl_e4m3_matmul(placed(w, pad, offset).view(torch.float8_e4m3fn), ws, rows, cols,
                          placed(x, pad, offset).view(torch.float8_e4m3fn), xs, count, y)
        want = y if want is None else want
        hg.same_bits(hg.bits(y), hg.bits(want), f"rows {pad} apart, {offset} in")
