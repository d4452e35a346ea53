"""The host rules of the calls over whole probes (log probabilities without logits, 8-bit
matrices) and of the objects that make them, on the CPU: refusals that are decided before any
device work, workspace sizes, and recorded calls."""
import numpy as np
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from checkpoint_averaging_amd import dlmerge as dl
from checkpoint_averaging_amd import synth
from checkpoint_averaging_amd.head import Head, LossHead
from oracle import head as oh

A = 0x7F0000000000        # never dereferenced: every call below fails before use


def _at(i):
    return A + (i << 36)


def _refused(status, fn, *a, **k):
    with pytest.raises(dl.DLError) as ei:
        fn(*a, **k)
    assert ei.value.status == status, (ei.value.status, status)


FORWARD = dict(x=_at(0), embed=_at(1), rows=4, vocab=100, width=32, targets=_at(2),
               logprobs=_at(3), entropy=_at(4), stats=_at(5), workspace=_at(6),
               workspace_bytes=1 << 30, dtype=dl.DL_BF16, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), dl.DL_E_INVAL),
    (dict(embed=None), dl.DL_E_INVAL),
    (dict(rows=-1), dl.DL_E_INVAL),
    (dict(rows=(1 << 30) + 1, workspace_bytes=1 << 60), dl.DL_E_INVAL),
    (dict(vocab=0), dl.DL_E_INVAL),
    (dict(vocab=(1 << 30) + 1, workspace_bytes=1 << 60), dl.DL_E_INVAL),
    (dict(width=0), dl.DL_E_INVAL),
    (dict(width=dh.DL_MAX_NORM_COLS + 1, ldx=1 << 20, lde=1 << 20), dl.DL_E_INVAL),
    (dict(rows=1 << 22, vocab=(1 << 21) + 1, workspace_bytes=1 << 60), dl.DL_E_INVAL),
    (dict(dtype=dh.DL_E4M3), dl.DL_E_INVAL),
    (dict(dtype=5), dl.DL_E_INVAL),
    (dict(ldx=31), dl.DL_E_INVAL),
    (dict(lde=31), dl.DL_E_INVAL),
    (dict(lde=1 << 62), dl.DL_E_INVAL),
    (dict(targets=None), dl.DL_E_INVAL),                                 # logprobs without
    (dict(logprobs=None), dl.DL_E_INVAL),
    (dict(workspace=None), dl.DL_E_INVAL),
    (dict(workspace_bytes=64), dl.DL_E_INVAL),
    (dict(workspace=_at(6) + 128), dl.DL_E_ALIGN),
    (dict(x=_at(0) + 1), dl.DL_E_ALIGN),
    (dict(targets=_at(2) + 4), dl.DL_E_ALIGN),
    (dict(entropy=_at(4) + 2), dl.DL_E_ALIGN),
    (dict(workspace=_at(0)), dl.DL_E_INVAL),
    (dict(entropy=_at(3)), dl.DL_E_INVAL),
    (dict(stats=_at(1)), dl.DL_E_INVAL),
])
def test_forward_refuses(kw, status):
    _refused(status, dh.dl_head_logprobs, **{**FORWARD, **kw})


BACKWARD = dict(x=_at(0), embed=_at(1), rows=4, vocab=100, width=32, targets=_at(2), stats=_at(5),
                dlogprobs=_at(3), dx=_at(7), dembed=_at(8), workspace=_at(6),
                workspace_bytes=1 << 32, dtype=dl.DL_F32, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), dl.DL_E_INVAL),
    (dict(embed=None), dl.DL_E_INVAL),
    (dict(targets=None), dl.DL_E_INVAL),
    (dict(stats=None), dl.DL_E_INVAL),
    (dict(dlogprobs=None), dl.DL_E_INVAL),
    (dict(dx=None, dembed=None), dl.DL_E_INVAL),                         # nothing asked for
    (dict(entropy=_at(4)), dl.DL_E_INVAL),                               # without its gradient
    (dict(dentropy=_at(4)), dl.DL_E_INVAL),
    (dict(workspace=None), dl.DL_E_INVAL),
    (dict(workspace_bytes=1 << 10), dl.DL_E_INVAL),
    (dict(lddx=31), dl.DL_E_INVAL),
    (dict(ldde=31), dl.DL_E_INVAL),
    (dict(dx=_at(0)), dl.DL_E_INVAL),                                    # over an input
    (dict(dembed=_at(1)), dl.DL_E_INVAL),
    (dict(dx=_at(8)), dl.DL_E_INVAL),
    (dict(dx=_at(7) + 2), dl.DL_E_ALIGN),
    (dict(dtype=dh.DL_E4M3), dl.DL_E_INVAL),
])
def test_backward_refuses(kw, status):
    _refused(status, dh.dl_head_logprobs_backward, **{**BACKWARD, **kw})


def test_workspace():
    """With the backward pass never less than without; no more than a few pieces of the
    vocabulary whatever its size, beside what goes with the rows."""
    for rows, vocab, width in [(1, 1, 1), (32, 73760, 2048), (33, 73760, 2048), (2048, 73760, 2048),
                               (8191, 50304, 128), (16384, 150_000, 4096)]:
        for dtype in (torch.float32, torch.bfloat16):
            fwd = dh.dl_head_workspace_bytes(rows, vocab, width, dtype)
            both = dh.dl_head_workspace_bytes(rows, vocab, width, dtype, backward=True)
            assert 0 < fwd <= both
            size = 4 if dtype == torch.float32 else 2
            assert both <= (640 << 20) + rows * width * (size + 4 * 16) + rows * vocab // 2
    assert dh.dl_head_workspace_bytes(0, 5, 5, torch.float32, True) == 0
    with pytest.raises(dl.DLError):
        dh.dl_head_workspace_bytes(4, 5, 0, torch.float32)
    with pytest.raises(dl.DLError):
        dh.dl_head_workspace_bytes(4, 5, 5, dh.DL_E4M3)


QUANT = dict(x=_at(0), rows=4, cols=100, codes=_at(1), scales=_at(2),
             scale_kind=dh.DL_SCALE_TILE128, values=_at(3), dtype=dl.DL_F32, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), dl.DL_E_INVAL),
    (dict(codes=None), dl.DL_E_INVAL),
    (dict(scales=None), dl.DL_E_INVAL),
    (dict(scale_kind=dh.DL_SCALE_ROW), dl.DL_E_INVAL),
    (dict(scale_kind=dh.DL_SCALE_BLOCK32), dl.DL_E_INVAL),
    (dict(scale_kind=dh.DL_SCALE_NONE), dl.DL_E_INVAL),
    (dict(rows=-1), dl.DL_E_INVAL),
    (dict(cols=0), dl.DL_E_INVAL),
    (dict(ldx=99), dl.DL_E_INVAL),
    (dict(ldc=99), dl.DL_E_INVAL),
    (dict(ldvalues=99), dl.DL_E_INVAL),
    (dict(dtype=dh.DL_E4M3), dl.DL_E_INVAL),
    (dict(x=_at(0) + 2), dl.DL_E_ALIGN),
    (dict(codes=_at(0)), dl.DL_E_INVAL),
    (dict(scales=_at(1)), dl.DL_E_INVAL),
    (dict(values=_at(0) + 4), dl.DL_E_INVAL),
])
def test_quantize_refuses(kw, status):
    _refused(status, dh.dl_e4m3_quantize, **{**QUANT, **kw})


MATMUL = dict(w=_at(0), w_scales=_at(1), rows=200, cols=100, x=_at(2), x_scales=_at(3), count=5,
              y=_at(4), y_dtype=dl.DL_BF16, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), dl.DL_E_INVAL),
    (dict(w_scales=None), dl.DL_E_INVAL),
    (dict(x=None), dl.DL_E_INVAL),
    (dict(x_scales=None), dl.DL_E_INVAL),
    (dict(y=None), dl.DL_E_INVAL),
    (dict(rows=-1), dl.DL_E_INVAL),
    (dict(count=-1), dl.DL_E_INVAL),
    (dict(cols=0), dl.DL_E_INVAL),
    (dict(count=(1 << 30) + 1), dl.DL_E_INVAL),
    (dict(cols=(1 << 30) + 1, ldw=1 << 31, ldx=1 << 31), dl.DL_E_INVAL),
    (dict(rows=(1 << 30) + 1, ldy=1 << 31), dl.DL_E_INVAL),
    (dict(rows=1 << 22, count=(1 << 21) + 1, ldy=1 << 22), dl.DL_E_INVAL),
    (dict(ldw=99), dl.DL_E_INVAL),
    (dict(ldx=99), dl.DL_E_INVAL),
    (dict(ldy=199), dl.DL_E_INVAL),
    (dict(y_dtype=dh.DL_E4M3), dl.DL_E_INVAL),
    (dict(y=_at(4) + 1), dl.DL_E_ALIGN),
    (dict(y=_at(0)), dl.DL_E_INVAL),
    (dict(y=_at(3)), dl.DL_E_INVAL),
])
def test_matmul_refuses(kw, status):
    _refused(status, dh.dl_e4m3_matmul, **{**MATMUL, **kw})


def test_norm_refuses_a_tile_scale():
    norm = dict(x=_at(0), rows=4, cols=100, weight=_at(1), y=_at(2), dtype=dl.DL_BF16,
                y_dtype=dh.DL_E4M3, scales=_at(4), stream=0)
    _refused(dl.DL_E_INVAL, dh.dl_rmsnorm, scale_kind=dh.DL_SCALE_TILE128, **norm)
    _refused(dl.DL_E_INVAL, dh.dl_rmsnorm, scale_kind=dh.DL_SCALE_BLOCK128,
             **{**norm, "scales": None})
    _refused(dl.DL_E_INVAL, dh.dl_rmsnorm, scale_kind=dh.DL_SCALE_BLOCK128,
             **{**norm, "y_dtype": dl.DL_BF16})


def test_oracle_of_tile_scales():
    """The smallest power of two with amax <= 448 b, over a sweep of magnitudes."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((300, 700)) * 10.0 ** rng.integers(-40, 38, (300, 1))).astype(np.float32)
    for high in (1, 128):
        e = oh.tile_bytes(x, high)
        for i in range(e.shape[0]):
            for j in range(e.shape[1]):
                amax = np.abs(x[i * high:(i + 1) * high, j * 128:(j + 1) * 128]).max().astype(np.float64)
                assert amax <= 448 * 2.0 ** (int(e[i, j]) - 127)
                assert e[i, j] == 0 or amax > 448 * 2.0 ** (int(e[i, j]) - 128)
    assert oh.tile_bytes(np.full((1, 1), 448.0, np.float32), 1)[0, 0] == 127
    codes, e, v = oh.e4m3_quantize(x, 128)
    b = oh.tile_spread(e, x.shape, 128)
    assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, b * 2.0 ** -10) * (1 + 1e-9)).all()


# --------------------------------------------------------------------------
# The objects: the library's calls replaced by ones that record their arguments
# --------------------------------------------------------------------------

WIDTH, VOCAB = 96, 1000
LAYOUT = synth.Layout("small", (("embed", VOCAB * WIDTH), ("final_norm.weight", WIDTH)))


@pytest.fixture
def calls(monkeypatch):
    made = []

    def record(module, name):
        monkeypatch.setattr(module, name, lambda *a, **k: made.append((name, a, k)))

    record(dl, "dl_matmul_f32")
    for name in ("dl_rmsnorm", "dl_rmsnorm_backward", "dl_w4_quantize", "dl_w4_matvec",
                 "dl_logprobs", "dl_e4m3_quantize", "dl_e4m3_matmul", "dl_head_logprobs",
                 "dl_head_logprobs_backward"):
        record(dh, name)
    return made


def test_answer_goes_by_what_was_published_last(calls):
    head = Head(LAYOUT, torch.zeros(LAYOUT.n_params), max_rows=80)
    x = torch.zeros(70, WIDTH)
    with pytest.raises(RuntimeError):
        head.answer(x)
    with pytest.raises(ValueError):
        head.publish(bits=5)
    with pytest.raises(RuntimeError):
        head.answer(x)
    four = ["dl_rmsnorm", "dl_w4_matvec", "dl_w4_matvec", "dl_w4_matvec", "dl_logprobs"]
    eight = ["dl_rmsnorm", "dl_e4m3_matmul", "dl_logprobs"]
    for bits, want in ((8, eight), (4, four), (8, eight), (8, eight)):
        head.publish(bits=bits)
        calls.clear()
        head.answer(x)
        assert [name for name, _, _ in calls] == want
    codes = head._codes
    head.publish(bits=8)
    assert head._codes is codes                                  # in place: graphs keep its address


def test_loss_head_keeps_its_buffers(calls):
    head = LossHead.of(LAYOUT, torch.zeros(LAYOUT.n_params), max_rows=500)
    assert head.weight.data_ptr() == head.embed.data_ptr() + 4 * VOCAB * WIDTH
    for rows in (3, 500, 40):
        x, t = torch.zeros(rows, WIDTH), torch.zeros(rows, dtype=torch.int64)
        head.score(x, None, t)
        head.backward(x, t, torch.zeros(rows), x.clone(), dembed=torch.zeros(VOCAB, WIDTH))
        need = dh.dl_head_workspace_bytes(rows, VOCAB, WIDTH, torch.float32, True)
        assert head._ws.numel() >= need
        assert head._norm_ws.numel() >= dh.dl_rmsnorm_workspace_bytes(rows, WIDTH)
    made = [k["workspace"].data_ptr() for name, _, k in calls if name.startswith("dl_head_")]
    assert len(made) == 6 and len(set(made)) == 1
    assert [name for name, _, _ in calls[:4]] == ["dl_rmsnorm", "dl_head_logprobs",
                                                  "dl_head_logprobs_backward",
                                                  "dl_rmsnorm_backward"]


def test_loss_head_refuses(calls):
    w, e = torch.ones(WIDTH), torch.zeros(VOCAB, WIDTH)
    for bad in (dict(weight=w[:-1]), dict(weight=w.bfloat16()), dict(embed=e.half()),
                dict(embed=e[0]), dict(max_rows=0)):
        with pytest.raises(ValueError):
            LossHead(**{**dict(weight=w, embed=e, max_rows=4), **bad})
    with pytest.raises(ValueError):
        LossHead.of(synth.PYTHIA_14M, torch.zeros(8), 4)         # layer norms, untied
    head = LossHead(w, e.bfloat16(), 4)
    t = torch.zeros(4, dtype=torch.int64)
    for x in (torch.zeros(5, WIDTH), torch.zeros(4, WIDTH - 1), torch.zeros(WIDTH)):
        with pytest.raises(ValueError):
            head.score(x)
        with pytest.raises(ValueError):
            head.backward(x.bfloat16(), t, torch.zeros(4), x)
    with pytest.raises(ValueError):
        head.backward(torch.zeros(4, WIDTH), t, torch.zeros(4), torch.zeros(4, WIDTH))
    assert not calls


@pytest.mark.parametrize("kind", [dh.DL_SCALE_TILE128, dh.DL_SCALE_BLOCK128, 5, -1])
def test_4_bit_product_refuses_scales_of_128(kind):
    w4 = dict(packed=_at(0), scales=_at(1), rows=4, cols=256, x=_at(2), count=2, y=_at(3),
              x_scales=_at(4), ldx=256, ldy=4, x_dtype=dh.DL_E4M3, y_dtype=dl.DL_F32, stream=0)
    _refused(dl.DL_E_INVAL, dh.dl_w4_matvec, x_scale_kind=kind, **w4)
