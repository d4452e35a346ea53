"""The output head's C ABI on the CPU: exported names, argument rules that
are decided before any device work, the binding's own checks, and the oracle's
tables against their published definitions."""
import os
import re

import numpy as np
import pytest
import torch

from checkpoint_averaging_amd import dlhead as dh
from checkpoint_averaging_amd import dlmerge as dl
from oracle import head as oh

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "dlhead.h")
A = 0x7F0000000000        # never dereferenced: every call below fails before use


def _at(i):
    return A + (i << 32)


def test_library_exports_every_declared_function():
    text = open(HEADER).read()
    declared = sorted(set(re.findall(r"^int (dl_\w+)\(", text, re.M)))
    assert sorted(dh.SYMBOLS) == declared
    for name in declared:
        assert hasattr(dl.raw_lib(), name), name
    for name in ("DL_E4M3", "DL_SCALE_NONE", "DL_SCALE_ROW", "DL_SCALE_BLOCK32"):
        m = re.search(rf"\b{name} = (\d+)", text)
        assert m and int(m.group(1)) == getattr(dh, name)
    for name in ("DL_MAX_NORM_COLS", "DL_MAX_VECTORS", "DL_MAX_TOP"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(dh, name)


def _refused(status, fn, *a, **k):
    with pytest.raises(dl.DLError) as ei:
        fn(*a, **k)
    assert ei.value.status == status, (ei.value.status, status)


NORM = dict(x=_at(0), rows=4, cols=100, weight=_at(1), y=_at(2), eps=1e-5, dtype=dl.DL_BF16,
            y_dtype=dl.DL_BF16, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), dl.DL_E_INVAL),
    (dict(weight=None), dl.DL_E_INVAL),
    (dict(y=None), dl.DL_E_INVAL),
    (dict(rows=-1), dl.DL_E_INVAL),
    (dict(rows=1 << 31), dl.DL_E_INVAL),
    (dict(cols=0), dl.DL_E_INVAL),
    (dict(cols=dh.DL_MAX_NORM_COLS + 1), dl.DL_E_INVAL),
    (dict(eps=-1.0), dl.DL_E_INVAL),
    (dict(eps=float("nan")), dl.DL_E_INVAL),
    (dict(eps=float("inf")), dl.DL_E_INVAL),
    (dict(ldx=99), dl.DL_E_INVAL),
    (dict(ldy=99), dl.DL_E_INVAL),
    (dict(ldx=1 << 62), dl.DL_E_INVAL),                                  # past 64 bits
    (dict(dtype=2), dl.DL_E_INVAL),
    (dict(dtype=7), dl.DL_E_INVAL),
    (dict(y_dtype=3), dl.DL_E_INVAL),
    (dict(y_dtype=dh.DL_E4M3), dl.DL_E_INVAL),                           # without scales
    (dict(y_dtype=dh.DL_E4M3, scale_kind=dh.DL_SCALE_ROW), dl.DL_E_INVAL),
    (dict(y_dtype=dh.DL_E4M3, scale_kind=3, scales=_at(4)), dl.DL_E_INVAL),
    (dict(scale_kind=dh.DL_SCALE_ROW, scales=_at(4)), dl.DL_E_INVAL),    # bf16 has none
    (dict(scales=_at(4)), dl.DL_E_INVAL),
    (dict(sum_=_at(5)), dl.DL_E_INVAL),                                  # without a residual
    (dict(x=_at(0) + 1), dl.DL_E_ALIGN),
    (dict(weight=_at(1) + 2), dl.DL_E_ALIGN),
    (dict(inv_rms=_at(6) + 2), dl.DL_E_ALIGN),
    (dict(y_dtype=dh.DL_E4M3, scale_kind=dh.DL_SCALE_ROW, scales=_at(4) + 2), dl.DL_E_ALIGN),
    (dict(y=_at(0)), dl.DL_E_INVAL),                                     # y over x
    (dict(y=_at(1)), dl.DL_E_INVAL),                                     # y over weight
    (dict(y=_at(0) + 2 * 100, ldx=200, ldy=200), dl.DL_E_INVAL),         # interleaved spans
    (dict(residual=_at(3), sum_=_at(3) + 2), dl.DL_E_INVAL),             # shifted over residual
    (dict(residual=_at(3), sum_=_at(3), ldres=104), dl.DL_E_INVAL),      # other leading dimension
    (dict(residual=_at(3), sum_=_at(2)), dl.DL_E_INVAL),                 # sum over y
    (dict(inv_rms=_at(2)), dl.DL_E_INVAL),                               # inv_rms over y
])
def test_rmsnorm_refuses(kw, status):
    _refused(status, dh.dl_rmsnorm, **{**NORM, **kw})


NORM_B = dict(dy=_at(0), sum_=_at(1), rows=4, cols=100, weight=_at(2), inv_rms=_at(3), dx=_at(4),
              dweight=_at(5), workspace=_at(6), workspace_bytes=1 << 30, dtype=dl.DL_F32, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), dl.DL_E_INVAL),
    (dict(sum_=None), dl.DL_E_INVAL),
    (dict(weight=None), dl.DL_E_INVAL),
    (dict(inv_rms=None), dl.DL_E_INVAL),
    (dict(dx=None), dl.DL_E_INVAL),
    (dict(cols=0), dl.DL_E_INVAL),
    (dict(rows=-2), dl.DL_E_INVAL),
    (dict(dtype=dh.DL_E4M3), dl.DL_E_INVAL),
    (dict(lddx=50), dl.DL_E_INVAL),
    (dict(dx=_at(1)), dl.DL_E_INVAL),                                    # dx over sum
    (dict(dx=_at(0) + 4), dl.DL_E_INVAL),                                # shifted over dy
    (dict(dweight=_at(2)), dl.DL_E_INVAL),
    (dict(dweight=_at(5) + 1), dl.DL_E_ALIGN),
    (dict(dy=_at(0) + 2), dl.DL_E_ALIGN),
])
def test_rmsnorm_backward_refuses(kw, status):
    _refused(status, dh.dl_rmsnorm_backward, **{**NORM_B, **kw})


def test_rmsnorm_backward_needs_its_workspace():
    need = dh.dl_rmsnorm_workspace_bytes(4096, 2048)
    args = {**NORM_B, "rows": 4096, "cols": 2048}
    if need > 0:
        _refused(dl.DL_E_INVAL, dh.dl_rmsnorm_backward, **{**args, "workspace_bytes": need - 1})
        _refused(dl.DL_E_INVAL, dh.dl_rmsnorm_backward, **{**args, "workspace": None})
        _refused(dl.DL_E_ALIGN, dh.dl_rmsnorm_backward, **{**args, "workspace": _at(6) + 128})
        _refused(dl.DL_E_INVAL, dh.dl_rmsnorm_backward, **{**args, "workspace": _at(5)})
    _refused(dl.DL_E_INVAL, dh.dl_rmsnorm_workspace_bytes, -1, 5)
    _refused(dl.DL_E_INVAL, dh.dl_rmsnorm_workspace_bytes, 5, 0)


QUANT = dict(w=_at(0), rows=4, cols=100, packed=_at(1), scales=_at(2), values=_at(3),
             dtype=dl.DL_F32, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), dl.DL_E_INVAL),
    (dict(packed=None), dl.DL_E_INVAL),
    (dict(scales=None), dl.DL_E_INVAL),
    (dict(cols=0), dl.DL_E_INVAL),
    (dict(rows=-1), dl.DL_E_INVAL),
    (dict(cols=1 << 31), dl.DL_E_INVAL),
    (dict(dtype=dh.DL_E4M3), dl.DL_E_INVAL),
    (dict(ldw=99), dl.DL_E_INVAL),
    (dict(ldvalues=99), dl.DL_E_INVAL),
    (dict(packed=_at(1) + 8), dl.DL_E_ALIGN),
    (dict(w=_at(0) + 2), dl.DL_E_ALIGN),
    (dict(packed=_at(0)), dl.DL_E_INVAL),
    (dict(scales=_at(1)), dl.DL_E_INVAL),
    (dict(values=_at(0) + 4), dl.DL_E_INVAL),
    (dict(values=_at(0), ldvalues=101), dl.DL_E_INVAL),
])
def test_quantize_refuses(kw, status):
    _refused(status, dh.dl_w4_quantize, **{**QUANT, **kw})


MATVEC = dict(packed=_at(0), scales=_at(1), rows=64, cols=100, x=_at(2), count=3, y=_at(3),
              x_dtype=dl.DL_BF16, y_dtype=dl.DL_F32, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(packed=None), dl.DL_E_INVAL),
    (dict(scales=None), dl.DL_E_INVAL),
    (dict(x=None), dl.DL_E_INVAL),
    (dict(y=None), dl.DL_E_INVAL),
    (dict(count=0), dl.DL_E_INVAL),
    (dict(count=dh.DL_MAX_VECTORS + 1), dl.DL_E_INVAL),
    (dict(cols=0), dl.DL_E_INVAL),
    (dict(rows=-1), dl.DL_E_INVAL),
    (dict(x_dtype=dl.DL_F32), dl.DL_E_INVAL),
    (dict(y_dtype=dh.DL_E4M3), dl.DL_E_INVAL),
    (dict(x_dtype=dh.DL_E4M3), dl.DL_E_INVAL),
    (dict(x_dtype=dh.DL_E4M3, x_scale_kind=dh.DL_SCALE_ROW), dl.DL_E_INVAL),
    (dict(x_scale_kind=dh.DL_SCALE_ROW, x_scales=_at(4)), dl.DL_E_INVAL),
    (dict(ldx=99), dl.DL_E_INVAL),
    (dict(ldy=63), dl.DL_E_INVAL),
    (dict(packed=_at(0) + 4), dl.DL_E_ALIGN),
    (dict(x=_at(2) + 1), dl.DL_E_ALIGN),
    (dict(y=_at(3) + 2), dl.DL_E_ALIGN),
    (dict(x_dtype=dh.DL_E4M3, x_scale_kind=dh.DL_SCALE_ROW, x_scales=_at(4) + 1), dl.DL_E_ALIGN),
    (dict(y=_at(0)), dl.DL_E_INVAL),
    (dict(y=_at(2)), dl.DL_E_INVAL),
])
def test_matvec_refuses(kw, status):
    _refused(status, dh.dl_w4_matvec, **{**MATVEC, **kw})


LOGP = dict(logits=_at(0), rows=5, vocab=100, targets=_at(1), logprobs=_at(2), entropy=_at(3),
            stats=_at(4), top_k=4, top_ids=_at(5), top_logprobs=_at(6), workspace=_at(7),
            workspace_bytes=1 << 30, dtype=dl.DL_F32, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), dl.DL_E_INVAL),
    (dict(vocab=0), dl.DL_E_INVAL),
    (dict(vocab=1 << 31), dl.DL_E_INVAL),
    (dict(rows=-1), dl.DL_E_INVAL),
    (dict(dtype=dh.DL_E4M3), dl.DL_E_INVAL),
    (dict(ldl=99), dl.DL_E_INVAL),
    (dict(targets=None), dl.DL_E_INVAL),                                 # log probs of what?
    (dict(logprobs=None), dl.DL_E_INVAL),
    (dict(top_k=-1), dl.DL_E_INVAL),
    (dict(top_k=dh.DL_MAX_TOP + 1), dl.DL_E_INVAL),
    (dict(top_k=4, vocab=3), dl.DL_E_INVAL),
    (dict(top_k=0), dl.DL_E_INVAL),                                      # arrays without a count
    (dict(top_ids=None), dl.DL_E_INVAL),
    (dict(top_logprobs=None), dl.DL_E_INVAL),
    (dict(logits=_at(0) + 2), dl.DL_E_ALIGN),
    (dict(targets=_at(1) + 4), dl.DL_E_ALIGN),
    (dict(top_ids=_at(5) + 4), dl.DL_E_ALIGN),
    (dict(logprobs=_at(0)), dl.DL_E_INVAL),
    (dict(entropy=_at(2)), dl.DL_E_INVAL),
    (dict(stats=_at(3)), dl.DL_E_INVAL),
    (dict(top_logprobs=_at(5)), dl.DL_E_INVAL),
])
def test_logprobs_refuses(kw, status):
    _refused(status, dh.dl_logprobs, **{**LOGP, **kw})


def test_logprobs_needs_its_workspace():
    need = dh.dl_logprobs_workspace_bytes(1, 73760, 8)
    args = {**LOGP, "rows": 1, "vocab": 73760, "top_k": 8}
    if need > 0:
        _refused(dl.DL_E_INVAL, dh.dl_logprobs, **{**args, "workspace_bytes": need - 1})
        _refused(dl.DL_E_INVAL, dh.dl_logprobs, **{**args, "workspace": None})
        _refused(dl.DL_E_ALIGN, dh.dl_logprobs, **{**args, "workspace": _at(7) + 8})
        _refused(dl.DL_E_INVAL, dh.dl_logprobs, **{**args, "workspace": _at(0)})
    _refused(dl.DL_E_INVAL, dh.dl_logprobs_workspace_bytes, 1, 0, 0)
    _refused(dl.DL_E_INVAL, dh.dl_logprobs_workspace_bytes, 1, 5, 6)


LOGP_B = dict(logits=_at(0), rows=5, vocab=100, targets=_at(1), stats=_at(2), dlogprobs=_at(3),
              dlogits=_at(4), entropy=_at(5), dentropy=_at(6), dtype=dl.DL_BF16, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), dl.DL_E_INVAL),
    (dict(targets=None), dl.DL_E_INVAL),
    (dict(stats=None), dl.DL_E_INVAL),
    (dict(dlogprobs=None), dl.DL_E_INVAL),
    (dict(dlogits=None), dl.DL_E_INVAL),
    (dict(entropy=None), dl.DL_E_INVAL),
    (dict(dentropy=None), dl.DL_E_INVAL),
    (dict(dtype=dh.DL_E4M3), dl.DL_E_INVAL),
    (dict(lddl=99), dl.DL_E_INVAL),
    (dict(dlogits=_at(0) + 2), dl.DL_E_INVAL),
    (dict(dlogits=_at(2)), dl.DL_E_INVAL),
    (dict(stats=_at(2) + 2), dl.DL_E_ALIGN),
])
def test_logprobs_backward_refuses(kw, status):
    _refused(status, dh.dl_logprobs_backward, **{**LOGP_B, **kw})


def test_no_rows_is_no_work():
    """rows = 0 returns before any device is asked for."""
    dh.dl_rmsnorm(**{**NORM, "rows": 0})
    dh.dl_w4_quantize(**{**QUANT, "rows": 0})
    dh.dl_w4_matvec(**{**MATVEC, "rows": 0})
    dh.dl_logprobs(**{**LOGP, "rows": 0})
    dh.dl_logprobs_backward(**{**LOGP_B, "rows": 0})
    dh.dl_rmsnorm_backward(**{**NORM_B, "rows": 0, "dweight": None})
    assert dh.dl_logprobs_workspace_bytes(0, 10, 2) == 0


def test_w4_bytes():
    assert dh.dl_w4_bytes(0, 1) == (0, 0)
    assert dh.dl_w4_bytes(3, 1) == (48, 3)
    assert dh.dl_w4_bytes(73760, 2048) == (73760 * 1024, 73760 * 64)
    assert dh.dl_w4_bytes(5, 33) == (160, 10)
    _refused(dl.DL_E_INVAL, dh.dl_w4_bytes, 5, 0)
    _refused(dl.DL_E_INVAL, dh.dl_w4_bytes, -1, 5)


def test_binding_refuses_host_tensors():
    t = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        dh.dl_rmsnorm(t, 4, 8, torch.zeros(8), torch.zeros(4, 8))
    with pytest.raises(TypeError):
        dh.dl_rmsnorm(_at(0), 4, 8, _at(1), _at(2))              # raw address without a type


# ---- the oracle's own definitions ------------------------------------------


def test_oracle_e4m3_table():
    """The format's corner values: largest 448, smallest normal 2^-6, smallest
    subnormal 2^-9, 127 is NaN; and torch's own conversion, value by value."""
    v = oh.e4m3_value(np.arange(256, dtype=np.uint8))
    assert v[126] == 448 and v[8] == 2.0 ** -6 and v[1] == 2.0 ** -9 and np.isnan(v[127])
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float()
    assert np.array_equal(v, t.numpy().astype(np.float64), equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 20001), np.ldexp(np.linspace(1, 2, 99), -10)])
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oh.e4m3_code(x.astype(np.float32)), want)


def test_oracle_bf16_rounding():
    x = np.random.default_rng(0).standard_normal(5000).astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(oh.bf16_bits(x), want)


def test_oracle_w4_roundings_by_hand():
    """One block whose largest element is 6 (b = 1): ties go to the even code."""
    w = np.zeros((1, 32), np.float32)
    w[0, :12] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.26, -5.1, 0.74, -0.0]
    packed, e, values = oh.w4_quantize(w)
    assert e[0, 0] == 127
    assert values[0, :12].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -0.5, -6, 0.5, 0]
    code = np.stack([packed & 15, packed >> 4], 2).reshape(-1)[:12]
    assert code.tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 9, 15, 1, 8]
    w[0, 0] = np.nextafter(np.float32(6), np.float32(7))         # one step over: b = 2
    assert oh.w4_quantize(w)[1][0, 0] == 128
    assert np.array_equal(oh.w4_values(packed, e, 32)[0, :11], values[0, :11])


def test_oracle_log_softmax_of_a_nearly_certain_token():
    x = np.full((1, 4), 0.0)
    x[0, 2] = 40.0
    lp, h, m, ls = oh.log_softmax(x)
    rest = 3 * np.exp(-40.0)
    assert abs(lp[0, 2] + rest) < 1e-3 * rest and m[0] == 40
    assert abs(h[0] - rest * 41) < 1e-3 * rest * 41


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((2, 7))
    t = np.array([3, 1])
    gl, gh = rng.standard_normal(2), rng.standard_normal(2)

    def f(x):
        lp, h, _, _ = oh.log_softmax(x)
        return float((gl * lp[[0, 1], t] + gh * h).sum())

    lp, h, _, _ = oh.log_softmax(x)
    d = oh.logprobs_backward(lp, h, t, gl, gh)
    for r in range(2):
        for c in range(7):
            e = np.zeros_like(x)
            e[r, c] = 1e-5
            assert abs((f(x + e) - f(x - e)) / 2e-5 - d[r, c]) < 1e-8
    s, w, dy = rng.standard_normal((3, 6)), rng.standard_normal(6), rng.standard_normal((3, 6))
    ds = rng.standard_normal((3, 6))

    def g(s, w):
        inv = 1 / np.sqrt((s * s).mean(1) + 1e-5)
        return float((dy * (s * inv[:, None] * w)).sum() + (ds * s).sum())

    inv = 1 / np.sqrt((s * s).mean(1) + 1e-5)
    dx, dw = oh.norm_backward(dy, ds, s, inv, w)
    for i in np.ndindex(3, 6):
        e = np.zeros_like(s)
        e[i] = 1e-5
        assert abs((g(s + e, w) - g(s - e, w)) / 2e-5 - dx[i]) < 1e-8
    for c in range(6):
        e = np.zeros(6)
        e[c] = 1e-5
        assert abs((g(s, w + e) - g(s, w - e)) / 2e-5 - dw[c]) < 1e-8
