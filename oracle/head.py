"""Plain numpy oracle of the output head: norm, 4-bit matrices, log
probabilities and their gradients, from the definitions.

Steps that the calls define operation by operation (what is rounded to 8 or 4
bits, power-of-two scales) are formed with the same single roundings and give
bits; sums and softmax are in binary64.
"""
from __future__ import annotations

import numpy as np

F32, F64 = np.float32, np.float64
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], F64)


def bf16_bits(x):
    """binary32 -> bfloat16 bits, nearest, ties to even (NaN stays NaN)."""
    b = np.ascontiguousarray(x, F32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_value(bits):
    return (bits.astype(np.uint32) << 16).view(F32)


def round_to(x, dtype):
    """Values of binary32 `x` rounded to "f32" or "bf16"."""
    return x.astype(F32) if dtype == "f32" else bf16_value(bf16_bits(x))


def e4m3_value(code):
    code = code.astype(np.int64)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((code & 127) == 127, np.nan, v)
    return np.where(code & 128, -v, v)


_E4M3 = e4m3_value(np.arange(127, dtype=np.uint8))       # the magnitudes, ascending


def _nearest(mag, table):
    """Index of the nearest entry of an ascending table, ties to the even index."""
    hi = np.clip(np.searchsorted(table, mag), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = mag - table[lo], table[hi] - mag
    return np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))


def e4m3_code(x):
    """Codes of binary32 values up to about 448, nearest, ties to even."""
    x = np.asarray(x, F64)
    return (_nearest(np.abs(x), _E4M3) | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)


def scale_value(byte):
    b = byte.astype(F64)
    return np.where(byte == 255, np.nan, 2.0 ** (b - 127))


def _blocks(y):
    """rows x kb x 32, padded with zeros."""
    rows, cols = y.shape
    kb = -(-cols // 32)
    p = np.zeros((rows, kb * 32), y.dtype)
    p[:, :cols] = y
    return p.reshape(rows, kb, 32)


def block_bytes(y, most):
    """Exponent byte of each 32 columns: the smallest power of two b >= 2^-127
    with amax <= most * b; 255 where the block holds a NaN or infinity."""
    a = np.abs(_blocks(y).astype(F64))
    amax = a.max(axis=2)
    ok = np.isfinite(a).all(axis=2)
    out = np.full(amax.shape, 255, np.uint8)
    for i in zip(*np.nonzero(ok)):
        e = 0
        if amax[i] > 0:
            e = max(0, int(np.floor(np.log2(amax[i]))) - int(np.log2(most)) - 1 + 127)
        while amax[i] > most * 2.0 ** (e - 127):
            e += 1
        out[i] = e
    return out


def norm_inv(s, eps):
    """1/sqrt(mean s^2 + eps) in binary64 (the call rounds it to binary32)."""
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        return 1.0 / np.sqrt((s.astype(F64) ** 2).mean(axis=1) + F64(F32(eps)))


def norm_values(s, inv32, weight):
    with np.errstate(invalid="ignore", over="ignore"):
        return (s.astype(F32) * inv32.astype(F32)[:, None]) * weight.astype(F32)


def e4m3_rows(y):
    """(codes, fp32 scales) with one scale a row."""
    amax = np.abs(y).max(axis=1).astype(F32)
    bad = ~np.isfinite(y).all(axis=1)
    fine = ~bad & (amax >= F32(2.0 ** -100))
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        scale = np.where(bad, F32(np.nan), np.where(fine, amax / F32(448), F32(0)))
        back = np.where(fine, F32(448) / amax, F32(0)).astype(F32)
    q = np.where(fine[:, None], np.where(np.isfinite(y), y, 0).astype(F32) * back[:, None], F32(0))
    return np.where(fine[:, None], e4m3_code(q), 0).astype(np.uint8), scale.astype(F32)


def e4m3_blocks(y):
    """(codes, exponent bytes) with one power of two for each 32 columns."""
    e = block_bytes(y, 448.0)
    b = np.where(e == 255, 1.0, 2.0 ** (e.astype(F64) - 127))
    q = np.where((e == 255)[:, :, None], 0.0, _blocks(y).astype(F64) / b[:, :, None])
    codes = e4m3_code(np.where(np.isfinite(q), q, 0.0)).reshape(y.shape[0], -1)
    codes = np.where(np.repeat(e == 255, 32, axis=1), 0, codes)
    return codes[:, :y.shape[1]].astype(np.uint8), e


def norm_backward(dy, dsum, s, inv, weight):
    """(dx, dweight) in binary64 from the call's own inv."""
    dy, s, w, inv = (np.asarray(v, F64) for v in (dy, s, weight, inv))
    g, h = dy * w, s * inv[:, None]
    dx = inv[:, None] * (g - h * (g * h).mean(axis=1, keepdims=True))
    if dsum is not None:
        dx = dx + dsum
    return dx, (dy * h).sum(axis=0)


def w4_quantize(w):
    """(packed, exponent bytes, values) of binary32 weights."""
    e = block_bytes(w, 6.0)
    bad = (e == 255)[:, :, None]
    b = np.where(e == 255, 1.0, 2.0 ** (e.astype(F64) - 127))[:, :, None]
    v = np.where(bad, 0.0, np.where(bad, 0.0, _blocks(w).astype(F64)) / b)
    code = _nearest(np.abs(v), E2M1)
    values = np.where(bad, np.nan, np.copysign(E2M1[code], v) * b)
    code = code | (np.where(bad, 0, np.signbit(v)).astype(np.int64) << 3)
    code = code.reshape(w.shape[0], -1)
    packed = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    return packed, e, values.reshape(w.shape[0], -1)[:, :w.shape[1]]


def w4_values(packed, scales, cols):
    """The matrix that codes and exponent bytes stand for, in binary64."""
    code = np.empty((packed.shape[0], packed.shape[1] * 2), np.int64)
    code[:, 0::2], code[:, 1::2] = packed & 15, packed >> 4
    v = np.where(code & 8, -E2M1[code & 7], E2M1[code & 7])
    return (v * np.repeat(scale_value(scales), 32, axis=1))[:, :cols]


def log_softmax(logits):
    """(log p, entropy, m, log S) of each row in binary64; a row with nothing
    unmasked has log p -infinity, entropy 0 and (-infinity, 0)."""
    x = logits.astype(F64)
    m = x.max(axis=1)
    nothing = np.isneginf(m)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        d = x - np.where(nothing, 0, m)[:, None]
        e = np.exp(d)
        at = np.argmax(x, axis=1)
        e1 = e.copy()
        e1[np.arange(len(m)), at] = 0
        log_s = np.where(nothing, 0, np.log1p(e1.sum(axis=1)))
        lp = d - log_s[:, None]
        p = np.exp(lp)
        h = -np.where(p > 0, p * lp, np.where(np.isnan(p), np.nan, 0)).sum(axis=1)
    bad = np.isnan(x).any(axis=1) | np.isposinf(x).any(axis=1)
    lp[bad], log_s[bad], h[bad] = np.nan, np.nan, np.nan
    lp[nothing], h[nothing] = -np.inf, 0
    return lp, h, m, log_s


def top_ids(logits, k):
    """Largest first, equal ones by the lowest index, NaN before all."""
    x = logits.astype(F64) + 0.0
    key = np.where(np.isnan(x), np.inf, x)
    out = []
    for row, nan in zip(key, np.isnan(x)):
        out.append(np.lexsort((np.arange(len(row)), -row, ~nan))[:k])
    return np.array(out, np.int64).reshape(len(x), k)


def logprobs_backward(lp, h, targets, dlogprobs, dentropy):
    """dlogits in binary64."""
    rows, vocab = lp.shape
    with np.errstate(invalid="ignore"):
        p = np.exp(lp)
        g = np.where(targets < 0, 0.0, dlogprobs.astype(F64))
        g = np.where(targets >= vocab, np.nan, g)
        d = -g[:, None] * p
        for r, t in enumerate(targets):
            if 0 <= t < vocab:
                d[r, t] = -g[r] * np.expm1(lp[r, t])
        if dentropy is not None:
            plp = np.where(p > 0, p * (lp + h[:, None]), np.where(np.isnan(p), np.nan, 0.0))
            d -= dentropy.astype(F64)[:, None] * plp
    return d
