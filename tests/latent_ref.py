"""Plain 64-bit definitions of the latent-cache operators, for the tests.

Written from the formulas with numpy; shares nothing with the CUDA path.
Caches are byte arrays [slots, row bytes] in one of three formats.
"""

from __future__ import annotations

import math

import numpy as np
import torch

NOPE, PE, ROW, GROUP = 512, 64, 576, 32
BF16, E4M3, MX = 0, 1, 2
ROW_BYTES = {BF16: 1152, E4M3: 576, MX: 656}
EPS_BF16, EPS_F16 = 2.0 ** -8, 2.0 ** -11  # half a step, relative
EPS_F8_WEIGHT = 2.0 ** -9 + EPS_F16  # an fp16 weight as three e5m2 terms: each leaves half a step, 2^-3, of what it took


def _lut():
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.nan if b & 0x7F == 0x7F else math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        v[b] = -x if b & 0x80 else x
    return v


LUT = _lut()


def bf16_bits(x32: np.ndarray) -> np.ndarray:
    """bf16 bit patterns of fp32 values, ties to even (NaN to the canonical quiet NaN, as the conversion
    instruction gives it)."""
    u = np.ascontiguousarray(x32, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x32), np.uint16(0x7FFF), r)


def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_bytes(x: np.ndarray) -> np.ndarray:
    """e4m3 bytes of fp64 values: nearest, ties to the even code, saturating; NaN 0x7F."""
    a = np.minimum(np.abs(x), 1e30)
    pos = LUT[:127]  # ascending magnitudes of codes 0..126
    mid = (pos[1:] + pos[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")    # ties go down
    hi = np.searchsorted(mid, a, side="right")   # ties go up
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi)).astype(np.uint8)
    code = np.minimum(code, 126).astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def mx_exponents(y32: np.ndarray) -> np.ndarray:
    """Least e with max |y| <= 448 * 2^e of each 32, over the finite values, within [-117, 119]."""
    a = np.abs(y32.astype(np.float64)).reshape(y32.shape[0], -1, GROUP)
    a = np.where(np.isfinite(a), a, 0.0).max(-1)
    e = np.full(a.shape, -117)
    for k in range(-117, 119):
        e = np.where(a > 448.0 * 2.0 ** k, k + 1, e)
    return e


def insert_rows(kv_c, k_pe, fmt, norm_weight=None, eps=1e-6, positions=None, cos_sin=None, kv_scale=None):
    """Byte rows [T, row bytes] of torch bf16 inputs on the host."""
    x = kv_c.double().numpy()
    with np.errstate(all="ignore"):
        if norm_weight is not None:
            w = norm_weight.double().numpy()
            y = (x / np.sqrt((x * x).sum(1, keepdims=True) / NOPE + float(np.float32(eps))) * w).astype(np.float32)
        else:
            y = x.astype(np.float32)
        pe = k_pe.float().numpy()
        pe_bits = k_pe.contiguous().view(torch.int16).numpy().view(np.uint16).copy()
        if cos_sin is not None:
            tab = cos_sin.numpy()
            for t in range(x.shape[0]):
                pos = int(positions[t])
                if 0 <= pos < tab.shape[0]:
                    c, s = tab[pos, :32], tab[pos, 32:]
                    a, b = pe[t, :32].copy(), pe[t, 32:].copy()
                    pe[t, :32] = a * c - b * s
                    pe[t, 32:] = b * c + a * s
                    pe_bits[t] = bf16_bits(pe[t])
        n = x.shape[0]
        if fmt == BF16:
            yb = bf16_bits(y) if norm_weight is not None else kv_c.contiguous().view(torch.int16).numpy().view(np.uint16)
            return np.concatenate([yb, pe_bits], 1).view(np.uint8).reshape(n, 1152)
        if fmt == E4M3:
            q = (np.concatenate([y, pe], 1) / np.float32(kv_scale)).astype(np.float32)
            return e4m3_bytes(q.astype(np.float64))
        e = mx_exponents(y)
        codes = e4m3_bytes((y.astype(np.float64).reshape(n, -1, GROUP) * 2.0 ** (-e.astype(np.float64))[..., None])
                           .reshape(n, NOPE))
        return np.concatenate([codes, (e + 127).astype(np.uint8), pe_bits.view(np.uint8).reshape(n, 128)], 1)


def values(rows: np.ndarray, fmt: int, kv_scale=None) -> np.ndarray:
    """fp64 values [n, 576] of byte rows."""
    if fmt == BF16:
        return bf16_values(np.ascontiguousarray(rows).view(np.uint16))
    if fmt == E4M3:
        return LUT[rows] * float(np.float32(kv_scale))
    x = LUT[rows[:, :NOPE]].reshape(-1, NOPE // GROUP, GROUP)
    x = x * 2.0 ** (rows[:, NOPE:NOPE + 16].astype(np.float64) - 127.0)[:, :, None]
    pe = bf16_values(np.ascontiguousarray(rows[:, NOPE + 16:]).view(np.uint16))
    return np.concatenate([x.reshape(-1, NOPE), pe], 1)


def attend(q, keys, sm_scale, f8=False):
    """One token: q fp64 [H, 576], keys fp64 [n, 576].  Returns out [H, 512], lse [H] and the bounds of what the
    kernel's arithmetic may be off by.

    Scores: products of 16-bit numbers are exact, their fp32 sum is off by at most 576 * 2^-23 sum |q k| (any
    order, truncating adders allowed), and the scale, the difference to the reference maximum and the power of two
    add a few units of 2^-23 of |s| and 2^-21.  A weight's relative error is that, d, plus half a step of its type,
    w; so the sum is off by (w + d) sum p |v| and the denominator by d, and the result by half a bf16 step.  The
    fp32 sum of the products adds n * 2^-23 of sum p |v|.  With e4m3 operands (f8) a weight is 2^7 times its power
    of two as fp16 and then as three e5m2 terms; the last term's smallest step is 2^-16, so a small weight is off by
    up to 2^-17 / 2^7 = 2^-24 of the reference weight, which is no larger than the row's largest.
    """
    H, n = q.shape[0], keys.shape[0]
    if n == 0:
        z = np.zeros((H, NOPE))
        return z, np.full(H, -np.inf), z, np.zeros(H)
    s = q @ keys.T * sm_scale
    mag = np.abs(q) @ np.abs(keys).T * abs(sm_scale)
    top = s.max(1, keepdims=True)
    p = np.exp(s - top)
    den = p.sum(1, keepdims=True)
    p = p / den
    v = keys[:, :NOPE]
    out = p @ v
    lse = top[:, 0] + np.log(den[:, 0])
    d = (576 * 2.0 ** -23 * mag + 8 * 2.0 ** -23 * np.abs(s)).max(1, keepdims=True) + 2.0 ** -21
    w = EPS_F8_WEIGHT if f8 else EPS_BF16
    pv = p @ np.abs(v)
    tol = (w + 2 * d + n * 2.0 ** -23) * pv + EPS_BF16 * np.abs(out) * 1.01 + 1e-30
    if f8:
        tol = tol + 2.0 ** -24 * np.abs(v).sum(0) / den
    lse_tol = d[:, 0] + (n + 8) * 2.0 ** -23 + np.abs(lse) * 2.0 ** -21
    return out, lse, tol, lse_tol
