"""What surrounds attention in a decode step, as plain fp64 definitions.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

* ``rotate`` -- rotary positions: pair j of a head's rotated dims turns by the
  angle position * inv_freq[j].
* ``store_e4m3``, ``store_nvfp4`` -- the nearest stored value (ties to the even
  code, saturated) of numbers in the two low-precision cache types, found by
  searching the decoded code tables of ``fp8`` and ``nvfp4``.
* ``adapters`` -- y plus each row's own low-rank product, with the magnitude
  that bounds the rounding error of any fp32 evaluation order.
* ``adjust_logits`` -- penalties, biases and a mask on one row of logits.
* ``greedy`` -- the lowest token of the largest logit above -inf, or -1.
"""

from __future__ import annotations

import numpy as np

from . import bf16, fp8, nvfp4


def rotate(x, positions, inv_freq, offset=0, interleaved=False, gain=1.0):
    """x fp64 [n, H, D] with dims [offset, offset + 2 len(inv_freq)) turned.

    The angle is formed and turned in extended precision, so that positions up
    to 2^31 lose nothing that fp64 would show."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    p = np.asarray(positions).astype(np.longdouble)[:, None]
    angle = p * np.asarray(inv_freq, dtype=np.float32).astype(np.longdouble)[None]
    cos = (gain * np.cos(angle)).astype(np.float64)[:, None]
    sin = (gain * np.sin(angle)).astype(np.float64)[:, None]
    ia = offset + (2 * np.arange(half) if interleaved else np.arange(half))
    ib = ia + (1 if interleaved else half)
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * cos - b * sin
    x[..., ib] = b * cos + a * sin
    return x


def _nearest(values, table):
    """Index of the nearest entry of an ascending table of non-negative values
    for non-negative numbers; ties go to the even index, large ones to the top."""
    v = np.asarray(values, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    mid = (table[lo] + table[hi]) / 2
    return np.where(v > mid, hi, np.where(v < mid, lo, np.where(lo % 2 == 0, lo, hi)))


_E4M3 = fp8.decode_e4m3(np.arange(0x7F, dtype=np.uint8))  # 0 .. 448, ascending
_E2M1 = nvfp4.decode_e2m1(np.arange(8))                   # 0 .. 6, ascending


def store_e4m3(v):
    """E4M3 bytes nearest to fp64 values (saturated at 448; NaN: 0x7F)."""
    v = np.asarray(v, dtype=np.float64)
    code = _nearest(np.nan_to_num(np.abs(v)), _E4M3).astype(np.uint8)
    code = np.where(np.isnan(v), np.uint8(0x7F), code)
    return np.where(np.signbit(v) & ~np.isnan(v), code | np.uint8(0x80), code)


def store_nvfp4(v, scale):
    """(codes uint8 [..., D/2], block scales uint8 [..., D/16]) of fp64 values."""
    v = np.asarray(v, dtype=np.float64)
    blocks = v.reshape(*v.shape[:-1], v.shape[-1] // 16, 16)
    s = store_e4m3(np.abs(blocks).max(-1) / (6 * scale))
    step = fp8.decode_e4m3(s)[..., None] * scale
    with np.errstate(invalid="ignore", divide="ignore"):
        u = np.where(step > 0, blocks / step, 0.0)
    code = _nearest(np.abs(u), _E2M1) | np.where(np.signbit(u), 8, 0)
    code = code.reshape(v.shape)
    return (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8), s


def adapters(x, y, a, b, ids, ranks=None, scales=None):
    """(out, magnitude): y[i] + scale * (bf16(x[i]) A^T) B^T of row i's adapter,
    and the same product of magnitudes (without y)."""
    xr = bf16.round_to_bf16(np.asarray(x, dtype=np.float64))
    out = np.array(y, dtype=np.float64)
    mag = np.zeros_like(out)
    for i, d in enumerate(ids):
        if d < 0:
            continue
        r = a.shape[1] if ranks is None else int(ranks[d])
        s = 1.0 if scales is None else float(scales[d])
        A, B = a[d, :r].astype(np.float64), b[d, :, :r].astype(np.float64)
        out[i] += s * (B @ (A @ xr[i]))
        mag[i] = abs(s) * (np.abs(B) @ (np.abs(A) @ np.abs(xr[i])))
    return out, mag


def adjust_logits(x, prompt=(), output=(), repetition=1.0, frequency=0.0, presence=0.0, bias=(),
                  allowed=None, dtype=np.float64):
    """One row of logits adjusted, every operation in `dtype`.  prompt, output:
    tokens; bias: (token, value) pairs; allowed: truth value per token or None."""
    f = dtype
    l = np.array(x, dtype=f)
    V = len(l)
    made = np.bincount(np.asarray(output, dtype=np.int64), minlength=V)
    seen = (made > 0) | (np.bincount(np.asarray(prompt, dtype=np.int64), minlength=V) > 0)
    rep = f(repetition)
    with np.errstate(all="ignore"):
        l = np.where(seen, np.where(l > 0, l / rep, l * rep), l)
        l = np.where(made > 0, l - f(frequency) * made.astype(f), l)
        l = np.where(made > 0, l - f(presence), l)
        sums = {}
        for v, w in bias:
            sums[v] = f(w) if v not in sums else f(sums[v] + f(w))
        for v, w in sums.items():
            l[v] = f(l[v] + w)
    if allowed is not None:
        l = np.where(allowed, l, f(-np.inf))
    return l


def greedy(l):
    """The lowest token among those with the largest logit > -inf, else -1."""
    l = np.where(np.isnan(l), -np.inf, l)
    return int(np.argmax(l)) if l.size and l.max() > -np.inf else -1
