"""Plain 64-bit definitions of the microscaled 4-bit formats and the quantised cache rows, in numpy.

Written from the formats' definitions (include/entropack.h); shares no code with the library.
Every function works on float64 arrays that hold bf16, fp16 or fp32 values exactly.
"""
import numpy as np

BLOCK = {"mxfp4": 32, "nvfp4": 16}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def floor_log2(x):
    """floor(log2 x) of positive numbers, exactly."""
    return np.frexp(x)[1] - 1


def to_grid(x, low, bits, top):
    """x to the nearest number with `bits` significand bits and an exponent of at least `low` (ties to
    even), at most `top` in size."""
    e = np.where(x != 0, floor_log2(np.where(x != 0, np.abs(x), 1.0)), low)
    step = np.ldexp(1.0, np.maximum(e, low) - (bits - 1))
    return np.clip(np.rint(x / step) * step, -top, top)


def e4m3(x):
    return to_grid(x, -6, 4, 448.0)


def e2m1(x):
    return to_grid(x, 0, 2, 6.0)


def e4m3_byte(v):
    """The byte of a non-negative E4M3 value (NaN: 0x7f)."""
    v = np.asarray(v, np.float64)
    fine = np.isfinite(v)
    w = np.where(fine, v, 0.0)
    e = np.maximum(np.where(w > 0, floor_log2(np.where(w > 0, w, 1.0)), -6), -6)
    m = np.rint(w / np.ldexp(1.0, e - 3)).astype(np.int64)  # 8..15, or 0..7 below 2^-6
    byte = np.where(m >= 8, ((e + 7) << 3) | (m - 8), m)
    return np.where(fine, byte, 0x7F).astype(np.uint8)


def e4m3_value(byte):
    b = np.asarray(byte).astype(np.int64) & 0x7F
    e, m = b >> 3, b & 7
    v = np.where(e > 0, np.ldexp(8.0 + m, e - 10), np.ldexp(1.0 * m, -9))
    return np.where(b == 0x7F, np.nan, v)


def e8m0_value(byte):
    b = np.asarray(byte).astype(np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))


def tensor_scale(x):
    a = np.abs(x[np.isfinite(x)])
    top = a.max() if a.size else 0.0
    k = -100
    if top > 0:
        k = max(floor_log2(top / 2688), -100)
        while top > 2688 * 2.0 ** k:
            k += 1
    return 2.0 ** k


def quantize(x, fmt, g=None):
    """(values / (q = block scale) as E2M1 values, scale bytes, g) of a matrix; elements padded to whole
    blocks.  g: None to take it from the data."""
    blk = BLOCK[fmt]
    rows, cols = x.shape
    b = np.zeros((rows, -(-cols // blk) * blk))
    b[:, :cols] = x
    b = b.reshape(rows, -1, blk)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1) if b.size else np.zeros(b.shape[:2])
    if fmt == "mxfp4":
        g = 1.0
        e = np.maximum(np.where(top > 0, floor_log2(np.where(top > 0, top, 1.0)) - 2, -127), -127)
        byte, q = (e + 127).astype(np.uint8), np.ldexp(1.0, e)
        byte[bad] = 255
    else:
        if g is None:
            g = tensor_scale(x)
        sb = e4m3(top / (6 * g))
        byte, q = e4m3_byte(sb), sb * g
        byte[bad] = 0x7F
    el = np.where(q[..., None] > 0, e2m1(b / np.where(q > 0, q, 1.0)[..., None]), 0.0)
    return el.reshape(rows, -1), byte, g


def scale_values(byte, fmt):
    return e8m0_value(byte) if fmt == "mxfp4" else e4m3_value(byte)


def unpack(data):
    """E2M1 values of packed rows."""
    return E2M1[np.stack((data & 15, data >> 4), -1).reshape(data.shape[0], -1)]


def values(el, byte, g, cols, fmt):
    v = el[:, :byte.shape[1] * BLOCK[fmt]].reshape(el.shape[0], -1, BLOCK[fmt]) * scale_values(byte, fmt)[..., None]
    return v.reshape(el.shape[0], -1)[:, :cols] * g


def cache_row(x, fmt):
    """(payload values, scale values) of 8-bit cache rows x [n, head_dim]."""
    bad = ~np.isfinite(x).all(-1)
    y = np.where(bad[:, None], 0.0, x)
    top = np.abs(y).max(-1)
    if fmt == "fp8":
        e = np.full(top.shape, -100)
        t = np.where(top > 0, top, 1.0)
        f = floor_log2(t / 448)
        f += t > 448 * np.ldexp(1.0, f)
        e = np.where(top > 0, np.maximum(f, -100), -100)
        s = np.ldexp(1.0, e)
        p = e4m3(y / s[:, None])
    else:
        s = np.where(top >= 2.0 ** -100, (top.astype(np.float32) * (np.float32(1) / np.float32(127))).astype(np.float64), 0.0)
        p = np.where(s[:, None] > 0, np.rint(y / np.where(s > 0, s, 1.0)[:, None]), 0.0)
    return p, np.where(bad, np.nan, s)
