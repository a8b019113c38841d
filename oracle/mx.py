"""fp64 NumPy restatement of the microscaled matrices: codes with a power of two for each run of 32
columns, RMSNorm with a quantised output, products and SwiGLU, and the packed layout."""

import numpy as np

RUN, ATOM = 32, 128
TOP = {8: 448.0, 4: 6.0}
NAN_E = 128  # exponent byte 255


def code_values(bits):
    """Values of the codes 0 .. 2^bits - 1: e4m3 (no infinities, 0x7f and 0xff NaN) or e2m1."""
    c = np.arange(1 << bits)
    mant, bias = (3, 7) if bits == 8 else (1, 1)
    e, m = (c >> mant) & ((1 << (bits - 1 - mant)) - 1), c & ((1 << mant) - 1)
    v = np.where(e == 0, m * 2.0 ** (1 - bias - mant), (1 + m / 2.0 ** mant) * 2.0 ** (e - float(bias)))
    if bits == 8:
        v[(c & 127) == 127] = np.nan
    return np.where(c >> (bits - 1), -v, v)


def nearest(y, bits):
    """Codes of |y| <= TOP: the nearest value, the even code on a tie."""
    mags = code_values(bits)[:1 << (bits - 1)]
    mags = mags[np.isfinite(mags)]
    mid = (mags[1:] + mags[:-1]) / 2
    a = np.abs(y)
    lo = np.searchsorted(mid, a, side="left")   # a tie belongs to the lower code
    hi = np.searchsorted(mid, a, side="right")  # ... to the upper
    code = np.where(lo % 2 == 0, lo, hi)
    return (code | (np.signbit(y).astype(np.int64) << (bits - 1))).astype(np.uint8)


def quantize(x, bits):
    """x [rows, cols] (fp64) -> codes [rows, runs, 32] and exponents [rows, runs] (NAN_E: not finite)."""
    x = np.asarray(x, np.float64)
    x = np.pad(x, ((0, 0), (0, -x.shape[1] % RUN))).reshape(x.shape[0], -1, RUN)
    bad = ~np.isfinite(x).all(-1)
    a = np.where(bad[..., None], 0.0, np.abs(x)).max(-1)
    f, ex = np.frexp(a / TOP[bits])  # a / TOP = f 2^ex, f in [0.5, 1): the division may round
    e = np.where(a > 0, ex - 1, -127)
    for _ in range(2):
        e = np.where(a > TOP[bits] * np.exp2(e.astype(np.float64)), e + 1, e)
    e = np.maximum(e, -127)
    y = np.where(bad[..., None], 0.0, x) / np.exp2(e.astype(np.float64))[..., None]
    return nearest(y, bits), np.where(bad, NAN_E, e)


def values(codes, e, bits, cols):
    s = np.where(e == NAN_E, np.nan, np.exp2(np.minimum(e, 127).astype(np.float64)))
    return (code_values(bits)[codes] * s[..., None]).reshape(codes.shape[0], -1)[:, :cols]


def held(x, bits):
    return values(*quantize(x, bits), bits, np.shape(x)[1])


def pack(codes, e, bits, fill=0xFF):
    """The packed bytes of the codes and scales; `fill`: bytes of rows that are not there."""
    R, runs = e.shape
    atoms = -(-runs // 4)
    c = np.zeros((R, atoms * ATOM), np.uint8)
    c[:, :runs * RUN] = codes.reshape(R, -1)
    if bits == 4:
        c = c[:, 0::2] | (c[:, 1::2] << 4)
    s = np.full((-(-R // 128) * 128, atoms * 4), fill, np.uint8)
    s[:R] = 0
    s[:R, :runs] = e + 127
    out = np.empty((-(-R // 128), atoms, 512), np.uint8)
    for r in range(128):
        for j in range(4):
            out[:, :, 16 * (r % 32) + 4 * (r // 32) + j] = s[r::128, j::4]
    return c.reshape(-1), out.reshape(-1)


def unpack_scales(sbytes, cols):
    """Exponent bytes [128 tiles, 4 atoms], those of rows that are not there included."""
    atoms = -(-cols // ATOM)
    s = np.asarray(sbytes).reshape(-1, atoms, 512)
    b = np.empty((s.shape[0] * 128, atoms * 4), np.int64)
    for r in range(128):
        for j in range(4):
            b[r::128, j::4] = s[:, :, 16 * (r % 32) + 4 * (r // 32) + j]
    return b


def unpack(cbytes, sbytes, rows, cols, bits):
    """Codes [rows, 4 atoms, 32] and exponents [rows, 4 atoms] of packed bytes, the padding included."""
    c = np.asarray(cbytes).reshape(rows, -1)
    if bits == 4:
        c = np.stack([c & 15, c >> 4], -1)
    return c.reshape(rows, -1, RUN), unpack_scales(sbytes, cols)[:rows] - 127


def rmsnorm(s, weight, eps):
    """s [rows, cols] already rounded to the stream's type; the unrounded norm."""
    s = np.asarray(s, np.float64)
    return s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * weight


def linear(x, w):
    return x @ w.T


def swiglu(x, gate, up):
    g = x @ gate.T
    return g / (1 + np.exp(-g)) * (x @ up.T)
