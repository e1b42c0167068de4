"""Float64 oracle of the block-scaled 8-bit (MX) storage and its operators.

NumPy only, written from the definition: e4m3 values (1 sign, 4 exponent bits with
bias 7, 3 mantissa bits; largest 448, smallest step 2^-9), one power of two 2^e
per 32 consecutive values of a row, e the smallest integer with
max |x| <= 448 * 2^e and e >= -127, stored as the byte e + 127; byte 255 marks a block
that holds a NaN or an infinity.
"""

import numpy as np

from .qi21_oracle import linear, rms_norm, silu

BLOCK = 32
E4M3_MAX = 448.0
NAN_BYTE = 255


def e4m3_round(v):
    """Nearest e4m3 value (ties to even) of finite |v| <= 448."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    _, x = np.frexp(np.where(a == 0, 1.0, a))          # a = m * 2^x, 1/2 <= m < 1
    step = np.ldexp(1.0, np.maximum(x - 1, -6) - 3)    # eight steps per binade, subnormals below 2^-6
    return np.rint(v / step) * step


def e4m3_decode(codes):
    """The value of each e4m3 byte."""
    c = np.asarray(codes, dtype=np.int64)
    sign, e, m = np.where(c & 0x80, -1.0, 1.0), (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.ldexp(1.0, e - 10))
    return np.where((c & 0x7F) == 0x7F, np.nan, sign * v)


def block_exponents(x):
    """e of every block of x [R, K] (finite), [R, K / 32] integers."""
    top = np.abs(np.asarray(x, dtype=np.float64)).reshape(x.shape[0], -1, BLOCK).max(-1)
    e = np.full(top.shape, -127, dtype=np.int64)
    _, near = np.frexp(top)
    for c in (near - 10, near - 9, near - 8):          # 448 is between 2^8 and 2^9
        ok = (top > np.ldexp(E4M3_MAX, c - 1)) & (top <= np.ldexp(E4M3_MAX, c))
        e = np.where(ok, np.maximum(c, -127), e)
    return e


def quantize(x):
    """(values / 2^e rounded to e4m3 [R, K], scale bytes [R, K / 32]); NaN where the block is not finite."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).reshape(x.shape[0], -1, BLOCK).all(-1)
    clean = np.where(np.repeat(bad, BLOCK, axis=1), 0.0, x)
    e = block_exponents(clean)
    q = e4m3_round(np.ldexp(clean, -np.repeat(e, BLOCK, axis=1)))
    return (np.where(np.repeat(bad, BLOCK, axis=1), np.nan, q), np.where(bad, NAN_BYTE, e + 127))


def values(q, byte):
    """What (q, scale bytes) stand for."""
    s = np.where(byte == NAN_BYTE, np.nan, np.ldexp(1.0, np.minimum(byte, 254) - 127))
    return np.asarray(q, dtype=np.float64) * np.repeat(s, BLOCK, axis=1)


def untile(scale, R, K):
    """Scale bytes [R, K / 32] from their tiles [ceil(R / 128), ceil(K / 128), 32, 4, 4], by the index rule."""
    scale = np.asarray(scale)
    r, b = np.arange(R)[:, None], np.arange(K // BLOCK)[None, :]
    return scale[r // 128, b // 4, r % 32, r % 128 // 32, b % 4].astype(np.int64)


def gelu_tanh(y):
    return 0.5 * y * (1 + np.tanh(np.sqrt(2 / np.pi) * (y + 0.044715 * y ** 3)))


def linear_mx(x, w, bias=None, act="none", residual=None, alpha=1.0):
    """alpha * act(x w^T + b) (+ residual) on the values that the operands stand for."""
    y = linear(x, w, bias)
    y = alpha * {"none": lambda t: t, "silu": silu, "gelu_tanh": gelu_tanh}[act](y)
    return y if residual is None else residual + y


def swiglu(x, w_il, bias_il=None):
    """silu(x Wg^T + bg) * (x Wu^T + bu), gate and up rows in alternating blocks of 128."""
    y = linear(x, w_il, bias_il)
    y = y.reshape(y.shape[0], -1, 2, 128)
    return (silu(y[:, :, 0]) * y[:, :, 1]).reshape(y.shape[0], -1)


__all__ = ["block_exponents", "e4m3_decode", "e4m3_round", "gelu_tanh", "linear_mx", "quantize", "rms_norm", "swiglu",
           "untile", "values"]
