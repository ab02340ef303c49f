"""MXFP4 in 64 bits (numpy): quantise, dequantise, SwiGLU, and operands for the product tests."""
import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([VALUES, -VALUES])
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # a tie goes down at an even border index, up at an odd one


def up(n, to):
    return -(-n // to) * to


def quantise(x):
    """x (rows x K, float64) -> codes (rows x up(K, 32), uint8, zero past K) and scale bytes (rows x ceil(K / 32))."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    b = np.zeros((rows, up(k, 32)))
    b[:, :k] = x
    b = b.reshape(rows, -(-k // 32), 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    e = np.where(top > 0, np.frexp(top)[1] - 1, -2000)  # floor(log2 amax)
    byte = np.clip(e - 2 + 127, 0, 254)
    t = np.ldexp(np.abs(b), 127 - byte[..., None])
    code = np.zeros(b.shape, dtype=np.uint8)
    for i, border in enumerate(BORDERS):
        code += (t >= border) if i & 1 else (t > border)
    code |= ((b < 0) | ((b == 0) & np.signbit(b))).astype(np.uint8) << 3
    byte = np.where(bad, 255, byte).astype(np.uint8)
    code[bad] = 0
    return code.reshape(rows, up(k, 32)), byte


def pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    c = np.empty((q.shape[0], q.shape[1] * 2), dtype=np.uint8)
    c[:, 0::2], c[:, 1::2] = q & 15, q >> 4
    return c


def values(code, byte):
    """float64 values of codes (rows x 32 nb) and scale bytes (rows x nb); NaN blocks where the byte is 255."""
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return VALUES[code] * np.repeat(s, 32, axis=-1)


def swiglu(x):
    k = x.shape[1] // 2
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        return x[:, :k] / (1.0 + np.exp(-x[:, :k])) * x[:, k:]
