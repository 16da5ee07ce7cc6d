"""The 8-bit row format from its definition, on the CPU, for the tests: which
bytes stand for what, and what rounding to it gives.  Everything in 64 bits."""
import numpy as np


def row_bytes(H):
    lines = -(-H // 128)
    return 128 * (lines + -(-lines * 4 // 128))


def e4m3_values():
    """What each of the 256 bytes stands for."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(b & 127) == 127] = np.nan
    return np.where(b >= 128, -v, v)


VALUES = e4m3_values()


def unpack(rows, H):
    """(values [..., H] in fp64, scale bytes [..., V / 32]) of packed rows."""
    V = -(-H // 128) * 128
    q, s = rows[..., :V], rows[..., V:V + V // 32].astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, np.where(s == 255, 0, s) - 127))
    with np.errstate(invalid="ignore"):
        v = VALUES[q].reshape(*q.shape[:-1], V // 32, 32) * f[..., None]
    return v.reshape(q.shape)[..., :H], s


def pack(x):
    """Packed rows of x [..., H] (any real type)."""
    x = np.asarray(x, dtype=np.float64)
    H = x.shape[-1]
    V = -(-H // 128) * 128
    v = np.zeros((*x.shape[:-1], V))
    v[..., :H] = x
    v = v.reshape(*x.shape[:-1], V // 32, 32)
    bad = ~np.isfinite(v).all(axis=-1)
    top = np.where(bad, 1.0, np.abs(np.where(np.isfinite(v), v, 0)).max(axis=-1))
    m, e = np.frexp(top)  # m in [1/2, 1), 448 = 7/8 * 2^9
    e = np.where(top == 0, -127, np.maximum(np.where(m <= 0.875, e - 9, e - 8), -127))
    scaled = np.ldexp(np.where(bad[..., None], 0, v), -e[..., None])
    mag = np.abs(scaled)
    step = np.exp2(np.floor(np.log2(np.maximum(mag, 2.0 ** -6))) - 3)
    near = np.rint(mag / step) * step  # ties to even
    grid = VALUES[:127]
    q = np.searchsorted(grid, near)
    assert np.array_equal(grid[q], near)
    q = np.where(np.signbit(scaled), q + 128, q)
    q = np.where(bad[..., None], 127, q)
    rows = np.zeros((*x.shape[:-1], row_bytes(H)), np.uint8)
    rows[..., :V] = q.reshape(*x.shape[:-1], V)
    rows[..., V:V + V // 32] = np.where(bad, 255, e + 127)
    return rows
