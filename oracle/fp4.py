"""4-bit floating point with block scales -- TEST INFRASTRUCTURE ONLY.

A code is E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign (8).  Blocks of 32
consecutive entries of a row have the smallest power of two that is at least
max |x| / 6 (2^-127 at least); blocks of 16 an E4M3 number times the tensor's
power of two 2^k, the smallest with max |x| <= 2688 2^k (k >= -127).  Quotients (max |x| / 6, x by an
E4M3 scale) are rounded to float32 before anything is decided by them.
"""

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
M32 = np.uint64(0xFFFFFFFF)
C0, C1, C2 = np.uint64(0x9E3779B1), np.uint64(0x6A09E667), np.uint64(0xBB67AE85)
#: E4M3 numbers by code (127 is NaN)
E4M3 = np.array([c * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def _mix(x):
    x = ((x ^ (x >> np.uint64(16))) * C1) & M32
    x = ((x ^ (x >> np.uint64(15))) * C2) & M32
    return x ^ (x >> np.uint64(16))


def fp4_bits(rows, cols, seed, axis):
    """16 random bits of each entry of a rows x cols operand (axis 1: the matrix as it is, 0: its transpose)."""
    seed = int(seed) & (2 ** 64 - 1)
    lo, hi = np.uint64(seed & 0xFFFFFFFF), np.uint64(seed >> 32)
    key = _mix(_mix((lo + C0 * np.uint64(axis)) & M32) ^ hi)
    pairs = (cols + 1) // 2
    j = np.arange(rows, dtype=np.uint64)[:, None] * np.uint64(pairs) + np.arange(pairs, dtype=np.uint64)
    h = _mix(((j & M32) * C0 + key + (j >> np.uint64(32)) * C1) & M32)
    return np.stack((h & np.uint64(0xFFFF), h >> np.uint64(16)), 2).reshape(rows, -1)[:, :cols].astype(np.int64)


def _power_at_least(a):
    """Exponent of the smallest power of two that is at least a > 0."""
    m, e = np.frexp(a)
    return np.where(m == 0.5, e - 1, e)


def fp4_quantize(x, block, bits=None):
    """(codes, scale codes, tensor factor) of float64 rows: codes rows x cols in 0 .. 15, one scale code per row and
    block, 2^k (blocks of 32: 1).  bits: 16 random bits per entry (stochastic rounding)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    blocks = -(-cols // block)
    z = np.zeros((rows, blocks * block))
    z[:, :cols] = x
    z = z.reshape(rows, blocks, block)
    bad = ~np.isfinite(z).all(2)
    a = np.where(np.isfinite(z), np.abs(z), 0.0)
    top = np.where(bad, 0.0, a.max(2))
    factor = 1.0
    if block == 32:
        e = np.maximum(_power_at_least(np.where(top > 0, top, 2.0 ** -140) / 6), -127)  # (x / 6 in float64 is at a power of two where x is)
        scale, code = np.ldexp(1.0, e), e + 127
        y = a / scale[:, :, None]
    else:
        largest = float(a.max(initial=0.0))
        k = max(int(_power_at_least(largest / 2688)), -127) if largest > 0 else -127
        factor = 2.0 ** k
        q = (top.astype(np.float32) / np.float32(6)).astype(np.float64) / factor
        up = np.searchsorted(E4M3, q, side="left")                     # the first that is at least q
        up = np.minimum(up, 126)
        if bits is None:
            down = np.maximum(up - 1, 0)
            d_up, d_down = E4M3[up] - q, q - E4M3[down]
            up = np.where((d_down < d_up) | ((d_down == d_up) & (down % 2 == 0)), down, up)
        code = up
        scale = E4M3[code][:, :, None]
        with np.errstate(divide="ignore", invalid="ignore"):
            y = ((a / factor).astype(np.float32) / scale.astype(np.float32)).astype(np.float64)
        y = np.minimum(np.where(scale > 0, y, 0.0), 6.0)
    low = np.searchsorted(GRID, y, side="right") - 1
    gap = np.append(np.diff(GRID), 1.0)[low]
    part = (y - GRID[low]) / gap
    if bits is None:
        up = (part > 0.5) | ((part == 0.5) & (low % 2 == 1))
    else:
        r = np.zeros((rows, blocks * block))
        r[:, :cols] = (bits + 0.5) / 65536
        up = part + r.reshape(z.shape) >= 1
    c = np.where(bad[:, :, None], 0, low + up + np.where(np.signbit(z), 8, 0))
    code = np.where(bad, 255 if block == 32 else 127, code)
    return c.reshape(rows, -1)[:, :cols].astype(np.uint8), code.astype(np.uint8), factor


def fp4_dequantize(codes, scale_codes, factor, block):
    """The numbers that codes stand for, float64."""
    s = scale_codes.astype(np.int64)
    if block == 32:
        v = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    else:
        v = np.where(s == 127, np.nan, E4M3[np.minimum(s, 126)]) * factor
    v = np.repeat(v, block, 1)[:, :codes.shape[1]]
    return np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7] * v


def fp4_pack(codes, scale_codes, block):
    """The bytes of codes and scales in the library's layout (fp4_matrix in include/muon.h)."""
    rows, cols = codes.shape
    full = np.zeros((rows, -(-cols // 32) * 32), np.uint8)
    full[:, :cols] = codes
    tiles = -(-cols // 256) * 64 // block
    out = np.zeros((-(-rows // 128) * tiles * 512,), np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(scale_codes.shape[1]), indexing="ij")
    out[(r // 128 * tiles + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = scale_codes
    return full[:, 0::2] | full[:, 1::2] << 4, out
