"""AdamW with moments in 32 bits or in 8, written out plainly on the CPU --
TEST INFRASTRUCTURE ONLY.

Per element, t = step (counted from 1):
    g' = grad_scale g
    m1 = beta1 m + (1 - beta1) g';     v1 = beta2 v + (1 - beta2) g'^2
    u  = m1 / (sqrt(v1) / sqrt(1 - beta2^t) + eps)
    p1 = p - (lr / (1 - beta1^t) u + lr wd p [mask])
the textbook algorithm with decoupled decay; the mask (cautious only) is 1
where u and p have the same sign.

8-bit moments: blocks of 256 elements share a power-of-two scale.  With
E = floor(log2 max |x|), at least -100, the first moment's scale is 2^(E-7)
with E4M3 codes (3 fraction bits, smallest normal exponent -6), the second's
2^(E-14) with E5M2 codes (2 bits, -14).  Codes are rounded stochastically with
r = (16 bits + 1/2) / 65536: floor(|x| / spacing + r) * spacing; bfloat16
parameters likewise with r = bits / 65536.

Modes: "fp64" is the definition.  "fp32" takes the moments and the product
sums in float32, one rounding per operation in the order above, so that codes
can be compared bit for bit; the update u is float64 in both.
"""

import numpy as np

BLOCK = 256
FORMATS = {"m": (3, -6, 7), "v": (2, -14, 14)}  # fraction bits, least normal exponent, exponent given to the scale
C0, C1, C2, M32 = 0x9E3779B1, 0x6A09E667, 0xBB67AE85, 0xFFFFFFFF


def _mix(x):
    x = np.asarray(x, np.uint64) & np.uint64(M32)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(C1)) & np.uint64(M32)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(C2)) & np.uint64(M32)
    return x ^ (x >> np.uint64(16))


def adamw_bits(seed, step, tensor, n, first=0):
    """32 random bits for elements first .. first+n-1 of tensor number `tensor`."""
    seed &= 2 ** 64 - 1
    s = int(_mix(int(_mix((seed + C0 * step) & M32)) ^ (seed >> 32)))
    key = int(_mix((s + C0 * tensor) & M32))
    i = np.arange(first, first + n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        x = (i & np.uint64(M32)) * np.uint64(C0) + np.uint64(key) + (i >> np.uint64(32)) * np.uint64(C1)
    return _mix(x & np.uint64(M32)).astype(np.uint32)


def _floor_log2(x):
    return np.frexp(x)[1] - 1


def adamw_quantize(x, bits16, kind):
    """Codes' values (in units of the scale) and scales of x: float arrays."""
    mant, least, shift = FORMATS[kind]
    n = x.size
    nb = -(-n // BLOCK)
    pad = lambda a: np.pad(np.asarray(a, np.float64), (0, nb * BLOCK - n)).reshape(nb, BLOCK)  # noqa: E731
    X, r = pad(x), (pad(bits16) + 0.5) / 65536
    a = np.abs(X).max(axis=1) if nb else np.zeros(0)
    bad = ~(a < 2.0 ** 127)
    E = np.clip(_floor_log2(np.where(bad | (a == 0), 1.0, a)), -100, None)
    E = np.where(a == 0, -100, E)
    with np.errstate(invalid="ignore"):
        y = np.ldexp(np.abs(X), (shift - E)[:, None])
        # codes are made from a float32 whose exponent field is the code's: below the smallest
        # normal number it keeps `23 - mant` more bits than the code
        low = np.ldexp(1.0, least - 23)
        y = np.where(y < 2.0 ** least, np.rint(y / low) * low, y)
        grid = np.ldexp(1.0, np.maximum(_floor_log2(np.where(y > 0, y, 2.0 ** least)), least) - mant)
        q = np.copysign(np.floor(y / grid + r) * grid, X)
    return q.reshape(-1)[:n], np.where(bad, np.nan, np.ldexp(1.0, E - shift))


def adamw_dequantize(q, scale):
    return q * np.repeat(scale, BLOCK)[:q.size]


def bf16_stochastic(x, h):
    """x (float64) rounded down or up to bfloat16 with the bits of h."""
    r = ((h.astype(np.uint64) * np.uint64(C0)) & np.uint64(M32)) >> np.uint64(16)
    x = np.asarray(x, np.float32).astype(np.float64)
    with np.errstate(invalid="ignore"):
        grid = np.ldexp(1.0, np.maximum(_floor_log2(np.where(x == 0, 1.0, np.abs(x))), -126) - 7)
        out = np.copysign(np.floor(np.abs(x) / grid + r / 65536.0) * grid, x)
    return np.where(np.isfinite(x), out, x)


def adamw_moments(g, m, v, beta1, beta2, grad_scale=1.0, mode="fp64"):
    if mode == "fp64":
        g = np.asarray(g, np.float64) * grad_scale
        return beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    f = np.float32
    g = np.asarray(g, f) * f(grad_scale)
    with np.errstate(over="ignore", invalid="ignore"):
        return (np.asarray(m, f) * f(beta1) + g * f(1 - beta1), np.asarray(v, f) * f(beta2) + (g * g) * f(1 - beta2))


def adamw_update(p, m1, v1, step, lr, beta1, beta2, eps, weight_decay, cautious=False):
    """(p1, u, decay term) in float64 from the new moments."""
    p, m1, v1 = (np.asarray(a, np.float64) for a in (p, m1, v1))
    with np.errstate(invalid="ignore", divide="ignore"):
        u = m1 / (np.sqrt(v1) / np.sqrt(1 - beta2 ** step) + eps)
        keep = ((u > 0) & (p > 0)) | ((u < 0) & (p < 0)) if cautious else np.ones(p.shape, bool)
        decay = np.where(keep, lr * weight_decay * p, 0.0)
        return p - (lr / (1 - beta1 ** step) * u + decay), u, decay
