"""How far gradients of one 8-bit block may differ (CPU, the oracle's step,
which the GPU's codes equal bit for bit).

Half of each block's gradients is smaller by a factor.  Rounding v's codes, a
quarter apart at most, leaves a relative variance of at most 0.0156 a step,
over the average's memory 0.0156 / (1 - beta2^2) at the very most and about
half of that in the mean over the place between two codes: 0.08 at beta2 0.95.
The mean of 1 / v then grows by that, the root mean square of u by half of
it: 4 %, 10 % allowed.  Its largest value may be twice the exact one's."""

import numpy as np
import pytest

import oracle

N, STEPS, B1, B2, EPS = 2048, 160, 0.9, 0.95, 1e-12


def updates(ratio, bits8):
    """u of the smaller half over the last hundred steps."""
    rng = np.random.default_rng(0)
    small = np.arange(N) % 256 >= 128
    m = v = np.zeros(N)
    out = []
    for t in range(1, STEPS + 1):
        g = (rng.standard_normal(N) * 1e-3 * np.where(small, ratio, 1.0)).astype(np.float32)
        m, v = oracle.adamw_moments(g, m, v, B1, B2, mode="fp32" if bits8 else "fp64")
        u = oracle.adamw_update(np.zeros(N), m, v, t, 1.0, B1, B2, EPS, 0.0)[1]
        if bits8:
            h = oracle.adamw_bits(3, t, 0, N)
            m, v = (oracle.adamw_dequantize(*oracle.adamw_quantize(x, r, k)).astype(np.float32)
                    for x, r, k in ((m, h & 0xFFFF, "m"), (v, h >> 16, "v")))
        if t > STEPS - 100:
            out.append(u[small])
    return np.array(out)


@pytest.mark.parametrize("power", [0, 4, 8, 12])
def test_updates_within_the_stated_range(power):
    got, want = updates(2.0 ** -power, True), updates(2.0 ** -power, False)
    rms = lambda x: np.sqrt((x ** 2).mean())  # noqa: E731
    assert abs(rms(got) / rms(want) - 1) <= 0.1
    assert np.abs(got).max() <= 2 * np.abs(want).max()


@pytest.mark.parametrize("power", [14, 17, 20])
def test_beyond_it_eps_is_the_bound(power):
    """What the header says of it: large, and below 2^-15 max |m| / eps plus an ordinary update."""
    got = updates(2.0 ** -power, True)
    assert np.abs(got).max() > 2  # not within the range
    assert np.abs(got).max() <= 2.0 ** -15 * 5e-3 / EPS + 10
