"""Pins of the oracle for the 4-bit format and layer norm (CPU): every code and
scale tried in rational arithmetic, the mean of the stochastic rounding, the
bytes of the layout, torch's autograd and differences."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle.fp4 import E4M3, GRID


def test_e4m3_numbers_are_torchs():
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(E4M3, want)


def nearest(y, even_of):
    """Index of the grid number nearest to a Fraction, ties to the even index."""
    grid = [Fraction(float(g)) for g in GRID]
    d = [abs(y - g) for g in grid]
    at = [i for i in range(8) if d[i] == min(d)]
    return at[0] if len(at) == 1 else [i for i in at if i % 2 == 0][0]


@pytest.mark.parametrize("block", [32, 16])
def test_codes_by_trying_all(block):
    rng = np.random.default_rng(block)
    x = oracle.round_to_bf16(rng.standard_normal((6, 2 * block)) * np.exp(3 * rng.standard_normal((6, 1))))
    x[0, :7] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]   # ties once the block's largest is 6
    x[0, 7:block] = 0.0
    x[0, 7] = -6.0
    codes, scales, factor = oracle.fp4_quantize(x, block)
    k = Fraction(factor)
    if block == 16:  # the smallest power of two that lets every block's scale fit
        assert Fraction(float(np.abs(x).max())) <= 2688 * k and Fraction(float(np.abs(x).max())) > 2688 * k / 2
    for r in range(x.shape[0]):
        for b in range(2):
            part = [Fraction(float(v)) for v in x[r, b * block:(b + 1) * block]]
            top = max(abs(v) for v in part)
            if block == 32:
                s = Fraction(2) ** (int(scales[r, b]) - 127)
                assert top <= 6 * s and (top > 3 * s or top == 0)
            else:
                q = Fraction(float(np.float32(float(top)) / np.float32(6))) / k
                d = [abs(Fraction(float(v)) - q) for v in E4M3]
                assert d[int(scales[r, b])] == min(d)
                s = Fraction(float(E4M3[scales[r, b]])) * k
            for i, v in enumerate(part):
                y = Fraction(float(np.float32(float(abs(v) / s)))) if s else Fraction(0)
                c = int(codes[r, b * block + i])
                assert c & 7 == nearest(min(y, Fraction(6)), GRID), (r, b, i)
                assert (c >> 3) == (1 if v < 0 else 0)


@pytest.mark.parametrize("block", [32, 16])
def test_stochastic_rounding_is_right_in_the_mean(block):
    """Over all 65536 random numbers, the mean of an entry's values is the entry up to half a unit of the random
    numbers' last bit: a step (at most 2 scales) / 131072."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((1, block)).astype(np.float32).astype(np.float64)
    total = np.zeros(block)
    for r in range(0, 65536, 64):
        xs = np.repeat(x, 64, 0)
        bits = np.repeat(np.arange(r, r + 64)[:, None], block, 1)
        c, s, f = oracle.fp4_quantize(xs, block, bits)
        total += oracle.fp4_dequantize(c, s, f, block).sum(0)
    scale = np.abs(x).max() / 6 * 1.25
    # (a quotient by an E4M3 scale is rounded to float32: 2^-24 of at most 6 scales)
    assert np.abs(total / 65536 - x[0]).max() <= 2 * scale / 131072 + 6 * scale * 2.0 ** -24


def test_nothing_is_cut_off_where_rounding_is_stochastic():
    x = np.random.default_rng(0).standard_normal((200, 64)).astype(np.float32).astype(np.float64)
    c, s, f = oracle.fp4_quantize(x, 16, np.zeros(x.shape, np.int64))
    v = E4M3[s] * f
    assert (np.abs(x).reshape(200, 4, 16).max(2) <= 6 * v * (1 + 2.0 ** -23)).all()


def test_blocks_that_are_not_finite():
    x = np.zeros((2, 64))
    x[0, 3], x[1, 40] = np.nan, np.inf
    x[0, 40] = 5.0
    # 5 by a scale of 1 is midway between 4 and 6; by 416 2^-9 (5 / 6 = 426.7 2^-9) it is above 6
    for block, nan, five in ((32, 255, 4.0), (16, 127, 6 * 416 / 512)):
        c, s, f = oracle.fp4_quantize(x, block)
        v = oracle.fp4_dequantize(c, s, f, block)
        assert s[0, 0] == nan and np.isnan(v[0, :block]).all() and v[0, 40] == five
        assert np.isnan(v[1, 32 if block == 32 else 32:48]).all() and not np.isnan(v[1, :32]).any()


def test_layout():
    codes = np.arange(130 * 70, dtype=np.int64).reshape(130, 70).astype(np.uint8) & 15
    scales = np.arange(130 * 3).reshape(130, 3).astype(np.uint8)
    b, s = oracle.fp4_pack(codes, scales, 32)
    assert b.shape == (130, 48) and b[129, 34] == codes[129, 68] | codes[129, 69] << 4 and not b[:, 35:].any()
    assert s.size == 2 * 2 * 512
    assert s[0 * 512 + 5 * 16 + 3 * 4 + 2] == scales[101, 2]
    assert s[2 * 512 + 1 * 16 + 0 * 4 + 1] == scales[129, 1]


def test_random_bits_differ_by_entry_axis_and_seed():
    a = oracle.fp4_bits(64, 65, 5, 1)
    assert 0.9 < np.unique(a).size / (65536 * (1 - np.exp(-a.size / 65536))) < 1.1
    assert (a != oracle.fp4_bits(64, 65, 5, 0)).mean() > 0.99
    assert (a != oracle.fp4_bits(64, 65, 5 + 2 ** 32, 1)).mean() > 0.99
    assert np.array_equal(a[:, :64], oracle.fp4_bits(64, 66, 5, 1)[:, :64])


def test_layer_norm_against_autograd_and_differences():
    rng = np.random.default_rng(1)
    x, w, b, g = rng.standard_normal((5, 9)), rng.standard_normal(9), rng.standard_normal(9), rng.standard_normal((5, 9))
    y, mean, rstd = oracle.layer_norm(x, w, b, 1e-3)
    t = [torch.tensor(v, requires_grad=True) for v in (x, w, b)]
    out = torch.nn.functional.layer_norm(t[0], (9,), t[1], t[2], 1e-3)
    assert np.abs(out.detach().numpy() - y).max() < 1e-13
    want = [v.numpy() for v in torch.autograd.grad(out, t, torch.tensor(g))]
    got = oracle.layer_norm_grad(g, x, mean, rstd, w)
    for a, c in zip(got, want):
        assert np.abs(a - c).max() < 1e-13
    f = lambda v: (oracle.layer_norm(v, w, b, 1e-3)[0] * g).sum()  # noqa: E731
    h = 1e-6
    for i, j in ((0, 0), (2, 5), (4, 8)):
        d = np.zeros_like(x)
        d[i, j] = h
        assert abs((f(x + d) - f(x - d)) / (2 * h) - got[0][i, j]) < 1e-8
