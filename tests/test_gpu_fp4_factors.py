"""4-bit matrices of a program's own arrays whose tensor's factor is any float32, as other programs' weights have it.

fp4_values rounds scale times factor and code times that to float32: (1 + u)^2 - 1 < 2.01 u, u = 2^-24, then to its
type.  fp4_mm rounds the product of the factors and its product with the sum to float32 (2.01 u of the result) and that
to its type, beside the sum's own error: at most K / 64 + 8 roundings of 2^-23 of the sum of magnitudes, times the
factors.  Numbers below 2^-126 have a spacing of 2^-149, half of which each of these roundings may add."""

import pytest
import torch

from newton_schulz_08_gb300 import muon
from tests.test_gpu_fp4 import operands, product

pytestmark = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32
U, LEAST = 2.0 ** -24, 2.0 ** -149
FACTORS = [(1 / 3, 0.7), (1.9999999, 1.25e-3), (-0.3, 5.0), (3e-39, 1e38), (1.5 * 2.0 ** -127, 1.1 * 2.0 ** 116),
           (1.7 * 2.0 ** -80, 1.1 * 2.0 ** -60), (1.3 * 2.0 ** 70, 1.9 * 2.0 ** 63), (0.0, 3.0), (2.0 ** -127, 2.0 ** 116), (1.0, 1.0)]


def half_step(kind):
    return 2.0 ** -8 if kind == B else U


def with_factor(q, factor):
    return muon.FP4(q.codes, q.scales, q.rows, q.cols, 16, scale=torch.tensor([factor, 1.0], device="cuda"))


def numbers(q):
    """Codes times block scales, exact."""
    return muon.fp4_values(with_factor(q, 1.0), F).double()


@pytest.mark.parametrize("factor", sorted({f for pair in FACTORS for f in pair}))
@pytest.mark.parametrize("kind", [B, F])
def test_values(kind, factor):
    q = operands(70, 10, 100, 16)[0]
    f = float(torch.tensor(factor, dtype=F))
    want = numbers(q) * f
    got = muon.fp4_values(with_factor(q, factor), kind).double()
    least = LEAST if kind == F else 2.0 ** -133
    inside = want.abs() < 2.0 ** 127
    assert bool((((got - want).abs() <= want.abs() * (half_step(kind) + 2.02 * U) + 4 * least) | ~inside).all())


@pytest.mark.parametrize("pair", FACTORS)
@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("m,n,k", [(40, 300, 64), (300, 40, 64), (130, 257, 300), (3, 200, 1600), (20, 300, 2500), (2600, 2599, 96)])
def test_products(m, n, k, dtype, pair):
    a, b = operands(m, n, k, 16)
    x, y = numbers(a), numbers(b)
    fa, fb = (float(torch.tensor(f, dtype=F)) for f in pair)
    want, size = x @ y.t() * (fa * fb), x.abs() @ y.abs().t() * abs(fa * fb)
    out = product(with_factor(a, pair[0]), with_factor(b, pair[1]), dtype=dtype).double()
    least = LEAST if dtype == F else 2.0 ** -133
    bound = want.abs() * (half_step(dtype) + 2.02 * U) + size * ((k / 64 + 8) * 2.0 ** -23) * (1 + 2.0 ** -7) + 2 * least
    inside = size < 2.0 ** 127
    assert bool((((out - want).abs() <= bound) | ~inside).all()), float(((out - want).abs() / bound)[inside].max())
    outside = want.abs() > 2.0 ** 128 * (1 + 2.0 ** -7)
    assert bool((out.isinf() | ~outside).all()) and not bool(out.isnan().any())
