"""Layer norm of rows that have no spread, or hardly any, and of rows near the ends of float32's range.

A constant row's sum and 1 / cols are rounded, so its mean may be some steps off in the first place; the mean of the
differences takes that off again. Its error is (D u)^2 of the constant then, D of up to a few hundred additions and
u = 2^-24: less than half a step of it, so that mean, differences and variance are exact."""

import numpy as np
import pytest
import torch

from newton_schulz_08_gb300 import muon
from tests.test_gpu_layer_norm import check_backward, check_forward, f64, make, within

pytestmark = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32
U = 2.0 ** -24
VALUES = (0.1, -1.7, 100000.3, 3.0e-30, -7.0e20)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("kind", [B, F])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 1)])
@pytest.mark.parametrize("rows,cols", [(1500, 3), (900, 127), (40, 768), (900, 768), (700, 1217), (700, 1600), (20, 1601),
                                       (30, 5001), (400, 12289), (12, 20001), (7, 60_001), (6, 100_000)])
def test_constant_rows(rows, cols, pad, offset, kind, residual):
    x, w, b = make(rows, cols, kind, pad, offset), make(1, cols, F, seed=1)[0], make(1, cols, F, seed=2)[0]
    # a residual of another pitch keeps long rows out of the kernels that hold them
    res = make(rows, cols, kind, pad + (3 if cols > 50_000 else 0), offset, seed=3) if residual else None
    flat = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for k, v in enumerate(VALUES):
        flat[k::9] = True
        x[k::9] = v
        if residual:
            res[k::9] = v / 4
    r = muon.layer_norm(x, w, b, residual=res)
    s = x if res is None else r.sum
    c = s[flat]
    assert torch.equal(r.mean[flat], c[:, 0].float())
    within(r.rstd[flat], np.full(c.shape[0], 1e-5 ** -0.5), 5 * U * 1e-5 ** -0.5, "rstd")
    assert torch.equal(r.y[flat], b.to(kind).expand_as(c))  # (x - mean) is 0
    others = muon.LayerNorm(r.y[~flat], r.mean[~flat], r.rstd[~flat])
    check_forward(others, s[~flat], w, b, 1e-5)
    none = muon.layer_norm(x, w, b, eps=0.0, residual=res)
    assert torch.equal(none.y.isnan().all(1), flat) and torch.equal(none.y.isnan().any(1), flat)


@pytest.mark.parametrize("rows,cols", [(900, 100), (900, 768), (300, 1601), (100, 12289), (4, 100_000)])
@pytest.mark.parametrize("kind", [B, F])
def test_rows_that_differ_in_one_entry(rows, cols, kind):
    """A spread of one step of the type in one entry, the least there is: still the formula's row, whose variance is
    known to (D + 8) u of itself as the differences are exact multiples of the spacing and so few."""
    x = torch.full((rows, cols), 1.25, device="cuda").to(kind)
    at = torch.arange(rows, device="cuda") % cols
    step = 2.0 ** -7 if kind == B else 2.0 ** -23
    x[torch.arange(rows, device="cuda"), at] = 1.25 + step
    r = muon.layer_norm(x, eps=0.0)
    D = 64 + cols / 1024
    true = f64(x)
    mean = true.mean(1)
    var = np.square(true - mean[:, None]).mean(1)
    # the mean is rounded to half its spacing, 2^-24, which the differences have then; and theirs in the mean of squares
    e_mean = 2.0 ** -24 + D * U * step / cols
    within(r.mean, mean, np.full(rows, e_mean), "mean")
    e_var = (2 * np.abs(true - mean[:, None]) * e_mean + e_mean ** 2).mean(1) + (D + 8) * U * var
    rstd = f64(r.rstd)
    assert ((rstd >= (var + e_var) ** -0.5 * (1 - 8 * U)) & (rstd <= np.maximum(var - e_var, 0) ** -0.5 * (1 + 8 * U))).all()


@pytest.mark.parametrize("rows,cols", [(41, 1), (41, 5), (900, 33), (37, 100), (301, 257), (900, 601), (41, 1000), (33, 1601),
                                       (900, 2047), (20, 5001), (9, 12_290), (5, 20_001)])
@pytest.mark.parametrize("kind", [B, F])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 1)])
@pytest.mark.parametrize("value,eps", [(2.0 ** 100, 1e-20), (-2.0 ** 113, 1e-12)])
def test_gradients_of_constant_rows_far_from_zero(value, eps, pad, offset, kind, rows, cols):
    """mean rstd is past float32's range, every difference is 0: grad_x = rstd (gw - mean(gw)), nothing for the weight's."""
    x, g, gs = (make(rows, cols, kind, pad, offset, seed=k) for k in range(3))
    w = make(1, cols, F, seed=3)[0]
    x[::5], x[-1] = value, value
    r = muon.layer_norm(x, w, eps=eps)
    assert bool((r.mean[::5].double() * r.rstd[::5].double()).abs().ge(2.0 ** 128).all())
    check_backward(muon.layer_norm_backward(g, x, r.mean, r.rstd, w, grad_sum=gs), g, x, r.mean, r.rstd, w, gs)
    check_backward(muon.layer_norm_backward(g, x, r.mean, r.rstd, w), g, x, r.mean, r.rstd, w, None)


def test_rows_past_float32s_range():
    """What the header says of them: NaN where the sum is infinite, rstd 0 (and the bias) where the sum of squares is."""
    x = torch.zeros(3, 64, device="cuda")
    x[0, ::2], x[0, 1::2] = 1e30, -1e30
    x[1] = 1e37
    b = torch.arange(64.0, device="cuda")
    r = muon.layer_norm(x, None, b)
    assert float(r.rstd[0]) == 0 and torch.equal(r.y[0], b)
    assert r.y[1].isnan().all() and torch.equal(r.y[2], b)
