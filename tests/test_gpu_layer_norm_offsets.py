"""Layer norm and its gradients where every array has a pitch and an offset of its own, and where rows that begin off 16
bytes alike are so many that each group of warps takes several; what lies before, between and behind rows stays.

Bounds are those of test_gpu_layer_norm."""

import pytest
import torch

from newton_schulz_08_gb300 import muon
from tests.test_gpu_layer_norm import check_backward, check_forward

pytestmark = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32
MARK = 3.0  # beside rows; not what padding in the kernels holds (zeros, or weights of 1)


class Rows:
    """rows x cols in a buffer that holds MARK elsewhere."""

    def __init__(self, rows, cols, kind, pad, offset, seed, mean=0.0):
        self.flat = torch.full((rows * (cols + pad) + 32,), MARK, dtype=kind, device="cuda")
        at = 16 + offset
        self.t = self.flat[at:at + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        g = torch.Generator("cuda").manual_seed(1000 * rows + cols + 7 * seed)
        self.t.copy_((torch.randn((rows, cols), generator=g, device="cuda") + mean).to(kind))

    def beside_is_left(self):
        held = self.t.clone()
        self.t.fill_(MARK)
        left = bool((self.flat == MARK).all())
        self.t.copy_(held)
        return left


# pad and offset of x, residual or grad, sum's gradient, result
LAYOUTS = [((0, 0), (1, 0), (0, 0), (0, 0)), ((3, 1), (5, 2), (1, 3), (2, 0)), ((1, 1), (1, 1), (1, 1), (0, 5)),
           ((0, 1), (0, 3), (0, 7), (0, 2)), ((8, 0), (8, 0), (7, 0), (8, 0)), ((7, 0), (8, 0), (8, 0), (1, 6))]
WIDTHS = [(70, 3), (70, 30), (300, 200), (90, 700), (40, 1601), (30, 2053), (25, 5001), (12, 8199), (9, 12289), (7, 16383),
          (6, 16385), (5, 20001)]


@pytest.mark.parametrize("rows,cols", WIDTHS)
@pytest.mark.parametrize("kind", [B, F])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_every_array_at_its_own_offset(layout, kind, rows, cols):
    x, res, gs, y = (Rows(rows, cols, kind, *p, seed=k) for k, p in enumerate(layout))
    g = Rows(rows, cols, kind, *layout[1], seed=9)
    w, b = (Rows(1, cols, F, 0, 1, seed=k, mean=1.0).t[0] for k in (11, 12))
    for residual in (None, res.t):
        r = muon.layer_norm(x.t, w, b, residual=residual, out=y.t)
        s = x.t if residual is None else r.sum
        if residual is not None:
            assert torch.equal(s, (x.t.float() + res.t.float()).to(kind))
        check_forward(r, s, w, b, 1e-5)
        assert y.beside_is_left()
    for grad_sum in (None, gs.t):
        r = muon.layer_norm(x.t, w, b)
        got = muon.layer_norm_backward(g.t, x.t, r.mean, r.rstd, w, grad_sum=grad_sum, out=y.t)
        check_backward(got, g.t, x.t, r.mean, r.rstd, w, grad_sum)
        assert y.beside_is_left()
        held = got[0].clone()
        again = muon.layer_norm_backward(g.t, x.t, r.mean, r.rstd, w, grad_sum=grad_sum, out=y.t)
        assert torch.equal(held, again[0]) and torch.equal(got[1], again[1]) and torch.equal(got[2], again[2])


@pytest.mark.parametrize("rows,cols", [(9000, 200), (7001, 601), (5000, 769), (5003, 1001), (4001, 1601), (3000, 2049), (2500, 4095),
                                       (1300, 8191)])
@pytest.mark.parametrize("kind", [B, F])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (2, 3)])
def test_rows_alike_many_a_group(pad, offset, kind, rows, cols):
    x, g, gs, y = (Rows(rows, cols, kind, pad, offset, seed=k) for k in range(4))
    w, b = (Rows(1, cols, F, 0, 0, seed=k, mean=1.0).t[0] for k in (11, 12))
    r = muon.layer_norm(x.t, w, b, out=y.t)
    check_forward(r, x.t, w, b, 1e-5)
    assert y.beside_is_left()
    for grad_sum in (None, gs.t):
        got = muon.layer_norm_backward(g.t, x.t, r.mean, r.rstd, w, grad_sum=grad_sum, out=y.t)
        check_backward(got, g.t, x.t, r.mean, r.rstd, w, grad_sum)
        assert y.beside_is_left()


@pytest.mark.parametrize("rows,cols", [(2000, 40), (2000, 201), (2000, 602), (1500, 1003), (1200, 1604), (700, 4097), (500, 9000)])
@pytest.mark.parametrize("kind", [B, F])
def test_rows_not_alike_many_a_group(kind, rows, cols):
    x, g, gs, y = (Rows(rows, cols, kind, p, o, seed=k) for k, (p, o) in enumerate(((0, 1), (1, 0), (2, 3), (5, 2))))
    w = Rows(1, cols, F, 0, 0, seed=5, mean=1.0).t[0]
    r = muon.layer_norm(x.t, w, residual=g.t, out=y.t)
    check_forward(r, r.sum, w, None, 1e-5)
    assert y.beside_is_left()
    r = muon.layer_norm(x.t, w)
    for grad_sum in (None, gs.t):
        got = muon.layer_norm_backward(g.t, x.t, r.mean, r.rstd, w, grad_sum=grad_sum, out=y.t)
        check_backward(got, g.t, x.t, r.mean, r.rstd, w, grad_sum)
        assert y.beside_is_left()


@pytest.mark.parametrize("at", ["grad", "grad_sum"])
@pytest.mark.parametrize("rows,cols", [(900, 201), (700, 1003), (300, 1601), (200, 5001)])
@pytest.mark.parametrize("kind", [B, F])
def test_gradient_in_place_at_other_offsets(kind, rows, cols, at):
    x, g, gs = (Rows(rows, cols, kind, p, o, seed=k) for k, (p, o) in enumerate(((0, 1), (1, 0), (3, 2))))
    w = Rows(1, cols, F, 0, 0, seed=5, mean=1.0).t[0]
    r = muon.layer_norm(x.t, w)
    want = muon.layer_norm_backward(g.t, x.t, r.mean, r.rstd, w, grad_sum=gs.t)
    check_backward(want, g.t, x.t, r.mean, r.rstd, w, gs.t)
    into = g if at == "grad" else gs
    got = muon.layer_norm_backward(g.t, x.t, r.mean, r.rstd, w, grad_sum=gs.t, out=into.t)
    assert all(torch.equal(a, c) for a, c in zip(got, want)) and into.beside_is_left()


def test_sums_over_many_rows_take_few_additions():
    """100000 rows of 64 float32 entries: four lanes a row, 16 entries each; a CTA has 64 rows at a time, of at most 608
    CTAs. So a lane adds 100000 / (64 x CTAs), at most ceil(100000 / 64 / 152) = 11 with a CTA an SM, then 3 over the
    lanes of a column, 7 over the warps, at most 608 / 32 = 19 parts and 5 over the warp that adds them: 45.  Each product
    g xhat has 4 roundings of its own, one of them with the sum."""
    rows = 100_000
    x, g = Rows(rows, 64, F, 0, 0, seed=0, mean=1.0).t, Rows(rows, 64, F, 0, 0, seed=1).t
    w = Rows(1, 64, F, 0, 0, seed=2).t[0]
    r = muon.layer_norm(x, w)
    _, gw, gb = muon.layer_norm_backward(g, x, r.mean, r.rstd, w)
    xhat = (x.double() - r.mean.double()[:, None]) * r.rstd.double()[:, None]
    gd, u = g.double(), 2.0 ** -24
    assert bool(((gw.double() - (gd * xhat).sum(0)).abs() <= 49 * u * (gd * xhat).abs().sum(0)).all())
    assert bool(((gb.double() - gd.sum(0)).abs() <= 46 * u * gd.abs().sum(0)).all())
