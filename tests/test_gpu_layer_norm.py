"""Layer norm and its gradients on the GPU against the float64 oracle.

Bounds, with u = 2^-24 and D = 64 + cols / 1024 additions in a chain (a
thread's entries, then lanes, warps): the mean is off by at most D u mean|x|;
a difference d = x - mean by that and u|d|; the variance by the mean of
2|d| err(d) and (D + 3) u of itself, rstd by half of that relative to
variance + eps and 4 u; products and the last sum by 4 u of their size; and the
result by half a step of its type (2^-8 or 2^-24).  The gradients take mean
and rstd as the kernel gave them; sums over rows are at most `rows` additions
of u each, relative to the sum of magnitudes."""

import numpy as np
import pytest
import torch

import oracle
from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32
U = 2.0 ** -24


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def half_step(kind):
    return 2.0 ** -8 if kind == B else U


def within(got, want, bound, what):
    off = np.abs(f64(got) - want)
    assert (off <= bound).all(), (what, float((off / np.maximum(bound, 1e-300)).max()))


def check_forward(r, x, w, b, eps):
    x = f64(x)
    n = x.shape[1]
    w = np.ones(n) if w is None else f64(w)
    b = np.zeros(n) if b is None else f64(b)
    y, mean, rstd = oracle.layer_norm(x, w, b, eps)
    D = 64 + n / 1024
    d = x - mean[:, None]
    e_mean = D * U * np.abs(x).mean(1) + U * np.abs(mean)
    e_d = e_mean[:, None] + U * np.abs(d)
    var = np.square(d).mean(1)
    e_var = (2 * np.abs(d) * e_d + e_d ** 2).mean(1) + (D + 3) * U * var
    rel = 0.5 * e_var / (var + eps) * (1 + e_var / (var + eps)) + 4 * U
    xhat = d * rstd[:, None]
    e_xhat = (e_d + U * np.abs(d)) * rstd[:, None] * (1 + rel[:, None]) + np.abs(xhat) * rel[:, None]
    e_y = np.abs(w) * e_xhat + 4 * U * (np.abs(xhat * w) + np.abs(b))
    within(r.mean, mean, e_mean, "mean")
    within(r.rstd, rstd, rstd * rel, "rstd")
    within(r.y, y, e_y + half_step(r.y.dtype) * (np.abs(y) + e_y) + 2.0 ** -133, "y")


def check_backward(got, g, x, mean, rstd, w, grad_sum, columns=True):
    grad_x, grad_w, grad_b = got
    g, x, mean, rstd = f64(g), f64(x), f64(mean), f64(rstd)
    rows, n = x.shape
    w1 = np.ones(n) if w is None else f64(w)
    want = oracle.layer_norm_grad(g, x, mean, rstd, w1)
    gs = np.zeros_like(x) if grad_sum is None else f64(grad_sum)
    D = 64 + n / 1024
    xhat, gw = (x - mean[:, None]) * rstd[:, None], g * w1
    c1, c2 = gw.mean(1, keepdims=True), (gw * xhat).mean(1, keepdims=True)
    e1 = (D + 2) * U * np.abs(gw).mean(1, keepdims=True)
    e2 = (D + 5) * U * np.abs(gw * xhat).mean(1, keepdims=True)
    e = rstd[:, None] * (e1 + np.abs(xhat) * e2 + 6 * U * (np.abs(gw) + np.abs(c1) + np.abs(xhat * c2))) + U * np.abs(gs)
    dx = want[0] + gs
    within(grad_x, dx, e + half_step(grad_x.dtype) * (np.abs(dx) + e) + 2.0 ** -133, "grad_x")
    if w is not None and columns:
        within(grad_w, want[1], (rows + 4) * U * np.abs(g * xhat).sum(0) + 2.0 ** -140, "grad_weight")
    if grad_b is not None:
        within(grad_b, want[2], (rows + 1) * U * np.abs(g).sum(0) + 2.0 ** -140, "grad_bias")


def make(rows, cols, kind, pad=0, offset=0, seed=0, mean=0.0):
    g = torch.Generator("cuda").manual_seed(1000 * rows + cols + 7 * seed)
    flat = torch.zeros(rows * (cols + pad) + 16, dtype=kind, device="cuda")
    x = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    x.copy_((torch.randn((rows, cols), generator=g, device="cuda") + mean).to(kind))
    return x


SIZES = [(1, 1), (3, 2), (5, 7), (4, 1600), (130, 31), (77, 256), (300, 257), (64, 512), (300, 768), (50, 1000), (20, 1024),
         (20, 1025), (33, 2048), (33, 2049), (700, 1600), (33, 4096), (9, 5000), (20, 8192), (9, 8193), (20, 12289), (9, 16384), (7, 16385),
         (5, 20000), (3, 40001), (2, 300_000), (3000, 96)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("kind,weights", [(B, F), (B, B), (F, F), (F, B)])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(rows, cols, kind, weights, residual):
    x, g = make(rows, cols, kind, mean=0.5), make(rows, cols, kind, seed=1)
    w, b = make(1, cols, weights, seed=2)[0], make(1, cols, weights, seed=3)[0]
    res, gs = (make(rows, cols, kind, seed=4), make(rows, cols, kind, seed=5)) if residual else (None, None)
    r = muon.layer_norm(x, w, b, eps=1e-5, residual=res)
    s = x
    if residual:
        s = r.sum
        assert torch.equal(s, (x.float() + res.float()).to(kind))
    check_forward(r, s, w, b, 1e-5)
    got = muon.layer_norm_backward(g, s, r.mean, r.rstd, w, grad_sum=gs)
    check_backward(got, g, s, r.mean, r.rstd, w, gs)
    again = muon.layer_norm_backward(g, s, r.mean, r.rstd, w, grad_sum=gs)
    assert all(torch.equal(a, c) for a, c in zip(got, again))


@pytest.mark.parametrize("kind", [B, F])
@pytest.mark.parametrize("cols", [40, 300, 1601, 12289, 20001])
@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (8, 0), (7, 3)])
def test_views(cols, kind, pad, offset):
    f = lambda k: make(37, cols, kind, pad, offset, seed=k)  # noqa: E731
    x, g, gs, w = f(0), f(1), f(2), make(1, cols, F, seed=3)[0]
    y = make(37, cols, kind, pad + 1, offset)
    flat = torch.as_strided(y, (37 * (cols + pad + 1) - pad - 1 + cols - cols,), (1,)).clone()
    r = muon.layer_norm(x, w, out=y)
    assert r.y is y
    check_forward(r, x, w, None, 1e-5)
    after = torch.as_strided(y, flat.shape, (1,)).clone()
    edge = torch.ones(37, cols + pad + 1, dtype=torch.bool, device="cuda")
    edge[:, :cols] = False
    edge = edge.view(-1)[:flat.numel()]
    assert torch.equal(after[edge], flat[edge])  # what lies between rows is left as it was
    got = muon.layer_norm_backward(g, x, r.mean, r.rstd, w, bias=False, grad_sum=gs, out=f(4))
    assert got[2] is None
    check_backward(got, g, x, r.mean, r.rstd, w, gs)


@pytest.mark.parametrize("cols", [100, 1600, 20001])
@pytest.mark.parametrize("kind", [B, F])
def test_in_place(cols, kind):
    x, g, gs = (make(50, cols, kind, seed=k) for k in range(3))
    w = make(1, cols, F, seed=3)[0]
    r = muon.layer_norm(x, w)
    want = muon.layer_norm_backward(g, x, r.mean, r.rstd, w, grad_sum=gs)
    for at in (g, gs):
        held = at.clone()
        got = muon.layer_norm_backward(g, x, r.mean, r.rstd, w, grad_sum=gs, out=at)
        assert got[0] is at and torch.equal(at, want[0]) and torch.equal(got[1], want[1])
        at.copy_(held)
    y = muon.layer_norm(x, w, out=x).y
    assert y is x and torch.equal(x, r.y)


@pytest.mark.parametrize("cols", [64, 1600, 20001])
def test_no_weight_no_bias(cols):
    x, g = make(40, cols, B), make(40, cols, B, seed=1)
    r = muon.layer_norm(x)
    check_forward(r, x, None, None, 1e-5)
    got = muon.layer_norm_backward(g, x, r.mean, r.rstd, bias=False)
    assert got[1] is None and got[2] is None
    check_backward(got, g, x, r.mean, r.rstd, None, None)
    b = make(1, cols, B, seed=2)[0]
    check_forward(muon.layer_norm(x, None, b), x, None, b, 1e-5)
    got = muon.layer_norm_backward(g, x, r.mean, r.rstd)
    assert got[1] is None
    check_backward(got, g, x, r.mean, r.rstd, None, None)


@pytest.mark.parametrize("cols", [64, 1600, 20001])
@pytest.mark.parametrize("kind", [B, F])
@pytest.mark.parametrize("mean", [100.0, 3e4])
def test_rows_far_from_zero(mean, kind, cols):
    """The variance is of differences with the mean: its error goes with those and with the mean's rounding."""
    x, w = make(30, cols, kind, mean=mean), make(1, cols, F, seed=1)[0]
    check_forward(muon.layer_norm(x, w), x, w, None, 1e-5)


@pytest.mark.parametrize("cols", [64, 1600, 20001])
def test_rows_that_are_constant_or_not_finite(cols):
    x = make(12, cols, F)
    x[1], x[2, 5], x[3, 0], x[4, cols - 1] = 3.0, float("nan"), float("inf"), -float("inf")
    r = muon.layer_norm(x)
    bad = torch.tensor([k in (2, 3, 4) for k in range(12)], device="cuda")
    assert torch.equal(r.y.isnan().all(1), bad) and torch.equal(r.y.isnan().any(1), bad)
    assert not r.y[1].any() and float(r.mean[1]) == 3.0
    zero = muon.layer_norm(x, eps=0.0)  # a constant row has no spread at all
    bad[1] = True
    assert torch.equal(zero.y.isnan().any(1), bad)
    ok = ~bad
    g = make(12, cols, F, seed=1)
    grad_x, _, grad_b = muon.layer_norm_backward(g, x, r.mean, r.rstd)
    check_backward((grad_x[ok], None, None), g[ok], x[ok], r.mean[ok], r.rstd[ok], None, None)
    assert not grad_b.isnan().any() and grad_x[2].isnan().all()


def test_no_rows():
    x = torch.zeros(0, 50, device="cuda")
    w = torch.ones(50, device="cuda")
    r = muon.layer_norm(x, w)
    assert r.y.shape == (0, 50) and r.mean.shape == (0,)
    gx, gw, gb = muon.layer_norm_backward(x, x, r.mean, r.rstd, w)
    assert gx.shape == (0, 50) and not gw.any() and not gb.any() and gw.shape == gb.shape == (50,)


def test_far_offsets():
    rows, cols = 140_000, 16_000
    x = torch.empty(rows, cols, dtype=B, device="cuda")
    x[::1000] = make(140, cols, B)
    x[-1] = make(1, cols, B, seed=1)[0]
    at = torch.cat([torch.arange(0, rows, 1000), torch.tensor([rows - 1])]).cuda()
    w = make(1, cols, F, seed=2)[0]
    r = muon.layer_norm(x, w)
    pick = muon.LayerNorm(r.y[at], r.mean[at], r.rstd[at])
    check_forward(pick, x[at], w, None, 1e-5)
    gx, _, _ = muon.layer_norm_backward(r.y, x, r.mean, r.rstd, w)
    check_backward((gx[at], None, None), pick.y, x[at], pick.mean, pick.rstd, w, None, columns=False)


def test_gradient_of_many_rows():
    """Sums over 100000 rows stay within what their length costs (the formula's bound, far from reached)."""
    x, g = make(100_000, 64, F, mean=1.0), make(100_000, 64, F, seed=1)
    w = make(1, 64, F, seed=2)[0]
    r = muon.layer_norm(x, w)
    _, gw, gb = muon.layer_norm_backward(g, x, r.mean, r.rstd, w)
    want = oracle.layer_norm_grad(f64(g), f64(x), f64(r.mean), f64(r.rstd), f64(w))
    # 608 CTAs of 4 warps: at most 42 rows a lane, 4 groups, 76 parts and 8 warps: 130 additions
    xhat = (f64(x) - f64(r.mean)[:, None]) * f64(r.rstd)[:, None]
    assert (np.abs(f64(gw) - want[1]) <= 134 * U * np.abs(f64(g) * xhat).sum(0)).all()
    assert (np.abs(f64(gb) - want[2]) <= 131 * U * np.abs(f64(g)).sum(0)).all()


def test_differences():
    """grad_x and grad_weight against differences of the kernel's own float32 results summed in float64."""
    x, w, g = make(3, 50, F), make(1, 50, F, seed=1)[0], make(3, 50, F, seed=2)
    r = muon.layer_norm(x, w)
    gx, gw, _ = muon.layer_norm_backward(g, x, r.mean, r.rstd, w)
    f = lambda a, b: float((muon.layer_norm(a, b).y.double() * g.double()).sum())  # noqa: E731
    h = 2.0 ** -7
    # (an error of 1e-6 of about 150 terms of size 1, over 2 h; and h^2 times a third derivative of a few)
    for i, j in ((0, 0), (1, 20), (2, 49)):
        d = torch.zeros_like(x)
        d[i, j] = h
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * h) - float(gx[i, j])) < 3e-3
        e = torch.zeros_like(w)
        e[j] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - float(gw[j])) < 3e-3


@pytest.mark.parametrize("cols", [100, 1600, 1601, 20001])
@pytest.mark.parametrize("kind", [B, F])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_sum_in_place(into, kind, cols):
    """The sum may take the place of x or of residual."""
    x, res, w = make(30, cols, kind), make(30, cols, kind, seed=1), make(1, cols, F, seed=2)[0]
    want = muon.layer_norm(x, w, residual=res)
    y, mean, rstd = torch.empty_like(x), torch.empty(30, device="cuda"), torch.empty(30, device="cuda")
    total = x if into == "x" else res
    muon._call(muon.lib().layer_norm, "layer_norm", 0, None, x.data_ptr(), muon._dtype_code(x), 30, cols, cols, res.data_ptr(),
               cols, w.data_ptr(), None, muon.MUON_F32, 1e-5, y.data_ptr(), cols, total.data_ptr(), cols, mean.data_ptr(),
               rstd.data_ptr())
    for a, b in ((total, want.sum), (y, want.y), (mean, want.mean), (rstd, want.rstd)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [520, 1601, 4099, 9001, 12289])
@pytest.mark.parametrize("kind", [B, F])
def test_in_place_odd(cols, kind):
    """Rows that share 16 bytes with their neighbours, results in place of what is read."""
    x, g, gs = (make(300, cols, kind, seed=k) for k in range(3))
    w, b = make(1, cols, F, seed=3)[0], make(1, cols, F, seed=4)[0]
    r = muon.layer_norm(x, w, b)
    check_forward(r, x, w, b, 1e-5)
    want = muon.layer_norm_backward(g, x, r.mean, r.rstd, w, grad_sum=gs)
    check_backward(want, g, x, r.mean, r.rstd, w, gs)
    for at in (g, gs):
        held = at.clone()
        got = muon.layer_norm_backward(g, x, r.mean, r.rstd, w, grad_sum=gs, out=at)
        assert torch.equal(at, want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        at.copy_(held)
    assert muon.layer_norm(x, w, b, out=x).y is x and torch.equal(x, r.y)


@pytest.mark.parametrize("rows,cols", [(5, 800), (70, 1601), (2000, 777), (40, 9000), (33, 12289), (4, 30001), (9, 2049)])
@pytest.mark.parametrize("kind", [B, F])
@pytest.mark.parametrize("pads", [(7, 0, 1), (0, 3, 2), (1, 1, 5)])
def test_results_at_other_offsets(pads, kind, rows, cols):
    """x and residual of one pitch, y of another, at offsets that move against one another from row to row."""
    x, res = make(rows, cols, kind, pads[0], pads[1]), make(rows, cols, kind, pads[0], pads[1], seed=1)
    w, b = make(1, cols, B, seed=2)[0], make(1, cols, B, seed=3)[0]
    for residual in (None, res):
        y = make(rows, cols, kind, pads[2], 1, seed=4)
        between = torch.as_strided(y, ((rows - 1) * y.stride(0) + cols,), (1,))
        edge = torch.ones(rows, cols + pads[2], dtype=torch.bool, device="cuda")
        edge[:, :cols] = False
        edge = edge.view(-1)[:between.numel()]
        between[edge] = 3.0
        r = muon.layer_norm(x, w, b, residual=residual, out=y)
        s = x if residual is None else r.sum
        if residual is not None:
            assert torch.equal(s, (x.float() + res.float()).to(kind))
        check_forward(r, s, w, b, 1e-5)
        assert (between[edge] == 3.0).all()
