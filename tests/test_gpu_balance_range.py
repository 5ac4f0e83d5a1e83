"""balance_loss and its backward where router scores are large: whole rows at
mask constants of every size, rows that stand far from zero.

Tolerances, before any run.  Exponents are differences within a row, so a
probability's error does not grow with the scores: with D the range of a
row's live scores, relatively 2^-21 (1 + D), and 2^-19 more for long sums (as
for scores of ordinary size).  lse is off by 2^-21 (1 + log E) + 2^-22 |lse|,
its square by 2 |lse| times that (2^-19 of the mean for the sum)."""

import numpy as np
import pytest
import torch

import oracle
from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu
KIND = {"f32": torch.float32, "bf16": torch.bfloat16}
CONSTANTS = (1e3, -1e3, 1e4, -1e4, 1e6, -1e6, -1e9, 1e10, -1e10, 1e12, -1e12, -1e18, 1e18)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("experts", [16, 21, 64, 256, 300, 520, 1024])
def test_rows_at_large_constants(experts, kind):
    """Every third row ordinary, every third a constant throughout, every third a constant plus ordinary scores."""
    rng = np.random.default_rng(experts)
    tokens, groups, top = 3 * 4 * len(CONSTANTS), 4, 2
    x = rng.standard_normal((tokens, experts)) * 1.5
    c = np.repeat(np.array(CONSTANTS), 12)
    x[1::3] = c[1::3, None]
    x[2::3] += c[2::3, None]
    X = torch.from_numpy(x.astype(np.float32)).to(KIND[kind]).cuda()
    x = host(X)
    ids = rng.integers(0, experts, (tokens, top))
    I = torch.from_numpy(ids).cuda()
    want = oracle.balance_loss(x, ids, None, groups)
    r = muon.balance_loss(X, I, groups=groups)
    p = np.exp(x - x.max(axis=1, keepdims=True))
    s = p.sum(axis=1, keepdims=True)
    p, lse = p / s, (x.max(axis=1, keepdims=True) + np.log(s))[:, 0]
    d = np.where(p > 0, x.max(axis=1, keepdims=True) - x, 0)
    eps = 2.0 ** -21 * (1 + float(d.max()))
    assert (np.abs(host(r.mean_probs) - want["mean"]) <= (eps + 2.0 ** -19) * want["mean"] + 1e-40).all()
    assert abs(float(r.balance) - want["balance"]) <= (eps + 2.0 ** -18) * want["balance"]
    t_lse = 2.0 ** -21 * (1 + np.log(experts)) + 2.0 ** -22 * np.abs(lse)
    assert abs(float(r.z) - want["z"]) <= (2 * np.abs(lse) * t_lse).mean() + 2.0 ** -19 * want["z"]
    one, zero = torch.ones(1, device="cuda"), torch.zeros(1, device="cuda")
    for gb, gz in ((one, zero), (zero, one)):
        G = host(muon.balance_loss_backward(X, r, gb, gz))
        wg = oracle.balance_loss_grad(x, ids, float(gb), float(gz), None, groups)
        f = want["counts"] / want["counts"].sum(axis=1, keepdims=True)
        w = np.repeat(experts / groups / (tokens // groups) * (f.max(axis=1, keepdims=True) * 2 + 1.0 / experts), tokens // groups, axis=0)
        w = float(gb) * w + float(gz) * 2 / tokens * (np.abs(lse) * (1 + 2.0 ** -19) + 1)[:, None]
        tol = 2 * eps * p * w + 2.0 ** -22 * np.abs(wg) + 2 * float(gz) / tokens * p * t_lse[:, None] + 1e-42
        if kind == "bf16":
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * 1.01 * np.abs(wg) + 2.0 ** -133
        bad = ~(np.abs(G - wg) <= tol)
        assert not bad.any(), (int(bad.sum()), np.unique(c[bad.any(axis=1)]))


def test_vector_and_tile_layouts_agree():
    """The same scores at a pitch that the vector path takes and at one that it does not."""
    x = torch.full((24, 64), 0.0, device="cuda") + torch.tensor([float(c) for c in (0, 1e4, -1e9, -1e10, 1e12, -1e20)], device="cuda").repeat(4)[:, None]
    ids = torch.arange(48, device="cuda").view(24, 2) % 64
    odd = torch.zeros((24, 65), device="cuda")[:, :64].copy_(x)
    one = torch.ones(1, device="cuda")
    a, b = (muon.balance_loss(t, ids) for t in (x, odd))
    for r, t in ((a, x), (b, odd)):
        assert float((r.mean_probs * 64 - 1).abs().max()) <= 2.0 ** -19 and abs(float(r.balance) - 1) <= 2.0 ** -18
        assert not muon.balance_loss_backward(t, r, one, torch.zeros(1, device="cuda")).isnan().any()
