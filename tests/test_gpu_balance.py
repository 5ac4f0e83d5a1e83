"""GPU parity of balance_loss and its backward with the oracle (float64).

Tolerances, before any run.  Counts and token numbers are exact.  A
probability is off by a few float32 roundings of its exponent's argument, up
to D = the row's range of logits: relatively 2^-21 (1 + D); means and the
balance loss inherit it (they are sums of positive terms in float32, 2^-19
more for long sums).  lse is off by 2^-21 (1 + max |lse|), z by twice that
times max |lse|.  A gradient entry is a product of p with a difference of
terms of size w = |gb| E / (G' N) (max f + sum f p) + 2 |gz lse| / N: off by
2^-20 (1 + D) p w, and half a spacing where it is bfloat16."""

import numpy as np
import pytest
import torch

import oracle
from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu
KIND = {"f32": torch.float32, "bf16": torch.bfloat16}


def case(tokens, experts, top, kind, seed=0, masked=0.0, drop=0.05, spread=1.5):
    rng = np.random.default_rng(seed + tokens * 31 + experts)
    x = torch.from_numpy((rng.standard_normal((tokens, experts)) * spread).astype(np.float32)).to(KIND[kind])
    ids = np.argsort(rng.random((tokens, experts)), axis=1)[:, :top]
    ids = np.where(rng.random(ids.shape) < drop, -1, ids)
    mask = rng.random(tokens) >= masked if masked else None
    return x, ids.astype(np.int64), mask


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(x, X, ids, mask, groups, gb=0.7, gz=0.3, out=None):
    want = oracle.balance_loss(x, ids, mask, groups)
    M = dev(mask)
    r = muon.balance_loss(X, dev(ids), mask=M, groups=groups)
    np.testing.assert_array_equal(r.counts.cpu().numpy(), want["counts"])
    np.testing.assert_array_equal(r.tokens.cpu().numpy(), want["tokens"])
    live = np.ones(len(x), bool) if mask is None else mask
    z = x[live] if live.any() else np.zeros((1, x.shape[1]))
    fin = np.where(np.isfinite(z), z, 0)
    D = float((fin.max(axis=1) - fin.min(axis=1)).max())
    lse = float(np.abs(np.log(np.exp(z - z.max(axis=1, keepdims=True)).sum(axis=1)) + z.max(axis=1)).max())
    eps = 2.0 ** -21 * (1 + D)
    assert (np.abs(host(r.mean_probs) - want["mean"]) <= (eps + 2.0 ** -19) * want["mean"] + 1e-40).all()
    assert abs(float(r.balance) - want["balance"]) <= (eps + 2.0 ** -18) * want["balance"]
    assert abs(float(r.z) - want["z"]) <= 2.0 ** -20 * (1 + lse) * max(lse, 1) + 2.0 ** -19 * want["z"]
    g = torch.tensor([gb], device="cuda"), torch.tensor([gz], device="cuda")
    G = muon.balance_loss_backward(X, r, *g, mask=M, out=out)
    wg = oracle.balance_loss_grad(x, ids, np.float32(gb), np.float32(gz), mask, groups)
    with np.errstate(invalid="ignore"):
        p = np.exp(x - x.max(axis=1, keepdims=True))
        p = p / p.sum(axis=1, keepdims=True)
    p = np.where(live[:, None], p, 0)
    E, some, kept = x.shape[1], max(1, (want["tokens"] > 0).sum()), max(1, want["tokens"].sum())
    f = want["counts"] / np.maximum(1, want["counts"].sum(axis=1, keepdims=True))
    n = np.maximum(1, want["tokens"])[:, None]
    w = abs(gb) * E / some / n * (f.max(axis=1, keepdims=True) * 2 + 1.0 / E)
    w = np.repeat(w, len(x) // groups, axis=0) + 2 * abs(gz) * max(lse, 1) / kept
    tol = 2 * eps * p * w + 2.0 ** -22 * np.abs(wg) + 1e-42
    if G.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * 1.01 * np.abs(wg) + 2.0 ** -133
    bad = np.abs(host(G) - wg) > tol
    assert not bad.any(), (int(bad.sum()), float(np.abs(host(G) - wg).max()))
    assert not host(G)[~live].any()
    return r


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("experts", [1, 2, 3, 8, 9, 31, 60, 64, 160, 161, 255, 256, 257, 511, 512, 520, 1000, 1024])
def test_every_number_of_experts(experts, kind):
    x, ids, mask = case(150, experts, min(4, experts), kind, masked=0.2)
    check(host(x), x.cuda(), ids, mask, 3)


@pytest.mark.parametrize("tokens,groups", [(1, 1), (2, 2), (7, 1), (8, 4), (33, 3), (1000, 1), (1000, 1000), (4096, 8),
                                           (20_003, 1), (30_000, 2)])
def test_tokens_and_groups(tokens, groups):
    x, ids, _ = case(tokens, 24, 2, "f32")
    check(host(x), x.cuda(), ids, None, groups)
    x, ids, mask = case(tokens, 17, 3, "bf16", masked=0.4)
    check(host(x), x.cuda(), ids, mask, groups)


def test_long_batch_in_float32():
    x, ids, mask = case(60_000, 64, 6, "f32", masked=0.1)
    check(host(x), x.cuda(), ids, mask, 1)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("experts,pad,shift", [(64, 1, 0), (64, 8, 0), (64, 0, 1), (10, 6, 8), (33, 3, 2)])
def test_row_pitch_offset_and_in_place(kind, experts, pad, shift):
    x, ids, mask = case(90, experts, 2, kind, masked=0.3)
    flat = torch.full((90 * (experts + pad) + shift,), 1e30, dtype=KIND[kind], device="cuda")[shift:]
    X = flat.view(90, experts + pad)[:, :experts]
    X.copy_(x)
    check(host(x), X, ids, mask, 2)
    check(host(x), X, ids, mask, 2, out=X)
    if pad:  # what lies between the rows is untouched
        assert bool((flat.view(90, -1)[:, experts:].float() > 9e29).all())


def test_groups_and_batches_without_tokens():
    x, ids, _ = case(40, 12, 3, "f32")
    mask = np.ones(40, bool)
    mask[10:20] = False
    check(host(x), x.cuda(), ids, mask, 4)
    x[10:20] = float("nan")  # masked tokens are not read
    r = check(np.nan_to_num(host(x)), x.cuda(), ids, mask, 4)
    assert not r.mean_probs[1].any()
    r = check(np.nan_to_num(host(x)), x.cuda(), ids, np.zeros(40, bool), 4)
    assert float(r.balance) == 0 and float(r.z) == 0
    r = muon.balance_loss(torch.zeros((0, 8), device="cuda"), torch.zeros((0, 2), dtype=torch.int64, device="cuda"), groups=3)
    assert float(r.balance) == 0 and not r.counts.any() and r.counts.shape == (3, 8)


def test_masked_gradient_is_zero_whatever_the_scale():
    x, ids, mask = case(20, 8, 2, "f32", masked=0.5)
    r = muon.balance_loss(x.cuda(), dev(ids), mask=dev(mask))
    bad = torch.tensor([float("inf")], device="cuda")
    G = muon.balance_loss_backward(x.cuda(), r, bad, bad, mask=dev(mask))
    assert not G[~dev(mask)].any()


def test_no_assignment_counts():
    x, ids, _ = case(30, 6, 2, "f32")
    ids[:] = -1
    ids[3] = 6
    ids[4] = 2 ** 40
    r = check(host(x), x.cuda(), ids, None, 1)
    assert not r.counts.any() and float(r.balance) == 0


def test_masked_experts_and_non_finite_rows():
    x, ids, _ = case(64, 20, 2, "f32")
    x[:, 15:] = -float("inf")
    check(host(x), x.cuda(), np.minimum(ids, 14), None, 2)
    x[5, 3] = float("nan")
    r = muon.balance_loss(x.cuda(), dev(ids), groups=2)
    assert torch.isnan(r.mean_probs).any(dim=1).tolist() == [True, False] and torch.isnan(r.balance)
    G = muon.balance_loss_backward(x.cuda(), r, torch.ones(1, device="cuda"), torch.ones(1, device="cuda"))
    assert torch.isnan(G[5]).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("experts", [16, 21, 256, 301, 520, 1024])
def test_experts_masked_with_the_lowest_value(experts, kind):
    """A mask of the type's lowest value over some experts, and over whole rows, whose
    probabilities are then equal; the balance loss and its gradient are as in any other row."""
    x, ids, _ = case(64, experts, 2, kind, seed=3)
    x[:, experts // 2] = x[::2, 3] = x[7] = x[33] = torch.finfo(KIND[kind]).min
    z = host(x)
    want, one, zero = oracle.balance_loss(z, ids, None, 4), torch.ones(1, device="cuda"), torch.zeros(1, device="cuda")
    X = x.cuda()
    r = muon.balance_loss(X, dev(ids), groups=4)
    live = np.where(z > -1e30, z, 0)
    D = float((live.max(axis=1) - live.min(axis=1)).max())
    eps = 2.0 ** -21 * (1 + D)
    assert (np.abs(host(r.mean_probs) - want["mean"]) <= (eps + 2.0 ** -19) * want["mean"] + 1e-40).all()
    assert abs(float(r.balance) - want["balance"]) <= (eps + 2.0 ** -18) * want["balance"]
    G = host(muon.balance_loss_backward(X, r, one, zero))
    wg = oracle.balance_loss_grad(z, ids, np.float32(1), np.float32(0), None, 4)
    p = np.exp(z - z.max(axis=1, keepdims=True))
    p = p / p.sum(axis=1, keepdims=True)
    f = want["counts"] / want["counts"].sum(axis=1, keepdims=True)
    w = np.repeat(experts / 4 / 16 * (f.max(axis=1, keepdims=True) * 2 + 1.0 / experts), 16, axis=0)
    tol = 2 * eps * p * w + 2.0 ** -22 * np.abs(wg) + 1e-42
    if kind == "bf16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * 1.01 * np.abs(wg) + 2.0 ** -133
    assert (np.abs(G - wg) <= tol).all()


def test_equal_calls_and_other_stream_give_equal_bits():
    x, ids, mask = case(50_000, 96, 4, "bf16", masked=0.1)
    X, I, M = x.cuda(), dev(ids), dev(mask)
    a = muon.balance_loss(X, I, mask=M, groups=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = muon.balance_loss(X, I, mask=M, groups=5)
    torch.cuda.current_stream().wait_stream(s)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_workspace_is_reused_whatever_it_holds():
    x, ids, _ = case(3000, 40, 2, "f32")
    ws = torch.full((muon.balance_loss_workspace_size(3000, 40, 3),), 0xAB, dtype=torch.uint8, device="cuda")
    a = muon.balance_loss(x.cuda(), dev(ids), groups=3, workspace=ws)
    b = muon.balance_loss(x.cuda(), dev(ids), groups=3)
    assert torch.equal(a.saved, b.saved) and torch.equal(a.mean_probs, b.mean_probs)
    with pytest.raises(muon.MuonError):
        muon.balance_loss(x.cuda(), dev(ids), groups=3, workspace=ws[:256])


def test_gradient_matches_differences():
    """Central differences of the GPU's own losses, step 2^-4 on one token of four: curvature 2^-9, rounding 2^-18."""
    x, ids, _ = case(4, 5, 2, "f32", drop=0.0)
    gb, gz = 1.0, 0.5

    def loss(y):
        r = muon.balance_loss(y.cuda(), dev(ids))
        return gb * float(r.balance) + gz * float(r.z)

    r = muon.balance_loss(x.cuda(), dev(ids))
    G = muon.balance_loss_backward(x.cuda(), r, torch.tensor([gb], device="cuda"), torch.tensor([gz], device="cuda"))
    for t in range(4):
        for e in range(5):
            d = torch.zeros_like(x)
            d[t, e] = 2.0 ** -4
            assert abs((loss(x + d) - loss(x - d)) / 2.0 ** -3 - float(G[t, e])) < 2.0 ** -9


def test_refusals_on_device():
    x, ids, mask = case(12, 8, 2, "f32", masked=0.2)
    X, I = x.cuda(), dev(ids)
    with pytest.raises(muon.MuonError):
        muon.balance_loss(X, I, groups=5)
    with pytest.raises(ValueError):
        muon.balance_loss(X, I, mask=torch.ones(11, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        muon.balance_loss(X, I, mask=torch.ones(12, device="cuda"))
    with pytest.raises(TypeError):
        muon.balance_loss(X.half(), I)
    r = muon.balance_loss(X, I)
    one = torch.ones(1, device="cuda")
    with pytest.raises(ValueError):
        muon.balance_loss_backward(X[:, :7], r, one, one)
    with pytest.raises(ValueError):
        muon.balance_loss_backward(X, r, one.double(), one)
