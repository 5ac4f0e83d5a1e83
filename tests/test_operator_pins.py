"""Pins of the oracle's AdamW, token log probabilities and balance loss (CPU):
against torch.optim.AdamW, torch's autograd and central differences in
float64, the 8-bit formats' representable values, and the mean of the
stochastic rounding."""

import numpy as np
import pytest
import torch

import oracle
from oracle import adamw as A


def test_adamw_matches_torch_over_steps():
    rng = np.random.default_rng(0)
    p = rng.standard_normal(50)
    P = torch.tensor(p, dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([P], lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    m = v = np.zeros(50)
    for t in range(1, 5):
        g = rng.standard_normal(50)
        P.grad = torch.tensor(g)
        opt.step()
        m, v = oracle.adamw_moments(g, m, v, 0.9, 0.95)
        p, _, _ = oracle.adamw_update(p, m, v, t, 3e-3, 0.9, 0.95, 1e-8, 0.1)
        assert np.abs(p - P.detach().numpy()).max() < 1e-14


@pytest.mark.parametrize("kind,dtype", [("m", torch.float8_e4m3fn), ("v", torch.float8_e5m2)])
def test_codes_are_representable_neighbours(kind, dtype):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal(700) * np.exp(rng.uniform(-30, 3, 700))).astype(np.float32)
    if kind == "v":
        x = np.abs(x)
    bits = rng.integers(0, 65536, 700)
    q, s = oracle.adamw_quantize(x, bits, kind)
    back = torch.tensor(q).to(dtype).to(torch.float64).numpy()
    np.testing.assert_array_equal(q, back)                      # representable
    top = {"m": 256.0, "v": 2.0 ** 15}[kind]
    assert np.abs(q).max() <= top and s.shape == (3,)
    y = x.astype(np.float64) / np.repeat(s, A.BLOCK)[:700]
    down, _ = oracle.adamw_quantize(x, np.zeros(700), kind)     # r = 1/131072: down unless all but at the next code
    up, _ = oracle.adamw_quantize(x, np.full(700, 65535), kind)
    mant, least, _ = A.FORMATS[kind]
    spacing = np.ldexp(1.0, np.maximum(np.frexp(np.abs(y))[1] - 1, least) - mant)  # fixed below the normal numbers
    assert (np.abs(down) <= np.abs(y) + spacing * 2.0 ** -16).all()
    assert (np.abs(up) >= np.abs(y) - spacing * 2.0 ** -16).all()
    assert ((np.abs(q) == np.abs(down)) | (np.abs(q) == np.abs(up))).all()


@pytest.mark.parametrize("kind", ["m", "v"])
def test_codes_zero_extreme_and_not_finite(kind):
    for x, scale_ok in [(np.zeros(5), True), (np.full(5, 2.0 ** -140), True), (np.array([1e38, 1.0]), True),
                        (np.array([3e38, 1.0]), False), (np.array([np.inf, 1.0]), False),
                        (np.array([np.nan, 1.0]), False)]:
        q, s = oracle.adamw_quantize(x.astype(np.float32), np.zeros(x.size), kind)
        assert np.isfinite(s).all() == scale_ok
        if scale_ok:
            v = oracle.adamw_dequantize(q, s)
            assert np.abs(v - x).max() <= 0.25 * np.abs(x).max() + 2.0 ** -116
    q, s = oracle.adamw_quantize(np.array([-3.0, 4.0]), np.zeros(2), "m")
    np.testing.assert_array_equal(oracle.adamw_dequantize(q, s), [-3.0, 4.0])  # exact values stay


def test_rounding_is_unbiased():
    """Mean of 40,000 roundings within 5 standard errors of the value, for both moments and bfloat16."""
    n = 40_000
    h = oracle.adamw_bits(12345678901, 7, 3, n)
    for value in (1.03, 1.24, 1.9):
        x = np.full(n, value, np.float32)
        for q in (oracle.adamw_dequantize(*oracle.adamw_quantize(x, h & 0xFFFF, "m")),
                  oracle.adamw_dequantize(*oracle.adamw_quantize(x, h >> 16, "v")),
                  oracle.bf16_stochastic(x, h)):
            assert abs(q.mean() - float(np.float32(value))) <= 5 * q.std() / np.sqrt(n) + 1e-7


def test_moving_average_follows_its_target():
    """beta2 = 0.999: from a 100 times too large second moment the 8-bit
    average falls as the exact one does (rounding to nearest would stay)."""
    n, v, q, s, exact = 256, None, None, None, 100.0
    q, s = oracle.adamw_quantize(np.full(n, 100.0, np.float32), np.zeros(n), "v")
    for t in range(1, 1001):
        v = oracle.adamw_dequantize(q, s)
        _, v = oracle.adamw_moments(np.ones(n), np.zeros(n), v, 0.9, 0.999, mode="fp32")
        exact = 0.999 * exact + 0.001
        q, s = oracle.adamw_quantize(v, oracle.adamw_bits(5, t, 0, n) >> 16, "v")
    mean = oracle.adamw_dequantize(q, s).mean()
    assert abs(mean / exact - 1) < 0.12   # 35 % spread of one element / sqrt(256), 5 standard errors


def test_random_bits_differ_by_step_tensor_and_seed():
    a = oracle.adamw_bits(1, 1, 0, 4096)
    for b in (oracle.adamw_bits(1, 2, 0, 4096), oracle.adamw_bits(1, 1, 1, 4096), oracle.adamw_bits(2, 1, 0, 4096),
              oracle.adamw_bits(1 + 2 ** 32, 1, 0, 4096), oracle.adamw_bits(1, 1, 0, 4096, first=1 << 32)):
        assert (a == b).mean() < 0.01
        for k in range(0, 32, 5):  # each bit agrees half the time
            assert abs((((a ^ b) >> k) & 1).mean() - 0.5) < 0.05


def rows_of(rng, rows, vocab):
    x = rng.standard_normal((rows, vocab)) * 3
    x[0, rng.random(vocab) < 0.3] = -np.inf
    x[0, 0] = 1.0
    return x


@pytest.mark.parametrize("vocab,scale", [(1, 1.0), (2, 0.7), (9, 1.0), (40, 1.25)])
def test_logprobs_and_gradient_match_autograd(vocab, scale):
    rng = np.random.default_rng(vocab)
    x = rows_of(rng, 4, vocab)
    y = np.array([0, vocab - 1, -1, vocab // 2])
    gl, ge = rng.standard_normal(4), rng.standard_normal(4)
    lp, lse, h, tlp, ids = oracle.token_logprobs(x, y, scale, min(3, vocab))
    X = torch.tensor(x, requires_grad=True)
    logp = torch.log_softmax(X * scale, 1)
    p = logp.exp()
    H = -(p * torch.where(p > 0, logp, torch.zeros_like(logp))).sum(1)
    keep = torch.tensor(y >= 0)
    want = logp[torch.arange(4), torch.tensor(y).clamp_min(0)]
    assert np.abs((want.detach().numpy() - lp)[y >= 0]).max() < 1e-12
    assert np.abs((H.detach().numpy() - h)[y >= 0]).max() < 1e-12 and lp[2] == 0 and (ids[2] == -1).all()
    loss = (torch.where(keep, want * torch.tensor(gl) + H * torch.tensor(ge), torch.zeros(4))).sum()
    (G,) = torch.autograd.grad(loss, X)
    got = oracle.token_logprobs_grad(x, y, gl, ge, scale)
    assert np.abs(torch.nan_to_num(G).numpy() - got).max() < 1e-12


def test_logprobs_gradient_matches_differences():
    rng = np.random.default_rng(3)
    x, y = rng.standard_normal((3, 7)), np.array([1, 6, 0])
    gl, ge, s = rng.standard_normal(3), rng.standard_normal(3), 0.8
    got = oracle.token_logprobs_grad(x, y, gl, ge, s)

    def loss(x):
        lp, _, h, _, _ = oracle.token_logprobs(x, y, s)
        return (gl * lp + ge * h).sum()

    for r in range(3):
        for j in range(7):
            d = np.zeros_like(x)
            d[r, j] = 1e-5
            assert abs((loss(x + d) - loss(x - d)) / 2e-5 - got[r, j]) < 1e-9


def test_logprobs_ranks_ties_by_index_and_empty_rows():
    x = np.array([[1.0, 2.0, 2.0, -np.inf, 2.0], [-np.inf] * 5, [0.0, -0.0, np.nan, 1.0, -1.0]])
    lp, lse, h, tlp, ids = oracle.token_logprobs(x, np.array([0, 1, 2]), 1.0, 4)
    assert ids.tolist() == [[1, 2, 4, 0], [0, 1, 2, 3], [3, 0, 1, 4]]
    assert lse[1] == -np.inf and lp[1] == -np.inf and h[1] == 0 and np.isnan(lp[2])


@pytest.mark.parametrize("groups,masked", [(1, False), (3, True)])
def test_balance_matches_autograd_and_differences(groups, masked):
    rng = np.random.default_rng(7 + groups)
    T, E, K = 12, 5, 2
    x, ids = rng.standard_normal((T, E)), rng.integers(-1, E, (T, K))
    mask = rng.random(T) < 0.7 if masked else None
    if masked:
        mask[:4] = False  # a group without tokens
    gb, gz = 0.3, 0.7
    r = oracle.balance_loss(x, ids, mask, groups)
    X = torch.tensor(x, requires_grad=True)
    keep = torch.ones(T, dtype=torch.bool) if mask is None else torch.tensor(mask)
    p, lse = torch.softmax(X, 1), torch.logsumexp(X, 1)
    losses = []
    for g in range(groups):
        rows = torch.arange(g * T // groups, (g + 1) * T // groups)
        rows = rows[keep[rows]]
        if len(rows):
            c = torch.tensor(r["counts"][g], dtype=torch.float64)
            losses.append(E * (c / c.sum().clamp_min(1) * p[rows].mean(0)).sum())
    b, z = torch.stack(losses).mean(), lse[keep].square().mean()
    assert abs(b.item() - r["balance"]) < 1e-13 and abs(z.item() - r["z"]) < 1e-13
    (G,) = torch.autograd.grad(gb * b + gz * z, X)
    got = oracle.balance_loss_grad(x, ids, gb, gz, mask, groups)
    assert np.abs(G.numpy() - got).max() < 1e-14

    def loss(x):
        q = oracle.balance_loss(x, ids, mask, groups)
        return gb * q["balance"] + gz * q["z"]

    for t, e in [(0, 0), (5, 4), (11, 2)]:
        d = np.zeros_like(x)
        d[t, e] = 1e-5
        assert abs((loss(x + d) - loss(x - d)) / 2e-5 - got[t, e]) < 1e-9


def test_balance_is_one_when_uniform_and_zero_when_empty():
    T, E = 8, 4
    ids = np.arange(T)[:, None] % E
    assert abs(oracle.balance_loss(np.zeros((T, E)), ids)["balance"] - 1) < 1e-15
    r = oracle.balance_loss(np.zeros((T, E)), ids, np.zeros(T, bool), 2)
    assert r["balance"] == 0 and r["z"] == 0 and not r["counts"].any()
