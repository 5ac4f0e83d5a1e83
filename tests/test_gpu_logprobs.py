"""GPU parity of token_logprobs, its backward and the joint loss call with the
oracle (float64).

Tolerances, before any run.  z = scale x and its exponent's argument carry a
few float32 roundings of numbers up to Z = max |z| of the row's live entries:
8 of them, 2^-21 (1 + Z), bounds lse, logprobs and the alternatives; the
entropy adds as many for the weighted sum: 2^-20 (1 + Z).  A probability is
relatively off by what its exponent is, so a gradient entry is off by
2^-20 (1 + Z) times (|gl| + |ge| (|log p| + |H| + 1)) p, plus 2^-22 of itself,
and half a spacing (2^-8) where it is rounded to bfloat16.  ids are exact."""

import numpy as np
import pytest
import torch

import oracle
from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu
KIND = {"f32": torch.float32, "bf16": torch.bfloat16}


def place(x, kind, pad=0, shift=0):
    """x on the GPU with rows `pad` elements further apart and the first one `shift` elements in."""
    rows, vocab = x.shape
    t = torch.full((rows * (vocab + pad) + shift,), 9e9, dtype=KIND[kind], device="cuda")[shift:]
    t = t.view(rows, vocab + pad)[:, :vocab]
    t.copy_(torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(KIND[kind]))
    return t


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def bounds(x, scale):
    z = np.where(np.isfinite(x), np.abs(x), 0).max(axis=1) * scale
    return 2.0 ** -21 * (1 + z)


def same(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    np.testing.assert_array_equal(np.where(fine, 0, want), np.where(np.isfinite(got), 0, got), err_msg=what)
    bad = np.abs(got[fine] - want[fine]) > np.broadcast_to(tol, want.shape)[fine]
    assert not bad.any(), f"{what}: {bad.sum()} beyond the bound, worst {np.abs(got[fine] - want[fine]).max():.3e}"


def check_score(r, x, y, scale, top):
    lp, lse, h, tlp, ids = oracle.token_logprobs(x, y, scale, top)
    tol = bounds(x, scale)
    same(host(r.logprobs), lp, tol, "logprobs")
    same(host(r.lse), lse, tol, "lse")
    same(host(r.entropy), h, 2 * tol, "entropy")
    if top:
        np.testing.assert_array_equal(r.top_ids.cpu().numpy(), ids)
        same(host(r.top_logprobs), tlp, tol[:, None], "top_logprobs")


def check_grad(G, x, y, gl, ge, scale, kind, live=None):
    """live: the entries whose size counts in the bound, where the rest is a mask (default: x)."""
    want = oracle.token_logprobs_grad(x, y, gl, ge, scale)
    with np.errstate(all="ignore"):
        z = x * scale
        d = z - z.max(axis=1, keepdims=True)
        logp = d - np.log(np.exp(d).sum(axis=1, keepdims=True))
        p = np.nan_to_num(np.exp(logp))
        h = -(p * np.where(p > 0, logp, 0)).sum(axis=1, keepdims=True)
        weight = np.abs(gl)[:, None] + (0 if ge is None else np.abs(ge)[:, None] * (np.abs(np.where(p > 0, logp, 0)) + np.abs(h) + 1))
    tol = scale * weight * p * 2 * bounds(x if live is None else live, scale)[:, None] + 2.0 ** -22 * np.abs(want) + 1e-42
    # an exponent that underflows in float32 gives 0
    tol = tol + scale * weight * 2.0 ** -125
    if kind == "bf16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -9 * 1.01 * np.abs(want) * 2 + 2.0 ** -133
    same(host(G), want, tol, "grad")


def case(rng, rows, vocab, kind, spread=3.0, masked=0.2):
    x = rng.standard_normal((rows, vocab)) * spread
    x[rng.random((rows, vocab)) < masked] = -np.inf
    x[:, 0] = np.where(np.isinf(x[:, 0]), 0.5, x[:, 0])
    x = torch.from_numpy(x.astype(np.float32)).to(KIND[kind]).float().numpy().astype(np.float64)
    y = rng.integers(0, vocab, rows)
    return x, y


def run_all(x, y, kind, scale, top, pad=0, shift=0, entropy=True, in_place=False):
    rng = np.random.default_rng(x.size)
    rows = x.shape[0]
    gl = rng.standard_normal(rows).astype(np.float32).astype(np.float64)
    ge = rng.standard_normal(rows).astype(np.float32).astype(np.float64) if entropy else None
    f = lambda a: None if a is None else torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    X, Y = place(x, kind, pad, shift), torch.from_numpy(y).cuda()
    r = muon.token_logprobs(X, Y, top=top, scale=scale)
    check_score(r, x, y, scale, top)
    L = muon.token_logprobs_loss(X, Y, f(gl), f(ge), top=top, scale=scale)
    check_score(L, x, y, scale, top)
    keep = (y < x.shape[1])
    assert keep.all()
    check_grad(L.grad, x, y, gl, ge, scale, kind)
    G = muon.token_logprobs_backward(X, Y, r.lse, f(gl), entropy=r.entropy if entropy else None, grad_entropy=f(ge),
                                     scale=scale, out=X if in_place else None)
    check_grad(G, x, y, gl, ge, scale, kind)
    if in_place:
        assert G.data_ptr() == X.data_ptr()
        X2 = place(x, kind, pad, shift)
        muon.token_logprobs_loss(X2, Y, f(gl), f(ge), scale=scale, out=X2)
        check_grad(X2, x, y, gl, ge, scale, kind)


SHAPES = [(1, 1), (3, 2), (5, 7), (2, 31), (4, 257), (3, 1000), (2, 4099), (7, 8192), (2, 50257), (1, 200_003)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_scores_and_gradients_over_sizes(rows, vocab, kind):
    rng = np.random.default_rng(rows * 7 + vocab)
    x, y = case(rng, rows, vocab, kind)
    run_all(x, y, kind, 1.0, min(5, vocab))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(1, 0), (8, 0), (0, 1), (3, 5), (24, 8)])
def test_row_pitch_and_offset(kind, pad, shift):
    rng = np.random.default_rng(pad + 10 * shift)
    for vocab in (5, 263, 1024, 3001):
        x, y = case(rng, 6, vocab, kind)
        run_all(x, y, kind, 0.8, min(3, vocab), pad, shift, in_place=True)


@pytest.mark.parametrize("top", [0, 1, 2, 17, 32])
@pytest.mark.parametrize("scale", [0.25, 1.0, 3.0])
def test_alternatives_and_temperature(top, scale):
    rng = np.random.default_rng(top)
    x, y = case(rng, 4, 700, "bf16")
    run_all(x, y, "bf16", scale, top, entropy=top % 2 == 0)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 31, 64, 65, 130, 257, 301, 513, 600, 1025])
def test_many_short_rows(vocab, kind):
    """Rows enough for every warp: a few lanes then take a row."""
    rng = np.random.default_rng(vocab)
    x, y = case(rng, 5003, vocab, kind)
    y[::11] = -1
    x[y < 0] = 0.0
    x[5::50] = -np.inf
    live = (y >= 0) & np.isfinite(x).any(axis=1)
    gl, ge = (rng.standard_normal(len(y)).astype(np.float32) for _ in range(2))
    GL, GE, Y, keep = torch.from_numpy(gl).cuda(), torch.from_numpy(ge).cuda(), torch.from_numpy(y).cuda(), torch.from_numpy(live).cuda()
    for pad, shift in ((0, 0), (1, 2)):
        X = place(x, kind, pad, shift)
        r = muon.token_logprobs(X, Y)
        B = muon.token_logprobs_backward(X, Y, r.lse, GL, r.entropy, GE)
        q = muon.token_logprobs_loss(X, Y, GL, GE, out=X)
        empty = (y >= 0) & ~live
        for o in (r, q):
            check_score(muon.TokenLogprobs(o.logprobs[keep], o.lse[keep], o.entropy[keep], None, None), x[live], y[live], 1.0, 0)
            assert (host(o.lse)[empty] == -np.inf).all() and not host(o.entropy)[empty].any() and not host(o.lse)[y < 0].any()
        for G in (B, q.grad):
            check_grad(G[keep], x[live], y[live], gl[live], ge[live], 1.0, kind)
            assert not host(G)[~live].any()


@pytest.mark.parametrize("rows", [1, 2, 19, 151, 153, 700, 1300])
def test_rows_from_one_to_many(rows):
    """From one row that many blocks share to many rows a block each."""
    rng = np.random.default_rng(rows)
    x, y = case(rng, rows, 5003 if rows < 200 else 811, "bf16")
    run_all(x, y, "bf16", 1.0, 4)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["constant", "rising", "falling", "few", "one_hot", "zeros"])
def test_alternatives_with_ties_and_orders(what, kind):
    """Ranks by value, then index: equal values, rising rows (every entry a new largest), few distinct values."""
    vocab = 9001
    j = np.arange(vocab, dtype=np.float64)
    rng = np.random.default_rng(1)
    row = {"constant": np.full(vocab, 1.5), "rising": j / 300, "falling": -j / 300, "few": rng.integers(0, 3, vocab) * 1.0,
           "one_hot": np.where(j == 5000, 30.0, 0.0), "zeros": np.where(rng.random(vocab) < 0.5, 0.0, -0.0)}[what]
    x = torch.from_numpy(np.stack([row, np.roll(row, 17)]).astype(np.float32)).to(KIND[kind]).float().numpy().astype(np.float64)
    run_all(x, np.array([3, 8999]), kind, 1.0, 32)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(9, 4500), (300, 12_346), (5, 60_000), (170, 60_001), (9, 130_001)])
def test_gradients_that_fall_differently_from_the_logits(rows, vocab, kind):
    """Pitches and offsets of logits and gradient that differ, so that every distance to the vectors' boundaries occurs."""
    rng = np.random.default_rng(vocab)
    x, y = case(rng, rows, vocab, kind)
    y[::7] = -1
    x[y < 0] = 0.0
    for pad, shift, out_pad, out_shift in ((1, 0, 0, 3), (3, 5, 2, 0)):
        X, Y = place(x, kind, pad, shift), torch.from_numpy(y).cuda()
        gl, ge = (rng.standard_normal(rows).astype(np.float32) for _ in range(2))
        GL, GE = torch.from_numpy(gl).cuda(), torch.from_numpy(ge).cuda()
        outs = [place(np.full((rows, vocab), 7.0), kind, out_pad, out_shift) for _ in range(2)]
        r = muon.token_logprobs_loss(X, Y, GL, GE, out=outs[0])
        muon.token_logprobs_backward(X, Y, r.lse, GL, r.entropy, GE, out=outs[1])
        live = y >= 0
        for G in outs:
            check_grad(G[torch.from_numpy(live).cuda()], x[live], y[live], gl[live], ge[live], 1.0, kind)
            assert not host(G)[~live].any()
            if out_pad:  # the gap between rows is left as it was
                whole = torch.as_strided(G, (rows - 1, out_pad), (vocab + out_pad, 1), G.storage_offset() + vocab)
                assert (whole == torch.tensor(9e9, device="cuda").to(KIND[kind])).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(3, 50_257), (400, 12_345), (700, 70_001), (800, 2047), (800, 1030), (800, 520), (800, 256), (800, 137)])
def test_alternatives_among_many_equal_entries(rows, vocab, kind):
    """Rows whose best entries are fewer than the alternatives asked for, all others equal (a mask, or a floor):
    the first of these follow by index; and rows of three values, with and without entries below the equal ones."""
    rng = np.random.default_rng(vocab)
    fill = [-np.inf, float(torch.finfo(KIND[kind]).min), -9984.0, 0.0]
    x = np.stack([np.full(vocab, fill[i % 4]) for i in range(rows)])
    for i in range(rows):
        few = rng.integers(0, vocab, (i // 4) % 24)  # and of these some twice
        x[i, few] = rng.integers(1, 5, len(few))
        low = rng.integers(0, vocab, vocab // 2)
        if i % 8 >= 4:
            x[i, low] = np.where(x[i, low] == fill[i % 4], -np.inf, x[i, low])
        if i % 16 == 15:
            x[i, : vocab // 2] = rng.integers(0, 3, vocab // 2)
    y = rng.integers(0, vocab, rows)
    X, Y = place(x, kind), torch.from_numpy(y).cuda()
    for top in (1, 20):
        order = np.argsort(-x, axis=1, kind="stable")[:, :top]
        gl = torch.ones(rows, device="cuda")
        for r in (muon.token_logprobs(X, Y, top=top), muon.token_logprobs_loss(X, Y, gl, top=top)):
            np.testing.assert_array_equal(r.top_ids.cpu().numpy(), order)
    few = np.array([i for i in range(0, rows, 37) if i % 4 != 1])
    check_score(muon.token_logprobs(X[few], Y[few], top=5), x[few], y[few], 1.0, 5)


def test_rows_left_out_are_not_read():
    """Targets below 0: zeros and -1 ids, gradient zero, even where the logits are NaN."""
    x = np.random.default_rng(0).standard_normal((6, 333))
    x = x.astype(np.float32).astype(np.float64)
    y = np.array([4, -100, 0, -1, 332, -2 ** 40])
    x[[1, 3, 5]] = np.nan
    X, Y = place(x, "f32"), torch.from_numpy(y).cuda()
    gl = np.ones(6)
    clean = np.where(y[:, None] < 0, 0.0, x)
    for r in (muon.token_logprobs(X, Y, top=2),
              muon.token_logprobs_loss(X, Y, torch.ones(6, device="cuda"), torch.ones(6, device="cuda"), top=2)):
        check_score(r, clean, y, 1.0, 2)
    check_grad(r.grad, clean, y, gl, gl, 1.0, "f32")
    G = muon.token_logprobs_backward(X, Y, r.lse, torch.ones(6, device="cuda"))
    check_grad(G, clean, y, gl, None, 1.0, "f32")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_masks_that_leave_little_or_nothing(kind):
    """All -inf; one live entry; the type's lowest value as a mask, in part and in whole; a masked target."""
    low = torch.finfo(KIND[kind]).min
    vocab = 601
    x = np.random.default_rng(5).standard_normal((8, vocab))
    x = torch.from_numpy(x.astype(np.float32)).to(KIND[kind]).float().numpy().astype(np.float64)
    x[0] = -np.inf
    x[1] = -np.inf
    x[1, 77] = -3.0
    x[2, 10:] = low
    x[3] = low
    x[4, 5] = -np.inf
    x[5, :300] = -np.inf
    x[6] = low
    x[6, 600] = -np.inf
    y = np.array([3, 77, 4, 100, 5, 400, 7, 1])
    for z in (x, x[::-1].copy()):
        yy = y if z is x else y[::-1].copy()
        with np.errstate(over="ignore", invalid="ignore"):
            X, Y = place(z, kind), torch.from_numpy(yy).cuda()
        r = muon.token_logprobs(X, Y, top=4)
        lp, lse, h, tlp, ids = oracle.token_logprobs(z, yy, 1.0, 4)
        # lse of a row of the lowest value is that value; its parts are of order 1, lost beside it in lse alone
        whole = (z <= -1e30).all(axis=1)
        tol = np.where(whole, 2.0 ** -21 * 10, 2.0 ** -21 * (1 + np.where(np.isfinite(z) & (z > -1e30), np.abs(z), 0).max(axis=1)))
        same(host(r.entropy), h, 2 * tol, "entropy")
        same(host(r.lse)[~whole], lse[~whole], tol[~whole], "lse")
        same(host(r.lse)[whole], lse[whole], 2.0 ** -22 * 3.4e38, "lse")
        np.testing.assert_array_equal(r.top_ids.cpu().numpy(), ids)
        same(host(r.logprobs), lp, np.where(np.abs(np.nan_to_num(lp, neginf=0)) > 1e30, 1e32, tol), "logprobs")
        G = muon.token_logprobs_loss(X, Y, torch.ones(8, device="cuda"), torch.ones(8, device="cuda")).grad
        B = muon.token_logprobs_backward(X, Y, r.lse, torch.ones(8, device="cuda"), entropy=r.entropy,
                                         grad_entropy=torch.ones(8, device="cuda"))
        for g in (G, B):
            with np.errstate(invalid="ignore"):
                live = np.where(whole[:, None], z - z.max(axis=1, keepdims=True), np.where(z > -1e30, z, -np.inf))
            check_grad(g, z, yy, np.ones(8), np.ones(8), 1.0, kind, live=live)


@pytest.mark.parametrize("rows,vocab", [(1, 40_000), (2, 300_001), (160, 60_000), (1, 1_000_003)])
def test_long_rows_masked_with_the_lowest_value(rows, vocab):
    """Whole rows and whole stretches of a row at the lowest value, over one block, several and rows read twice."""
    low = torch.finfo(torch.bfloat16).min
    X = torch.randn((rows, vocab), device="cuda").bfloat16()
    X[:, vocab // 3:] = low
    X[0] = low
    X[0, 0] = -float("inf")
    Y = torch.randint(0, vocab // 3, (rows,), device="cuda")
    one = torch.ones(rows, device="cuda")
    r = muon.token_logprobs_loss(X, Y, one, one, top=2)
    B = muon.token_logprobs_backward(X, Y, r.lse, one, entropy=r.entropy, grad_entropy=one)
    for k in sorted({0, rows - 1}):
        x, y = host(X[k:k + 1]), Y[k:k + 1].cpu().numpy()
        lp, lse, h, tlp, ids = oracle.token_logprobs(x, y, 1.0, 2)
        assert abs(float(r.entropy[k]) - h[0]) < 2.0 ** -20 * 20 and ids[0].tolist() == r.top_ids[k].tolist()
        if lp[0] > -1e30:  # a random target may be the one masked with -inf
            assert abs(float(r.logprobs[k]) - lp[0]) < 2.0 ** -21 * 20
        for g in (r.grad, B):
            live = np.where(x > -1e30, x, 0)
            check_grad(g[k:k + 1], x, y, np.ones(1), np.ones(1), 1.0, "bf16", live=live)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(2, 120_000), (3, 500_009), (1, 1_200_000)])
def test_long_rows(rows, vocab, kind):
    """Rows of several blocks' shared memory, and longer than a cluster holds."""
    x, y = case(np.random.default_rng(vocab), rows, vocab, kind, masked=0.01)
    run_all(x, y, kind, 1.0, 20, in_place=True)


def test_target_past_the_vocabulary_and_non_finite_rows():
    x = np.random.default_rng(2).standard_normal((5, 100)).astype(np.float32).astype(np.float64)
    x[1, 50], x[2, 60] = np.nan, np.inf
    y = np.array([100, 3, 4, 2 ** 40, 7])
    X, Y = place(x, "f32"), torch.from_numpy(y).cuda()
    one = torch.ones(5, device="cuda")
    r = muon.token_logprobs_loss(X, Y, one, top=3)
    assert torch.isnan(r.logprobs).tolist() == [True, True, True, True, False]
    assert torch.isnan(r.lse).tolist() == [False, True, True, False, False]
    assert torch.isnan(r.entropy).tolist() == [False, True, True, False, False]
    np.testing.assert_array_equal(r.top_ids.cpu().numpy()[[0, 1, 3, 4]], oracle.token_logprobs(x, y, 1.0, 3)[4][[0, 1, 3, 4]])
    assert int(r.top_ids[2, 0]) == 60
    for g in (r.grad, muon.token_logprobs_backward(X, Y, r.lse, one)):
        assert torch.isnan(g).all(dim=1).tolist() == [True, True, True, True, False]


def test_offsets_past_32_bits():
    """Three rows 2^30 + 8 elements apart, and 70,000 rows of a wide pitch: element offsets pass 2^31."""
    pitch, vocab = (1 << 30) + 8, 1003
    flat = torch.zeros(2 * pitch + vocab + 16, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(8)
    x, y = case(rng, 3, vocab, "bf16")
    X = torch.as_strided(flat, (3, vocab), (pitch, 1), 1)
    X.copy_(torch.from_numpy(x.astype(np.float32)).cuda())
    Y = torch.from_numpy(y).cuda()
    gl = torch.ones(3, device="cuda")
    r = muon.token_logprobs_loss(X, Y, gl, top=3, out=X)
    check_score(r, x, y, 1.0, 3)
    check_grad(X, x, y, np.ones(3), None, 1.0, "bf16")
    del flat, X, r
    rows, pitch = 70_000, 32_768
    flat = torch.zeros(rows * pitch, dtype=torch.bfloat16, device="cuda")
    X = flat.view(rows, pitch)[:, :50]
    xs = torch.randn((rows, 50), device="cuda").bfloat16()
    X.copy_(xs)
    Y = torch.randint(0, 50, (rows,), device="cuda")
    r = muon.token_logprobs(X, Y, top=1)
    want = torch.log_softmax(xs.double(), 1).gather(1, Y[:, None])[:, 0]
    assert float((r.logprobs - want).abs().max()) < 2.0 ** -21 * 7
    G = muon.token_logprobs_backward(X, Y, r.lse, torch.ones(rows, device="cuda"), out=X)
    p = torch.softmax(xs.double(), 1)
    p.neg_().scatter_add_(1, Y[:, None], torch.ones_like(p[:, :1]))
    assert float((G.double() - p).abs().max()) < 2.0 ** -8


def test_gradient_matches_differences_of_the_score():
    """Central differences of the GPU's own float32 results, step 2^-6: curvature 2^-12, rounding 2^-19 / 2^-6."""
    rng = np.random.default_rng(11)
    vocab = 6
    x = rng.standard_normal((1, vocab)).astype(np.float32).astype(np.float64)
    y = np.array([2])
    gl, ge = 0.7, -0.4
    probes = np.repeat(x, 2 * vocab, axis=0)
    for j in range(vocab):
        probes[2 * j, j] += 2.0 ** -6
        probes[2 * j + 1, j] -= 2.0 ** -6
    r = muon.token_logprobs(place(probes, "f32"), torch.full((2 * vocab,), 2, device="cuda"))
    loss = gl * host(r.logprobs) + ge * host(r.entropy)
    slope = (loss[0::2] - loss[1::2]) / 2.0 ** -5
    g = muon.token_logprobs_loss(place(x, "f32"), torch.from_numpy(y).cuda(), torch.tensor([gl], device="cuda"),
                                 torch.tensor([ge], device="cuda")).grad
    assert np.abs(host(g)[0] - slope).max() < 2.0 ** -11


def test_other_stream_and_equal_calls():
    x, y = case(np.random.default_rng(4), 40, 12_345, "bf16")
    X, Y = place(x, "bf16"), torch.from_numpy(y).cuda()
    gl = torch.randn(40, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = muon.token_logprobs_loss(X, Y, gl, gl, top=9)
    torch.cuda.current_stream().wait_stream(s)
    b = muon.token_logprobs_loss(X, Y, gl, gl, top=9)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_no_rows():
    X, Y = torch.zeros((0, 50), device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    r = muon.token_logprobs(X, Y, top=2)
    assert r.logprobs.shape == (0,) and r.top_ids.shape == (0, 2)


def test_refusals_on_device():
    X, Y = torch.zeros((4, 8), device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad in (dict(top=9), dict(top=33), dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(muon.MuonError):
            muon.token_logprobs(X, Y, **bad)
    with pytest.raises(TypeError):
        muon.token_logprobs(X.half(), Y)
    with pytest.raises(ValueError):
        muon.token_logprobs(X, Y.int())
    with pytest.raises(ValueError):
        muon.token_logprobs(X, Y[:3])
    with pytest.raises(ValueError):
        muon.token_logprobs(X, Y.cpu())
    with pytest.raises(muon.MuonError) as e:  # an output shifted against its input
        flat = torch.zeros(40, device="cuda")
        muon.token_logprobs_backward(flat[:32].view(4, 8), Y, torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda"),
                                     out=flat[4:36].view(4, 8))
    assert e.value.status == muon.MUON_ERR_ALIASING
