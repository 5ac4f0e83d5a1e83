"""token_logprobs, its backward and the joint loss call where scaled logits are
large: low and very high temperatures, whole rows at mask constants between
the ordinary ones and the type's lowest value, dominant entries.

Tolerances, before any run.  An exponent is a difference with a row's (near)
largest entry, so errors do not grow with |z| but with |z - max z|.  With
d = z - max z of an entry and V entries, in units of 2^-24: the difference,
its product with the scale and c2 = scale log2(e) are 4 |d| off, the power 4
more; S averages them with the entries' shares (|d| to log V there), and its
logarithm adds log V.  Hence 2^-21 (1 + |log p| + log V) for a log
probability, 2^-22 |lse| more for lse (its own rounding, and the product with the
largest logit), and for the entropy twice the first with the share-weighted
square of log p, as p log p moves by |log p| times what log p does:
2^-20 (1 + log V + sum p (log p)^2 + (log V)^2).  A probability is relatively
off by 2^-20 (1 + |log p| + log V).  The backward pass takes log S from lse:
2^-22 |lse| more, at most 2^-12: 2^-24 of |lse| up to 4096, beyond which it
takes log S again.  Gradients
in bfloat16, of 8 significant bits, add half a spacing: 2^-8."""

import numpy as np
import pytest
import torch

import oracle
from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu
KIND = {"f32": torch.float32, "bf16": torch.bfloat16}


def rounded(x, kind):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(KIND[kind]).double().numpy()


def put(x, kind, pad=0):
    rows, vocab = x.shape
    t = torch.zeros((rows, vocab + pad), dtype=KIND[kind], device="cuda")[:, :vocab]
    return t.copy_(torch.from_numpy(x.astype(np.float32)).cuda().to(KIND[kind]))


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def reference(x, y, gl, ge, scale, top):
    """What the oracle gives, with the tolerances."""
    vocab = x.shape[1]
    lp, lse, h, tlp, ids = oracle.token_logprobs(x, y, scale, top)
    with np.errstate(all="ignore"):
        d = x * scale - (x * scale).max(axis=1, keepdims=True)
        logp = d - np.log(np.exp(d).sum(axis=1, keepdims=True))
    p = np.exp(logp)
    live = np.where(p > 0, logp, 0)
    lv = np.log(vocab)
    t_lp = lambda v: 2.0 ** -21 * (1 + np.abs(v) + lv)  # noqa: E731
    t_h = 2.0 ** -20 * (1 + lv + (p * live ** 2).sum(axis=1) + lv ** 2)
    weight = np.abs(gl)[:, None] + np.abs(ge)[:, None] * (np.abs(live) + h[:, None] + 1)
    want = oracle.token_logprobs_grad(x, y, gl, ge, scale)
    rel = 2.0 ** -20 * (1 + np.abs(live) + lv)
    return (lp, lse, h, tlp, ids), t_lp, t_h, want, scale * weight * p, rel


def close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    np.testing.assert_array_equal(got[~fine], want[~fine], err_msg=what)
    off = np.abs(got - np.where(fine, want, 0))[fine] / np.broadcast_to(tol, want.shape)[fine]
    off = np.where(np.isfinite(off), off, np.inf)
    assert not (off > 1).any(), f"{what}: {(off > 1).sum()} beyond the bound, worst {off.max():.3g} times it"


def check_scores(r, want, t_lp, t_h, top, what):
    lp, lse, h, tlp, ids = want
    close(host(r.logprobs), lp, t_lp(np.where(np.isfinite(lp), lp, 0)), what + " logprobs")
    assert (host(r.logprobs) <= 0).all(), what
    inner = np.where(np.isfinite(lse), lse, 0)
    close(host(r.lse), lse, t_lp(0) + 2.0 ** -22 * np.abs(inner), what + " lse")
    close(host(r.entropy), h, t_h, what + " entropy")
    if top:
        np.testing.assert_array_equal(r.top_ids.cpu().numpy(), ids, err_msg=what)
        close(host(r.top_logprobs), tlp, t_lp(np.where(np.isfinite(tlp), tlp, 0)), what + " top_logprobs")


def check_grad(G, want, size, rel, scale, kind, what):
    tol = size * rel + 2.0 ** -22 * np.abs(want) + scale * 2.0 ** -115 + 1e-42  # exponents that underflow give 0
    if kind == "bf16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    close(host(G), want, tol, what)


class Case:
    def __init__(self, x, y, kind, scale, top=3, pad=0):
        rng = np.random.default_rng(x.size)
        self.kind, self.scale, self.top = kind, float(np.float32(scale)), top
        gl, ge = (rng.standard_normal(x.shape[0]).astype(np.float32).astype(np.float64) for _ in range(2))
        self.GL, self.GE = (torch.from_numpy(a.astype(np.float32)).cuda() for a in (gl, ge))
        self.X, self.Y = put(x, kind, pad), torch.from_numpy(y).cuda()
        self.want, self.t_lp, self.t_h, self.grad, self.size, self.rel = reference(x, y, gl, ge, self.scale, top)
        lse = np.where(np.isfinite(self.want[1]), self.want[1], 0)
        self.saved = 2.0 ** -22 * np.minimum(np.abs(lse), 1024)[:, None]
        # a longer row is scored, and then takes the backward pass
        self.held = x.shape[1] * (4 if kind == "f32" else 2) + 32 <= 208 * 1024

    def scores_and_loss(self):
        for k in (self.top, 0):
            r = muon.token_logprobs(self.X, self.Y, top=k, scale=self.scale)
            check_scores(r, self.want, self.t_lp, self.t_h, k, f"score, top {k}:")
            q = muon.token_logprobs_loss(self.X, self.Y, self.GL, self.GE, top=k, scale=self.scale)
            check_scores(q, self.want, self.t_lp, self.t_h, k, f"loss, top {k}:")
            if self.held:
                check_grad(q.grad, self.grad, self.size, self.rel, self.scale, self.kind, f"loss gradient, top {k}")


#: rows and vocabularies: several rows a warp, one, one block, several, rows kept over two blocks, rows read twice
SHAPES = [(6000, 150), (40, 301), (24, 2999), (24, 9001), (20, 50_304), (160, 40_001), (160, 70_001), (16, 130_001)]
CONSTANTS = (-1e4, -65504.0, -1e6, -1e9, -1e10, -1e12, -1e20, 1e4, 1e6, 1e9, 1e12)


def rows_of(rng, rows, vocab, kind):
    """Rows in turn: ordinary; a constant throughout; the constant but for -inf entries; the constant plus noise; and one
    entry (or two equal ones) that stands above such a row.  The targets are an entry of the largest, or any."""
    x, y = np.empty((rows, vocab)), rng.integers(0, vocab, rows)
    for i in range(rows):
        c, what = CONSTANTS[(i // 5) % len(CONSTANTS)], i % 5
        x[i] = rng.standard_normal(vocab) * 3 if what in (0, 3) else 0.0
        x[i] += 0.0 if what == 0 else c
        if what == 2:
            x[i, rng.random(vocab) < 0.3] = -np.inf
            x[i, rng.integers(0, vocab)] = c
        if what == 4:
            x[i, rng.integers(0, vocab, 1 + (i // 5) % 2)] = c + abs(c) / 16
    x = rounded(x, kind)
    best = x.argmax(axis=1)
    return x, np.where(rng.random(rows) < 0.5, best, np.where(np.isfinite(x[np.arange(rows), y]), y, best))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_rows_at_large_constants(rows, vocab, kind):
    x, y = rows_of(np.random.default_rng(vocab), rows, vocab, kind)
    Case(x, y, kind, 1.0).scores_and_loss()


def hot_rows(rows, vocab, kind):
    """Ordinary logits with one to three equal ones on top, masked entries, every tenth row uniform."""
    rng = np.random.default_rng(vocab)
    x = rng.standard_normal((rows, vocab)) * 3
    x[rng.random(x.shape) < 0.2] = -np.inf
    x[::10] = 47.25
    for i in range(rows):
        x[i, rng.integers(0, vocab, 1 + i % 3)] = 50.0 - 0.25 * (i % 16)
    x = rounded(x, kind)
    y = rng.integers(0, vocab, rows)
    best = x.argmax(axis=1)
    return x, np.where((rng.random(rows) < 0.5) | ~np.isfinite(x[np.arange(rows), y]), best, y)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 100.0, 1e3, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("rows,vocab", [(6000, 150), (40, 301), (24, 9001), (20, 50_304), (160, 70_001), (16, 130_001)])
def test_low_and_high_temperatures(rows, vocab, scale, kind):
    Case(*hot_rows(rows, vocab, kind), kind, scale, pad=3).scores_and_loss()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_a_row_does_not_depend_on_its_neighbours(kind):
    """Short rows that share a warp with rows at a constant: the bits of the rows alone."""
    rng = np.random.default_rng(3)
    x = rounded(rng.standard_normal((8192, 130)), kind)
    y = torch.from_numpy(rng.integers(0, 130, 8192)).cuda()
    w = x.copy()
    w[1::2] = -1e9
    gl = torch.ones(8192, device="cuda")
    a, b = (muon.token_logprobs_loss(put(z, kind), y, gl, gl) for z in (x, rounded(w, kind)))
    for p, q in zip((*a[:3], a.grad), (*b[:3], b.grad)):
        assert torch.equal(p[::2], q[::2])


def backward(c, loss):
    if loss and not c.held:
        for k in (c.top, 0):
            q = muon.token_logprobs_loss(c.X, c.Y, c.GL, c.GE, top=k, scale=c.scale)
            check_grad(q.grad, c.grad, c.size, c.rel + c.saved, c.scale, c.kind, f"loss gradient, top {k}")
    r = muon.token_logprobs(c.X, c.Y, scale=c.scale)
    for out in (None, c.X):
        G = muon.token_logprobs_backward(c.X, c.Y, r.lse, c.GL, entropy=r.entropy, grad_entropy=c.GE, scale=c.scale, out=out)
        check_grad(G, c.grad, c.size, c.rel + c.saved, c.scale, c.kind, "backward" + (" in place" if out is not None else ""))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_backward_of_rows_at_large_constants(rows, vocab, kind):
    x, y = rows_of(np.random.default_rng(vocab), rows, vocab, kind)
    backward(Case(x, y, kind, 1.0), True)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 100.0, 1e4, 1e6])
@pytest.mark.parametrize("rows,vocab", [(6000, 150), (40, 301), (24, 9001), (16, 130_001)])
def test_backward_at_low_and_high_temperatures(rows, vocab, scale, kind):
    backward(Case(*hot_rows(rows, vocab, kind), kind, scale, pad=3), True)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [130, 9001])
def test_backward_where_lse_overflows(vocab, kind):
    """The lowest value at scale 4: lse is -inf, as for an empty row, which has no gradient; the row is uniform."""
    x = np.full((4, vocab), float(torch.finfo(KIND[kind]).min))
    x[2] = -np.inf
    X, y, one = put(x, kind), torch.tensor([1, 2, 3, -1], device="cuda"), torch.ones(4, device="cuda")
    r = muon.token_logprobs(X, y, scale=4.0)
    assert r.lse.tolist() == [-np.inf] * 3 + [0.0]
    want = -4.0 / vocab * np.ones((4, vocab))
    want[[0, 1], [1, 2]] += 4.0
    want[2:] = 0
    for G in (muon.token_logprobs_backward(X, y, r.lse, one, scale=4.0), muon.token_logprobs_loss(X, y, one, scale=4.0).grad):
        # a probability 2^-20 (1 + 2 log V) off, half a spacing of bfloat16
        assert (np.abs(host(G) - want) <= (2.0 ** -15 + (2.0 ** -8 if kind == "bf16" else 0)) * np.abs(want)).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [25_000, 50_304, 130_000])
def test_entropy_of_long_rows_with_a_peak(vocab, kind):
    """Few large shares beside very many small ones, which a long chain of additions would lose: over all rows the root
    mean square of the relative error.  A chain of n additions errs by about sqrt(n) 2^-25 where one sum holds
    everything; parts of up to 52 entries and 64 parts leave 2.6e-7, the powers and the logarithm 2^-23: 2^-21 in all."""
    gen = torch.Generator("cuda").manual_seed(vocab)
    for rows in (20, 400):  # several blocks a row, one block a row
        common = -torch.log(torch.randperm(vocab, generator=gen, device="cuda").float() + 2.0)
        x = torch.randn((rows, vocab), generator=gen, device="cuda").mul_(2.0).add_(common).to(KIND[kind])
        y = torch.zeros(rows, dtype=torch.int64, device="cuda")
        logp = torch.log_softmax(x.double() * 1.25, 1)
        want = -(logp.exp() * logp).sum(1)
        one = torch.ones(rows, device="cuda")
        for r in (muon.token_logprobs(x, y, scale=1.25), muon.token_logprobs(x, y, top=3, scale=1.25),
                  muon.token_logprobs_loss(x, y, one, scale=1.25)):
            assert float(((r.entropy.double() - want) / want).square().mean().sqrt()) <= 2.0 ** -21
