"""Rows that are left out between rows that several blocks share: what the
blocks tell one another for one row must not reach another."""

import numpy as np
import pytest
import torch

from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("every", [2, 3, 7])
@pytest.mark.parametrize("top", [0, 2])
@pytest.mark.parametrize("vocab,kind", [(30_001, torch.float32), (40_960, torch.float32), (60_001, torch.bfloat16), (80_000, torch.bfloat16)])
def test_kept_rows_have_the_bits_of_a_batch_without_gaps(vocab, kind, top, every):
    """Rows of two blocks each, several to a pair of blocks; kept and left out in turn, in runs, and at random."""
    rows = 1200
    gen = torch.Generator("cuda").manual_seed(vocab + every)
    x = torch.randn((rows, vocab), generator=gen, device="cuda").mul_(2).to(kind)
    x += torch.arange(rows, device="cuda").to(kind)[:, None] % 13  # sums of a row taken for another's would differ
    y = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    gl, ge = (torch.randn(rows, generator=gen, device="cuda") for _ in range(2))
    want = muon.token_logprobs_loss(x, y, gl, ge, top=top)
    i = np.arange(rows)
    for out in (i % every == 1, i // 152 % every == 1, np.random.default_rng(every).random(rows) < 0.5):
        left = torch.from_numpy(out).cuda()
        got = muon.token_logprobs_loss(x, torch.where(left, -1, y), gl, ge, top=top)
        for a, b in zip(got, want):
            if a is not None:
                assert torch.equal(a[~left], b[~left])
        assert not got.grad[left].any() and not got.lse[left].any()
        del got


@pytest.mark.parametrize("vocab,kind", [(8190, torch.bfloat16), (12_285, torch.bfloat16), (16_382, torch.bfloat16), (4095, torch.float32),
                                        (32_765, torch.bfloat16), (65_531, torch.bfloat16), (65_534, torch.bfloat16), (28_669, torch.float32)])
def test_rows_whose_number_of_vectors_changes_from_one_to_the_next(vocab, kind):
    """Odd pitches, vocabularies next to whole groups of copies: rows of one block after another, one vector more or less each."""
    rows = 2600
    gen = torch.Generator("cuda").manual_seed(vocab)
    y = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    gl = torch.ones(rows, device="cuda")
    for pad in (0, 1, 2):
        x = torch.empty((rows, vocab + pad), dtype=kind, device="cuda")[:, :vocab]
        x.copy_(torch.randn((rows, vocab), generator=gen, device="cuda").add_(torch.arange(rows, device="cuda")[:, None] % 7))
        r = muon.token_logprobs_loss(x, y, gl, top=pad, out=torch.empty_strided(x.shape, x.stride(), dtype=kind, device="cuda"))
        for k in range(0, rows, 650):  # in float64, a part at a time
            p = torch.softmax(x[k:k + 650].double(), 1)
            p.neg_()
            p[torch.arange(len(p), device="cuda"), y[k:k + 650]] += 1
            # a probability 2^-20 (1 + 2 log V) off, float32 rounding or half a spacing of bfloat16 (8 significant bits)
            tol = p.abs().mul_(2.0 ** -15 + (2.0 ** -8 if kind == torch.bfloat16 else 0)).add_(2.0 ** -40)
            assert bool(((r.grad[k:k + 650].double() - p).abs() <= tol).all())
