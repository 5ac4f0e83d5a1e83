"""The operators together: the small mixture-of-experts training of
examples/moe_step.py, recording in a CUDA graph, and the debug build (device-
side range checks), whose results equal the release library's bit for bit."""

import ctypes
import importlib.util
import os

import pytest
import torch

from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("moe_step", os.path.join(ROOT, "examples", "moe_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_learns_and_balances():
    """60 steps: before its first update the model's loss is about log(512) =
    6.24, at the end at most half of that (10 % of the targets are noise:
    they alone cost 0.95), and the balance loss of one eighth of the tokens
    for each expert is 1."""
    history = example().train(60)
    first, last = float(history[0][0]), [float(h[0]) for h in history[-3:]]
    assert first > 5.5 and max(last) < 3.1, (first, last)
    assert float(history[-1][2]) < 2.0
    assert all(int(h[3].sum()) == 2048 for h in history)


def operators(seed):
    """Every operator once, over vector, strided, tiled, clustered and held layouts; all outputs."""
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    out = []
    for bits in (32, 8):
        for odd in (0, 1):
            P = [r(n + odd)[odd:] for n in (5, 256, 1000, 9000)] + [r(3001 + odd).bfloat16()[odd:]]
            G = [torch.randn(p.shape, generator=g, device="cuda").bfloat16() for p in P]
            S = [muon.adamw_state(p, bits) for p in P]
            for step in (1, 2):
                muon.adamw_step(P, G, S, step, cautious=bool(odd), seed=4)
            out += [*P, *(t.view(torch.uint8) if t.element_size() == 1 else t for s in S for t in s)]
    for rows, vocab, kind in ((3, 50_257, torch.bfloat16), (400, 12_345, torch.float32), (70, 777, torch.bfloat16),
                              (1, 300_001, torch.float32), (9, 5, torch.float32), (2, 70_000, torch.float32)):
        x, y = r(rows, vocab).to(kind), torch.randint(-1, vocab, (rows,), generator=g, device="cuda")
        a = muon.token_logprobs(x, y, top=min(5, vocab))
        b = muon.token_logprobs_loss(x, y, r(rows), r(rows), top=1)
        out += [*a[:5], *b, muon.token_logprobs_backward(x, y, a.lse, r(rows))]
    for tokens, experts, kind in ((1000, 64, torch.bfloat16), (1000, 37, torch.bfloat16), (64, 300, torch.float32)):
        x, ids = r(tokens, experts).to(kind), torch.randint(-1, experts, (tokens, 3), generator=g, device="cuda")
        mask = torch.rand(tokens, generator=g, device="cuda") < 0.8
        b = muon.balance_loss(x, ids, mask=mask, groups=4)
        out += [*b, muon.balance_loss_backward(x, b, r(1), r(1), mask=mask)]
    torch.cuda.synchronize()
    return out


def test_debug_build_passes_its_checks_and_matches_release(monkeypatch):
    want = operators(3)
    D, n = muon.load(muon.DEBUG_LIB_PATH), ctypes.c_longlong(-1)
    assert D.muon_debug_check_failures(n) == 0  # a debug build; clears the counters
    monkeypatch.setattr(muon, "_lib", D)
    got = operators(3)
    assert D.muon_debug_check_failures(n) == 0 and n.value == 0
    assert len(got) == len(want)
    for a, b in zip(got, want):
        a, b = a.contiguous(), b.contiguous()
        assert torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))


def test_recorded_in_a_graph():
    """The losses and the AdamW step (its step number as recorded) replayed from a CUDA graph."""
    x, y = torch.randn((64, 5000), device="cuda").bfloat16(), torch.randint(0, 5000, (64,), device="cuda")
    s, ids = torch.randn((256, 16), device="cuda"), torch.randint(0, 16, (256, 2), device="cuda")
    one, gl = torch.ones(1, device="cuda"), torch.full((64,), -1 / 64, device="cuda")
    p, grad = torch.randn(3000, device="cuda"), torch.randn(3000, device="cuda")
    q, sp, sq = p.clone(), muon.adamw_state(p, 8), muon.adamw_state(p, 8)

    def work(p, state):
        a = muon.token_logprobs_loss(x, y, gl, top=4)
        b = muon.balance_loss(s, ids)
        c = muon.balance_loss_backward(s, b, one, one)
        muon.adamw_step([p], [grad], [state], 1)
        return [*a[:5], a.grad, *b[:5], c]

    want = work(q, sq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        got = work(p, sp)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got + [p], want + [q]):
        assert torch.equal(a, b)
