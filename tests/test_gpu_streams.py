"""The `stream` argument: a call under another stream than the current one may
take no memory that the current stream is given meanwhile, or still uses."""

import pytest
import torch

from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu


def calls():
    """Every entry point that allocates: name -> f(stream), outputs as a flat list."""
    g = torch.Generator("cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, y = r(300, 5000), torch.randint(0, 5000, (300,), generator=g, device="cuda")
    gl, s = r(300), r(4096, 64)
    ids, one = torch.randint(0, 64, (4096, 4), generator=g, device="cuda"), torch.ones(1, device="cuda")
    lse, b = muon.token_logprobs(x, y).lse, muon.balance_loss(s, ids, groups=4)
    G, a, w = r(2, 192, 320), r(256, 512).bfloat16(), r(384, 512).bfloat16()
    _, af, wf = muon.fp8_mm(a, w, 0.02, 0.02)
    go, m = r(256, 384).bfloat16(), [r(192, 320) for _ in range(2)]

    def muon_step(st):
        p, buf = [t.clone() for t in m], [torch.zeros_like(t) for t in m]
        torch.cuda.synchronize()
        muon.muon_step(p, m, buf, stream=st)
        return p

    flat = lambda out: [t.view(torch.uint8) if t.element_size() == 1 else t for t in out if t is not None]  # noqa: E731
    return {
        "token_logprobs": lambda st: flat(muon.token_logprobs(x, y, top=4, stream=st)),
        "token_logprobs_backward": lambda st: [muon.token_logprobs_backward(x, y, lse, gl, stream=st)],
        "token_logprobs_loss": lambda st: flat(muon.token_logprobs_loss(x, y, gl, gl, top=4, stream=st)),
        "balance_loss": lambda st: flat(muon.balance_loss(s, ids, groups=4, stream=st)),
        "balance_loss_backward": lambda st: [muon.balance_loss_backward(s, b, one, one, stream=st)],
        "ns5": lambda st: [muon.ns5(G, 5, stream=st)],
        "ns5_bank": lambda st: muon.ns5_bank(m, 5, stream=st),
        "ns5_noalloc": lambda st: [muon.ns5_noalloc(G, 5, stream=st)],
        "fp8_mm": lambda st: flat(muon.fp8_mm(a, w, 0.02, 0.02, stream=st)),
        "fp8_mm_backward": lambda st: flat(muon.fp8_mm_backward(go, af, wf, 0.02, 0.02, 1e-3, stream=st)),
        "muon_step": muon_step,
    }


NAMES = list(("token_logprobs token_logprobs_backward token_logprobs_loss balance_loss balance_loss_backward "
              "ns5 ns5_bank ns5_noalloc fp8_mm fp8_mm_backward muon_step").split())


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_belongs_to_its_stream(name, as_handle, monkeypatch):
    f, s, under = calls()[name], torch.cuda.Stream(), []
    want = f(None)
    torch.cuda.synchronize()
    empty = torch.empty

    def spy(*args, **kw):
        under.append(torch.cuda.current_stream().cuda_stream)
        return empty(*args, **kw)

    monkeypatch.setattr(torch, "empty", spy)
    got = f(s.cuda_stream if as_handle else s)
    monkeypatch.undo()
    assert under and set(under) == {s.cuda_stream}
    torch.cuda.current_stream().wait_stream(s)
    for p, q in zip(got, want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("name", NAMES)
def test_later_allocations_do_not_reach_a_call_in_waiting(name):
    """The other stream is busy when the call comes; the current one then fills blocks of every size that was free."""
    f, s = calls()[name], torch.cuda.Stream()
    want = f(None)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)  # some 20 ms
    got = f(s)
    fill = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for k in range(9, 24) for n in [1 << k, 3 << k - 1] * 4]
    torch.cuda.current_stream().synchronize()
    del fill
    torch.cuda.current_stream().wait_stream(s)
    for p, q in zip(got, want):
        assert torch.equal(p, q)


def test_default_stream_by_its_handle():
    f, s = calls()["balance_loss"], torch.cuda.Stream()
    want = f(None)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = f(0)
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)


def test_stream_of_another_device_is_refused():
    class Elsewhere:
        device, cuda_stream = torch.device("cuda", 1), 1234

    with pytest.raises(ValueError):
        muon.token_logprobs(torch.zeros((2, 4), device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"), stream=Elsewhere())
