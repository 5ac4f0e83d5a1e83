"""The operators around a linear layer together, as a training step and a
decoding step use them; other streams, CUDA graphs, and the debug build, whose
results equal the release library's bit for bit."""

import ctypes

import pytest
import torch

from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32


def rand(*shape, seed=0, kind=B):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(kind)


class Block:
    """x + down(relu(up(norm(x)))) with 4-bit products, and its gradients by hand."""

    def __init__(self, width=192, hidden=320, block=32):
        self.block = block
        self.gain, self.bias = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
        self.up, self.down = rand(hidden, width, seed=1, kind=F) * 0.1, rand(width, hidden, seed=2, kind=F) * 0.1

    def linear(self, x, w):
        x, x_t = muon.fp4_quantize(x, block=self.block, axis="both")
        w, w_t = muon.fp4_quantize(w, block=self.block, axis="both")
        return muon.fp4_mm(x, w), (x_t, w_t)

    def linear_backward(self, g, saved, seed):
        x_t, w_t = saved
        g, g_t = muon.fp4_quantize(g, block=self.block, axis="both", seed=seed)
        return muon.fp4_mm(g, w_t), muon.fp4_mm(g_t, x_t, dtype=F)

    def forward(self, x, residual):
        n = muon.layer_norm(x, self.gain, self.bias, residual=residual)
        h, up = self.linear(n.y, self.up)
        a = torch.relu(h)
        out, down = self.linear(a, self.down)
        return out, (n, h, up, down)

    def backward(self, g, saved, seed):
        n, h, up, down = saved
        ga, g_down = self.linear_backward(g, down, seed)
        gy, g_up = self.linear_backward(ga * (h > 0), up, seed + 1)
        gx, g_gain, g_bias = muon.layer_norm_backward(gy, n.sum, n.mean, n.rstd, self.gain, grad_sum=g)
        return gx, g_up, g_down, g_gain, g_bias


class Values(torch.autograd.Function):
    """A linear layer on the 4-bit operands' numbers, its gradient with the same operands."""

    @staticmethod
    def forward(ctx, x, w, block, seed):
        q = lambda t, axis: muon.fp4_values(muon.fp4_quantize(t, block=block, axis=axis), F).double()  # noqa: E731
        ctx.saved = q(x, 0), q(w, 0), block, seed
        return (q(x, 1) @ q(w, 1).t()).to(B).double()

    @staticmethod
    def backward(ctx, g):
        x_t, w_t, block, seed = ctx.saved
        q = lambda axis: muon.fp4_values(muon.fp4_quantize(g.to(B), block=block, axis=axis, seed=seed), F).double()  # noqa: E731
        return (q(1) @ w_t.t()).to(B).double(), q(0) @ x_t.t(), None, None


@pytest.mark.parametrize("block", [32, 16])
def test_block_of_a_model(block):
    """Forward and gradients against autograd in float64 on the same quantised operands.  Roundings to bfloat16 are
    taken at the same places; where a float64 and an fp32 sum round apart (2^-8 of a value, in one in some thousand), an
    operand of the next product may fall to the next code, so results are compared in norm: 2^-6."""
    m = Block(block=block)
    x, res, g = rand(500, 192, seed=3), rand(500, 192, seed=4), rand(500, 192, seed=5) * 0.01
    out, saved = m.forward(x, res)
    got = m.backward(g, saved, 11)
    s = (x.float() + res.float()).to(B).double().requires_grad_(True)
    gain, bias = (t.double().requires_grad_(True) for t in (m.gain, m.bias))
    up, down = (t.clone().requires_grad_(True) for t in (m.up, m.down))
    y = torch.nn.functional.layer_norm(s, (192,), gain, bias)
    y = y + (y.detach().to(B).double() - y.detach())           # rounded, its gradient passed on
    h = Values.apply(y.to(B), up, block, 12)
    want = Values.apply(torch.relu(h).to(B), down, block, 11)
    near = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm()) < 2.0 ** -6  # noqa: E731
    assert near(out, want.detach())
    grads = torch.autograd.grad(want, [s, up, down, gain, bias], g.double())
    for a, b, name in zip(got, (grads[0] + g.double(), *grads[1:]), ("x", "up", "down", "gain", "bias")):
        assert near(a, b), name


def test_training_step_feeds_the_optimizers():
    """The gradients go to the Muon and AdamW steps as they are."""
    m = Block()
    out, saved = m.forward(rand(256, 192, seed=3), rand(256, 192, seed=4))
    gx, g_up, g_down, g_gain, g_bias = m.backward(out, saved, 0)
    before = [t.clone() for t in (m.up, m.down, m.gain, m.bias)]
    muon.muon_step([m.up, m.down], [g_up, g_down], [torch.zeros_like(m.up), torch.zeros_like(m.down)])
    muon.adamw_step([m.gain, m.bias], [g_gain, g_bias], [muon.adamw_state(m.gain), muon.adamw_state(m.bias)], 1)
    for a, b in zip((m.up, m.down, m.gain, m.bias), before):
        assert a.isfinite().all() and not torch.equal(a, b)


@pytest.mark.parametrize("block", [32, 16])
def test_decoding_rows_are_the_prompts(block):
    """A token alone gives the bits that it has among others (blocks of 16: where the tensor's largest entry is the same)."""
    m = Block(block=block)
    x, res = rand(40, 192, seed=3), rand(40, 192, seed=4)
    n = muon.layer_norm(x, m.gain, m.bias, residual=res)
    one = muon.layer_norm(x[7:8], m.gain, m.bias, residual=res[7:8])
    assert torch.equal(one.y, n.y[7:8]) and torch.equal(one.sum, n.sum[7:8])
    w = muon.fp4_quantize(m.up, block=block)
    y = n.y.clone()
    y[:, 0] = 6.0
    a = muon.fp4_mm(muon.fp4_quantize(y, block=block), w, dtype=F)
    b = muon.fp4_mm(muon.fp4_quantize(y[7:8], block=block), w, dtype=F)
    assert torch.equal(a[7:8], b)


# ------------------------------------------------- streams, graphs, debug build
def calls():
    x, res, g, w = rand(300, 500, seed=1), rand(300, 500, seed=2), rand(300, 500, seed=3), rand(500, seed=4, kind=F)
    wide = rand(20, 20001, seed=5)
    n, nw = muon.layer_norm(x, w), muon.layer_norm(wide)
    a, b = muon.fp4_quantize(x), muon.fp4_quantize(rand(400, 500, seed=6))
    c, d = muon.fp4_quantize(rand(2600, 96, seed=7), block=16), muon.fp4_quantize(rand(2500, 96, seed=8), block=16)
    flat = lambda out: [t for t in muon._tensors(out) if t.numel()]  # noqa: E731
    return {
        "layer_norm": lambda st: flat(muon.layer_norm(x, w, w, residual=res, stream=st)),
        "layer_norm_wide": lambda st: flat(muon.layer_norm(wide, stream=st)),
        "layer_norm_backward": lambda st: flat(muon.layer_norm_backward(g, x, n.mean, n.rstd, w, grad_sum=res, stream=st)),
        "layer_norm_backward_wide": lambda st: flat(muon.layer_norm_backward(wide, wide, nw.mean, nw.rstd, stream=st)),
        "fp4_quantize": lambda st: flat(muon.fp4_quantize(x, axis="both", seed=3, stream=st)),
        "fp4_quantize_16": lambda st: flat(muon.fp4_quantize(x, block=16, axis="both", stream=st)),
        "fp4_values": lambda st: flat(muon.fp4_values(a, stream=st)),
        "fp4_mm": lambda st: flat(muon.fp4_mm(a, b, stream=st)),
        "fp4_mm_pairs": lambda st: flat(muon.fp4_mm(c, d, dtype=F, stream=st)),
    }


NAMES = list(("layer_norm layer_norm_wide layer_norm_backward layer_norm_backward_wide fp4_quantize fp4_quantize_16 "
              "fp4_values fp4_mm fp4_mm_pairs").split())


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
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_busy_streams_and_two_calls_at_once(name):
    """Behind a long kernel on another stream, and two calls side by side."""
    f = calls()[name]
    want = f(None)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.ones(1 << 26, device="cuda")
    with torch.cuda.stream(s):
        for _ in range(20):
            busy.mul_(1.0)
    a, b = f(s), f(t)
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, want):
        assert torch.equal(x, z) and torch.equal(y, z)


@pytest.mark.parametrize("name", NAMES)
def test_recorded_in_a_graph(name):
    """Two recordings of a call, replayed one after another and then both again, with a call between them."""
    f = calls()[name]
    want = f(None)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="relaxed"):
            outs.append(f(None))
        graphs.append(g)
    for _ in range(2):
        for g, out in zip(graphs, outs):
            for t in out:
                t.zero_()
            g.replay()
            again = f(None)
            torch.cuda.synchronize()
            for a, b, c in zip(out, again, want):
                assert torch.equal(a, c) and torch.equal(b, c)


def operators():
    """Every operator over its layouts: aligned and not, narrow and wide, few and many tiles; all outputs."""
    out = []
    for kind in (B, F):
        for rows, cols, pad in ((5, 7, 0), (300, 520, 0), (300, 520, 3), (64, 1600, 8), (40, 2100, 0), (20, 12289, 0), (9, 16384, 0), (3, 40001, 0)):
            x, g = rand(rows, cols + pad, seed=1, kind=kind)[:, :cols], rand(rows, cols + pad, seed=2, kind=kind)[:, :cols]
            w = rand(cols, seed=3, kind=F)
            r = muon.layer_norm(x, w, w, residual=g)
            out += [*r, *muon.layer_norm_backward(g, r.sum, r.mean, r.rstd, w, grad_sum=x)]
            for block in (32, 16):
                for seed in (None, 9):
                    q, t = muon.fp4_quantize(x, block=block, axis="both", seed=seed)
                    out += [*muon._tensors((q, t)), muon.fp4_values(q), muon.fp4_values(t, F)]
                out += [muon.fp4_mm(q, q), muon.fp4_mm(q, muon.fp4_quantize(g, block=block), dtype=F)]
    for block in (32, 16):
        a, b = muon.fp4_quantize(rand(3000, 300, seed=1), block=block), muon.fp4_quantize(rand(2999, 300, seed=2), block=block)
        out += [muon.fp4_mm(a, b), muon.fp4_mm(b, a, dtype=F)]
    torch.cuda.synchronize()
    return out


def test_debug_build_passes_its_checks_and_matches_release(monkeypatch):
    want = operators()
    D, n = muon.load(muon.DEBUG_LIB_PATH), ctypes.c_longlong(-1)
    assert D.muon_debug_check_failures(n) == 0  # a debug build; clears the counters
    monkeypatch.setattr(muon, "_lib", D)
    got = operators()
    assert D.muon_debug_check_failures(n) == 0 and n.value == 0
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().reshape(-1).view(torch.uint8), b.contiguous().reshape(-1).view(torch.uint8))
