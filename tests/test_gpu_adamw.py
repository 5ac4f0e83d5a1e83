"""GPU parity of adamw_step and AdamW with the oracle.

Moments, codes and scales are decisions in float32 with one rounding per
operation: they must equal the oracle's "fp32" mode bit for bit.  Parameters:
the oracle takes u from those moments in float64.  The kernel's u has a square
root, a product, a sum and a quotient of at most 2 float32 ulps each (8 x 2^-23
in all, 2^-20 allowed); the parameter adds four roundings.  A bfloat16
parameter must be what the stochastic rounding makes of some value within that
error.  The float32 moments are also bounded against the float64 definition
(three roundings: 2^-22 of the terms' magnitudes)."""

import numpy as np
import pytest
import torch

import oracle
from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu
HP = dict(beta1=0.9, beta2=0.95, eps=1e-8)
KIND = {"f32": torch.float32, "bf16": torch.bfloat16}


class Tensor:
    """One parameter with its gradient and moments on the GPU, and what the oracle starts from."""

    def __init__(self, n, param="f32", grad="bf16", bits=32, seed=0, lr=3e-3, wd=0.1, odd=False, warm=True):
        rng = np.random.default_rng(1000 * seed + n)
        self.n, self.bits, self.lr, self.wd, self.kind = n, bits, lr, wd, param
        dev = lambda a, k: self.place(torch.from_numpy(a.astype(np.float32)).to("cuda").to(k), odd)  # noqa: E731
        self.P = dev(rng.standard_normal(n) * 0.02, KIND[param])
        self.G = dev(rng.standard_normal(n) * 1e-3, KIND[grad])
        self.S = muon.adamw_state(self.P, bits)
        if warm:
            m = torch.from_numpy((rng.standard_normal(n) * 3e-4).astype(np.float32))
            v = torch.from_numpy((rng.standard_normal(n) * 1e-3).astype(np.float32)) ** 2
            if bits == 32:
                self.S[0].copy_(m)
                self.S[1].copy_(v)
            else:
                for k, x, kind in ((0, m, "m"), (2, v, "v")):
                    q, s = oracle.adamw_quantize(x.numpy(), np.full(n, 32768), kind)
                    self.S[k].copy_(torch.from_numpy(q.astype(np.float32)).to(self.S[k].dtype))
                    self.S[k + 1].copy_(torch.from_numpy(s.astype(np.float32)))
        self.snapshot()

    @staticmethod
    def place(t, odd):
        if not odd:
            return t
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:]
        flat.copy_(t)
        return flat

    def snapshot(self):
        host = lambda t: t.float().cpu().numpy()  # noqa: E731
        self.p, self.g = host(self.P).astype(np.float64), host(self.G)
        if self.bits == 32:
            self.m, self.v = host(self.S[0]), host(self.S[1])
        else:
            self.m = oracle.adamw_dequantize(host(self.S[0]), host(self.S[1])).astype(np.float32)
            self.v = oracle.adamw_dequantize(host(self.S[2]), host(self.S[3])).astype(np.float32)

    def check(self, step, index, seed=0, cautious=False, scale=1.0, hp=HP):
        got = [t.float().cpu().numpy() for t in self.S]
        m, v = oracle.adamw_moments(self.g, self.m, self.v, hp["beta1"], hp["beta2"], scale, "fp32")
        h = oracle.adamw_bits(seed, step, index, self.n)
        if self.bits == 32:
            want = [m, v]
            m64, v64 = oracle.adamw_moments(self.g, self.m.astype(np.float64), self.v.astype(np.float64), hp["beta1"],
                                            hp["beta2"], scale)
            if np.isfinite(self.g).all():
                g = np.abs(self.g.astype(np.float64) * scale)
                assert (np.abs(got[0] - m64) <= 2.0 ** -22 * (np.abs(self.m) + g) + 1e-44).all()
                assert (np.abs(got[1] - v64) <= 2.0 ** -22 * (self.v + g * g) + 1e-44).all()
        else:
            want = [*oracle.adamw_quantize(m, h & 0xFFFF, "m"), *oracle.adamw_quantize(v, h >> 16, "v")]
            for k in (0, 2):  # codes of a block whose scale is NaN say nothing
                dead = np.repeat(np.isnan(want[k + 1]), 256)[:self.n]
                got[k] = np.where(dead, 0, got[k])
                want[k] = np.where(dead, 0, want[k])
        for a, b in zip(got, want):
            np.testing.assert_array_equal(a.astype(np.float64), np.asarray(b, np.float64))
        p, u, decay = oracle.adamw_update(self.p, m, v, step, self.lr, hp["beta1"], hp["beta2"], hp["eps"], self.wd,
                                          cautious)
        gp = self.P.float().cpu().numpy().astype(np.float64)
        with np.errstate(invalid="ignore"):
            move = self.lr / (1 - hp["beta1"] ** step) * np.abs(u)
            err = 2.0 ** -20 * move + 2.0 ** -23 * (np.abs(self.p) + move + np.abs(decay)) + 1e-44
        live = np.isfinite(p)
        np.testing.assert_array_equal(np.isfinite(gp), live)
        np.testing.assert_array_equal(np.isnan(gp), np.isnan(p))
        p, gp, err, h = p[live], gp[live], err[live], h[live]
        if self.kind == "f32":
            assert (np.abs(gp - p) <= err).all(), np.abs((gp - p) / err).max()
        else:
            low, high = oracle.bf16_stochastic(p - err, h), oracle.bf16_stochastic(p + err, h)
            # rounding by the magnitude is monotonic on either side of zero
            assert ((gp >= np.minimum(low, high)) & (gp <= np.maximum(low, high))).all()


def step_all(ts, step, **kw):
    muon.adamw_step([t.P for t in ts], [t.G for t in ts], [t.S for t in ts], step, lr=[t.lr for t in ts],
                    weight_decay=[t.wd for t in ts], **{**HP, **kw})


SIZES = [1, 2, 7, 8, 31, 255, 256, 257, 511, 768, 8191, 8192, 8193, 20_011]


@pytest.mark.parametrize("param", ["f32", "bf16"])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("odd", [False, True])
def test_every_type_over_ragged_sizes(param, grad, bits, odd):
    ts = [Tensor(n, param, grad, bits, seed=i, odd=odd) for i, n in enumerate(SIZES)]
    step_all(ts, 3, seed=77)
    for i, t in enumerate(ts):
        t.check(3, i, 77)


@pytest.mark.parametrize("cautious", [False, True])
@pytest.mark.parametrize("scale", [None, 0.25, 0.37])
def test_mixed_types_rates_and_clipping(cautious, scale):
    kinds = [(p, g, b) for p in ("f32", "bf16") for g in ("f32", "bf16") for b in (32, 8)]
    ts = [Tensor(300 + 17 * i, p, g, b, seed=i, lr=1e-3 * (i + 1), wd=0.0 if i % 3 == 0 else 0.1, odd=i == 5)
          for i, (p, g, b) in enumerate(kinds)]
    s = None if scale is None else torch.tensor([scale], device="cuda")
    step_all(ts, 1, seed=2 ** 40 + 9, cautious=cautious, grad_scale=s)
    for i, t in enumerate(ts):
        t.check(1, i, 2 ** 40 + 9, cautious, np.float32(1.0 if scale is None else scale))


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_chain_from_zero_state(bits):
    ts = [Tensor(n, "bf16" if n % 2 else "f32", "f32", bits, seed=n, warm=False) for n in (256, 1001)]
    opt = muon.AdamW([t.P for t in ts], grads=[t.G for t in ts], states=[t.S for t in ts], lr=3e-3, weight_decay=0.1,
                     seed=5, **HP)
    for step in range(1, 6):
        opt.step()
        for i, t in enumerate(ts):
            t.check(step, i, 5)
            t.snapshot()
    assert opt.steps == 5
    for (m, v), t in zip(opt.state_values(), ts):
        np.testing.assert_array_equal(m.cpu().numpy(), t.m)
        np.testing.assert_array_equal(v.cpu().numpy(), t.v)


def test_more_tensors_than_a_launch_holds():
    """900 tensors of two kinds and lengths, some empty."""
    ts = [Tensor((i * 37) % 530, "f32", "bf16", 8 if i % 5 == 0 else 32, seed=i) for i in range(900)]
    assert any(t.n == 0 for t in ts)
    step_all(ts, 4, seed=3)
    for i, t in enumerate(ts):
        if t.n:
            t.check(4, i, 3)


def test_plan_with_other_gradients_and_rates():
    ts = [Tensor(700, seed=1), Tensor(300, bits=8, seed=2)]
    opt = muon.AdamW([t.P for t in ts], states=[t.S for t in ts], lr=1.0, weight_decay=1.0, seed=1, step=6, **HP)
    with pytest.raises(ValueError):
        opt.step()  # no gradients yet
    opt.set_rates([t.lr for t in ts], 0.1)
    opt.step([t.G for t in ts])
    for i, t in enumerate(ts):
        t.check(7, i, 1)
        t.snapshot()
    new = [torch.randn_like(t.G.float()) * 1e-3 for t in ts]  # another type too
    opt.step(new)
    for i, t in enumerate(ts):
        t.g = new[i].cpu().numpy()
        t.check(8, i, 1)
    with pytest.raises(ValueError):
        opt.set_grads(new[:1])
    with pytest.raises(muon.MuonError) as e:
        opt.set_grads([ts[0].P, new[1]])  # a gradient that is the parameter
    assert e.value.status == muon.MUON_ERR_ALIASING


@pytest.mark.parametrize("bits", [32, 8])
def test_non_finite_gradients_stay_where_they_are(bits):
    """32 bits: the element alone; 8 bits: its block of 256 gets NaN scales, the parameters only the element."""
    t = Tensor(1000, "f32", "f32", bits, seed=9)
    t.G[300], t.G[999] = float("nan"), float("inf")
    t.snapshot()
    step_all([t], 2, seed=1)
    t.check(2, 0, 1)
    assert int((~torch.isfinite(t.P)).sum()) == 2
    if bits == 8:
        assert torch.isnan(t.S[1]).tolist() == [False, True, False, True]


@pytest.mark.parametrize("bits", [32, 8])
def test_extreme_magnitudes(bits):
    """Zeros, the smallest and very large gradients; blocks whose scale is at its least."""
    t = Tensor(1024, "f32", "f32", bits, seed=4, warm=False)
    g = torch.zeros(1024)
    g[256:512] = torch.logspace(-44, -20, 256)
    g[512:768] = torch.logspace(-20, 15, 256)
    g[768:] = torch.tensor([1e18, -1e-18]).repeat(128)
    t.G.copy_(g)
    t.snapshot()
    step_all([t], 1, seed=8)
    t.check(1, 0, 8)
    assert bool(torch.isfinite(t.P).all())


def test_eps_zero_follows_ieee():
    """A zero gradient and zero moments with eps = 0: 0 / 0."""
    t = Tensor(512, "f32", "f32", seed=4, warm=False)
    t.G[:100] = 0
    t.snapshot()
    hp = dict(HP, eps=0.0)
    step_all([t], 1, eps=0.0)
    t.check(1, 0, hp=hp)
    assert int(torch.isnan(t.P).sum()) == 100


def test_large_tensor_and_other_stream():
    """Past 2^24 elements, on a stream of its own; equal calls give equal bits."""
    n = (1 << 24) + 1234
    a, b = (Tensor(n, "bf16", "bf16", 8, seed=3) for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    muon.adamw_step([a.P], [a.G], [a.S], 2, lr=a.lr, weight_decay=a.wd, seed=4, stream=s, **HP)
    torch.cuda.current_stream().wait_stream(s)
    step_all([b], 2, seed=4)
    b.check(2, 0, 4)
    for x, y in zip((a.P, *a.S), (b.P, *b.S)):
        assert torch.equal(x.view(torch.uint8) if x.element_size() == 1 else x, y.view(torch.uint8) if y.element_size() == 1 else y)


def test_matches_torch_adamw_over_steps():
    """32-bit moments, float32: torch.optim.AdamW in float64 over 20 steps."""
    rng = np.random.default_rng(2)
    p = torch.from_numpy(rng.standard_normal(5000).astype(np.float32) * 0.02)
    P, Q = p.cuda(), p.double().requires_grad_(True)
    ref = torch.optim.AdamW([Q], lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    G = torch.zeros_like(P)
    opt = muon.AdamW([P], grads=[G], lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    for _ in range(20):
        g = torch.from_numpy(rng.standard_normal(5000).astype(np.float32) * 1e-3)
        G.copy_(g)
        Q.grad = g.double()
        ref.step()
        opt.step()
    # 20 steps of at most 2^-23 (|p| + moves) rounding each, moves up to about 1e-3
    assert (P.cpu().double() - Q.detach()).abs().max() <= 20 * 2.0 ** -22 * (0.1 + 1e-2)


def test_unsupported_arguments_raise_on_device():
    t = Tensor(300)
    with pytest.raises(muon.MuonError):
        step_all([t], 0)
    with pytest.raises(muon.MuonError):
        muon.adamw_step([t.P], [t.P], [t.S], 1)  # gradient and parameter are one
    with pytest.raises(ValueError):
        step_all([t], 1, grad_scale=torch.ones(1))
    with pytest.raises(ValueError):
        step_all([t], 1, grad_scale=torch.ones(2, device="cuda"))


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("numel", [255, 256, 257, 512, 519, 520, 521, 768, 100_003])
def test_bits_do_not_depend_on_where_arrays_begin(numel, bits):
    """bfloat16 parameters and gradients at every distance to a 16-byte boundary: the same bits as on one, the neighbours untouched."""
    gen = torch.Generator("cuda").manual_seed(numel)
    p, g = (torch.randn(numel, generator=gen, device="cuda").mul_(s).bfloat16() for s in (0.02, 1e-3))

    def run(po, go):
        whole = torch.full((numel + 32,), 3.0, dtype=torch.bfloat16, device="cuda")
        grads = torch.full((numel + 32,), float("nan"), dtype=torch.bfloat16, device="cuda")
        P, G = whole[8 + po:8 + po + numel], grads[8 + go:8 + go + numel]
        P.copy_(p), G.copy_(g)
        state = muon.adamw_state(P, bits)
        for step in (1, 2):
            muon.adamw_step([P], [G], [state], step, lr=1e-3, seed=7)
        assert (whole[:8 + po] == 3.0).all() and (whole[8 + po + numel:] == 3.0).all()
        return [t.reshape(-1).contiguous().view(torch.uint8) for t in (P, *state)]

    want = run(0, 0)
    for po, go in [(k, 0) for k in range(1, 8)] + [(0, 3), (1, 6), (5, 5), (7, 2)]:
        for a, b in zip(run(po, go), want):
            assert torch.equal(a, b), (po, go)
