"""4-bit quantisation and product on the GPU against the oracle.

Codes, scales and values are compared bit for bit.  Products: every product of
two values is exact in fp32; the sum's error is that of fp32 accumulation, at
most K / 64 + 8 roundings (one per instruction of 64 entries, the joining of
up to 8 parts) of 2^-23 (a rounding may truncate) of the sum of magnitudes,
and the last rounding half a step of out's type, 2^-8 or 2^-24 of the value."""

import numpy as np
import pytest
import torch

import oracle
from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32


def rand(*shape, seed=0, spread=2.0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    return x * (torch.randn((shape[0], 1), generator=g, device="cuda") * spread).exp()


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def check_operand(q, x, block, seed, axis):
    """q against the oracle's quantisation of float64 rows x."""
    bits = None if seed is None else oracle.fp4_bits(*x.shape, seed, axis)
    codes, scales, factor = oracle.fp4_quantize(x, block, bits)
    b, s = oracle.fp4_pack(codes, scales, block)
    assert q.shape == x.shape and q.block == block
    assert np.array_equal(q.codes.cpu().numpy(), b)
    assert np.array_equal(q.scales.cpu().numpy(), s)
    if block == 16:
        assert float(q.scale[0]) == factor
        assert float(q.scale[1]) == np.abs(np.where(np.isfinite(x), x, 0.0)).max(initial=0.0)
    want = oracle.fp4_dequantize(codes, scales, factor, block)
    with np.errstate(over="ignore"):  # 2^128 may be the nearest code's number: infinite in float32
        want = want.astype(np.float32)
    assert np.array_equal(muon.fp4_values(q, F).cpu().numpy(), want, equal_nan=True)


SIZES = [(1, 1), (1, 31), (2, 33), (127, 129), (128, 256), (129, 257), (300, 520), (5, 2049), (1025, 8)]


@pytest.mark.parametrize("seed", [None, 0, 2 ** 63 + 12345])
@pytest.mark.parametrize("block", [32, 16])
@pytest.mark.parametrize("kind", [B, F])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantise(rows, cols, kind, block, seed):
    x = rand(rows, cols, seed=rows).to(kind)
    along, across = muon.fp4_quantize(x, block=block, axis="both", seed=seed)
    check_operand(along, f64(x), block, seed, 1)
    check_operand(across, f64(x).T, block, seed, 0)
    for axis, both in ((1, along), (0, across)):
        one = muon.fp4_quantize(x, block=block, axis=axis, seed=seed)
        assert torch.equal(one.codes, both.codes) and torch.equal(one.scales, both.scales)


@pytest.mark.parametrize("block", [32, 16])
@pytest.mark.parametrize("kind", [B, F])
@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 5), (8, 8)])
def test_quantise_views(offset, pad, kind, block):
    whole = rand(70, 300 + pad, seed=offset).to(kind)
    flat = torch.zeros(whole.numel() + 16, dtype=kind, device="cuda")
    flat[offset:offset + whole.numel()] = whole.reshape(-1)
    x = flat[offset:offset + whole.numel()].view(whole.shape)[:, :300]
    along, across = muon.fp4_quantize(x, block=block, axis="both", seed=9)
    check_operand(along, f64(x), block, 9, 1)
    check_operand(across, f64(x).T, block, 9, 0)


@pytest.mark.parametrize("seed", [None, 5])
@pytest.mark.parametrize("block", [32, 16])
def test_every_bfloat16_value(block, seed):
    """All 65536 patterns, in order (neighbours share a block) and mixed; NaN and infinities among them."""
    x = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(B).view(256, 256)
    check_operand(muon.fp4_quantize(x, block=block, seed=seed), f64(x), block, seed, 1)
    y = x.reshape(-1)[torch.randperm(65536, generator=torch.Generator("cuda").manual_seed(1), device="cuda")].view(64, 1024)
    for q, z, axis in zip(muon.fp4_quantize(y, block=block, axis="both", seed=seed), (f64(y), f64(y).T), (1, 0)):
        check_operand(q, z, block, seed, axis)


LARGEST, LEAST = 3.3895e38, 2.0 ** -133


@pytest.mark.parametrize("block", [32, 16])
@pytest.mark.parametrize("kind", [B, F])
@pytest.mark.parametrize("fill", ["zeros", "minus zeros", "largest", "least", "lowest and one", "ties", "powers"])
def test_quantise_special(fill, kind, block):
    x = torch.zeros(64, 64, device="cuda")
    if fill == "minus zeros":
        x = -x
    elif fill == "largest":
        x += LARGEST
        x[:, ::2] *= -1
    elif fill == "least":
        x += LEAST
        x[3] = 2.0 ** -126
    elif fill == "lowest and one":
        x += 1.0
        x[:, 5] = -LARGEST
    elif fill == "ties":
        x[:] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 8, device="cuda")
        x *= torch.pow(2.0, torch.arange(64, device="cuda") - 32.0)[:, None]
    elif fill == "powers":
        x = torch.pow(2.0, torch.arange(4096, device="cuda").remainder(250) - 126.0).view(64, 64)
    x = x.to(kind)
    for seed in (None, 1):
        for q, z, axis in zip(muon.fp4_quantize(x, block=block, axis="both", seed=seed), (f64(x), f64(x).T), (1, 0)):
            check_operand(q, z, block, seed, axis)


def test_quotients_next_to_a_border():
    """Quotients by E4M3 scales within a float32 spacing of a code's border decide as the IEEE quotient does."""
    s = torch.tensor([(8 + m) / 8 for m in range(8)], device="cuda")
    t = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    p = (s[:, None] * t).reshape(-1)
    bits = p.view(torch.int32)[:, None] + torch.arange(-4, 5, device="cuda", dtype=torch.int32)
    near = bits.view(F).reshape(8, -1)
    x = torch.zeros(8, 64, device="cuda")
    x[:, :63] = near
    for k in range(4):
        x[:, 16 * k] = 6 * s  # the block's largest: its scale is s (times the power of two)
    for seed in (None, 3):
        check_operand(muon.fp4_quantize(x, block=16, seed=seed), f64(x), 16, seed, 1)


def test_values_types_and_pitch():
    x = rand(130, 77).to(B)
    for block in (32, 16):
        q = muon.fp4_quantize(x, block=block)
        want = muon.fp4_values(q, F)
        assert torch.equal(muon.fp4_values(q), want.to(B)) and torch.equal(want.to(B).to(F), want)
        for kind in (B, F):
            for pad in (1, 3, 51):
                wide = torch.full((130, 77 + pad), 7.0, dtype=kind, device="cuda")
                muon.fp4_values(q, out=wide[:, :77])
                assert torch.equal(wide[:, :77], want.to(kind)) and (wide[:, 77:] == 7).all()


# ------------------------------------------------------------------ products
def check_product(a, b, out):
    x, y = muon.fp4_values(a, F).double(), muon.fp4_values(b, F).double()
    want, size = x @ y.t(), x.abs() @ y.abs().t()
    half = 2.0 ** -8 if out.dtype == B else 2.0 ** -24
    bound = want.abs() * half + size * ((a.cols / 64 + 9) * 2.0 ** -23) + 2.0 ** -133
    off = (out.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


def operands(m, n, k, block, seed=0, spread=1.0):
    return (muon.fp4_quantize(rand(m, k, seed=seed, spread=spread).to(B), block=block),
            muon.fp4_quantize(rand(n, k, seed=seed + 1, spread=spread).to(B), block=block, seed=4))


def product(a, b, **kw):
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")  # what it held before does not matter
    out = muon.fp4_mm(a, b, workspace=ws, **kw)
    assert muon.muon_device_status(ws) == muon.MUON_OK
    return out


SHAPES = [(1, 1, 1), (1, 5, 33), (3, 200, 300), (31, 33, 64), (32, 128, 65), (33, 129, 255), (64, 64, 256), (65, 300, 257),
          (129, 70, 1000), (200, 4800, 1600), (1, 9000, 512), (9000, 2, 511), (700, 900, 4111), (100, 100, 20000),
          (2560, 2560, 96), (2300, 2400, 1601), (300, 30000, 130), (4097, 2049, 512)]


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("block", [32, 16])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k, block, dtype):
    a, b = operands(m, n, k, block)
    out = product(a, b, dtype=dtype)
    assert out.dtype == dtype and out.shape == (m, n)
    check_product(a, b, out)
    assert torch.equal(out, product(a, b, dtype=dtype))


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("m,n", [(40, 300), (300, 40), (300, 301), (2600, 2599)])
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (2, 3)])
def test_product_into_views(offset, pad, m, n, dtype):
    a, b = operands(m, n, 320, 32, seed=3)
    flat = torch.full(((m + 2) * (n + pad) + 16,), 7.0, dtype=dtype, device="cuda")
    out = flat[offset:offset + m * (n + pad)].view(m, n + pad)[:, :n]
    product(a, b, out=out)
    check_product(a, b, out)
    out.fill_(7.0)
    assert (flat == 7.0).all()  # and nothing beside it was written


@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 3)])
@pytest.mark.parametrize("m,n,k", [(30, 700, 1600), (700, 30, 2500), (20, 300, 2500), (5, 6400, 3300), (6400, 3, 4500), (9, 8192, 4500),
                                   (50, 6400, 6000), (64, 500, 9000), (100, 6400, 10_000), (6401, 100, 10_000), (130, 1200, 2100)])
def test_product_of_shared_sums(m, n, k, offset, pad):
    """Tiles whose K blocks are shared by 2, 4 or 8 CTAs, some of them without a block."""
    for block, dtype in ((32, B), (16, F)):
        a, b = operands(m, n, k, block, seed=5)
        flat = torch.full(((m + 2) * (n + pad) + 16,), 7.0, dtype=dtype, device="cuda")
        out = flat[offset:offset + m * (n + pad)].view(m, n + pad)[:, :n]
        product(a, b, out=out)
        check_product(a, b, out)
        assert torch.equal(out, product(a, b, dtype=dtype))
        out.fill_(7.0)
        assert (flat == 7.0).all()


def test_product_of_extreme_tensors():
    """Factors of 2^-127 and 2^116: their product is taken before anything is lost."""
    x, y = rand(50, 96, spread=0.1), rand(60, 96, seed=1, spread=0.1)
    for block in (16, 32):
        a = muon.fp4_quantize((x * 2.0 ** -120).to(F), block=block)
        b = muon.fp4_quantize((y * 2.0 ** 120).to(F), block=block)
        check_product(a, b, product(a, b, dtype=F))
        c = product(a, a, dtype=F)
        assert torch.equal(c, torch.zeros_like(c))
        zero = muon.fp4_quantize(torch.zeros(7, 96, device="cuda"), block=block)
        assert torch.equal(product(zero, b, dtype=F), torch.zeros(7, 60, device="cuda"))


@pytest.mark.parametrize("m,n", [(40, 300), (2600, 2600)])
@pytest.mark.parametrize("block", [32, 16])
def test_blocks_that_are_not_finite(block, m, n):
    x, y = rand(m, 200).to(B), rand(n, 200, seed=1).to(B)
    x[3, 7], y[n - 1, 199], x[m - 1, 0] = float("nan"), float("inf"), -float("inf")
    out = product(muon.fp4_quantize(x, block=block), muon.fp4_quantize(y, block=block))
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[3] = bad[m - 1] = True
    bad[:, n - 1] = True
    assert torch.equal(out.isnan(), bad)


def test_empty():
    x = torch.zeros(0, 40, device="cuda")
    a, b = muon.fp4_quantize(x, axis="both")
    assert a.shape == (0, 40) and b.shape == (40, 0)
    w = muon.fp4_quantize(rand(50, 40))
    assert muon.fp4_mm(a, w).shape == (0, 50) and muon.fp4_mm(w, a).shape == (50, 0)
    assert torch.equal(product(b, b, dtype=F), torch.zeros(40, 40, device="cuda"))  # empty sums
    assert muon.fp4_values(a).shape == (0, 40)


def test_far_offsets():
    """An output, and an input, whose offsets pass 2^31 elements."""
    m, n = 66_000, 33_000
    a, b = operands(m, n, 64, 32)
    out = product(a, b)
    rows = torch.tensor([0, 1, 40_000, m - 257, m - 1], device="cuda")
    x, y = muon.fp4_values(a, F).double()[rows], muon.fp4_values(b, F).double()
    want = x @ y.t()
    bound = want.abs() * 2.0 ** -8 + (x.abs() @ y.abs().t()) * 10 * 2.0 ** -23
    assert bool(((out[rows].double() - want).abs() <= bound).all())
    q, q_t = muon.fp4_quantize(out, axis="both")
    cut = muon.fp4_quantize(out[m - 128:].clone())
    assert torch.equal(q.codes[m - 128:], cut.codes)
    cut = muon.fp4_quantize(out[:, n - 40:].clone(), axis=0)
    assert torch.equal(q_t.codes[n - 40:], cut.codes)


@pytest.mark.parametrize("m,n,k", [(40, 300, 2000), (2600, 2600, 600)])
def test_a_wait_that_runs_out(m, n, k):
    """With MMAs that are never issued the bounded waits end and the status says so; the next call is right again."""
    a, b = operands(m, n, k, 32)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    muon.muon_set_debug("wait_budget_cycles", 2_000_000)
    muon.muon_set_debug("inject_stall", 1)
    try:
        muon.fp4_mm(a, b, workspace=ws)
        assert muon.muon_device_status(ws) == muon.MUON_ERR_DEVICE_TIMEOUT
    finally:
        muon.muon_set_debug("inject_stall", 0)
        muon.muon_set_debug("wait_budget_cycles", 4_000_000_000)
    check_product(a, b, product(a, b))


def test_refusals_on_the_device():
    a, b = operands(40, 50, 64, 32)
    with pytest.raises(ValueError):
        muon.fp4_mm(a, muon.fp4_quantize(rand(50, 64), block=16))
    with pytest.raises(ValueError):
        muon.fp4_mm(a, muon.fp4_quantize(rand(50, 65)))
    with pytest.raises(ValueError):
        muon.fp4_mm(a, b, out=torch.empty(50, 40, device="cuda"))
    with pytest.raises(TypeError):
        muon.fp4_mm(a, b, dtype=torch.float16)
    with pytest.raises(muon.MuonError):
        muon.fp4_mm(a, b, workspace=torch.zeros(128, dtype=torch.uint8, device="cuda"))
