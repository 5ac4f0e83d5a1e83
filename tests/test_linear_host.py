"""Host-side checks of fp4_quantize, fp4_values, fp4_mm, layer_norm and
layer_norm_backward (no GPU): sizes, no-ops and every refusal, with fake device
addresses that no call gets as far as touching; and the binding's own checks."""

import ctypes
import os

import pytest
import torch

from newton_schulz_08_gb300 import muon

A, STEP = 0x7F0000000000, 0x10000000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(muon.LIB_PATH):
        from newton_schulz_08_gb300 import build
        build.build()
    return muon.lib()


def at(k, off=0):
    return A + k * STEP + off


def matrix(k=0, rows=100, cols=200, block=32, **kw):
    d = dict(codes=at(3 * k), scales=at(3 * k + 1), scale=at(3 * k + 2) if block == 16 else 0, rows=rows, cols=cols,
             block=block, reserved=0)
    d.update(kw)
    return muon.fp4_matrix(*[d[f[0]] for f in muon.fp4_matrix._fields_])


def code(name):
    return getattr(muon, "MUON_ERR_" + name)


def test_sizes(L):
    assert L.fp4_codes_size(3, 1) == 3 * 16 and L.fp4_codes_size(3, 33) == 3 * 32 and L.fp4_codes_size(0, 5) == 0
    assert L.fp4_scales_size(1, 1, 32) == 1024 and L.fp4_scales_size(129, 257, 32) == 2 * 4 * 512
    assert L.fp4_scales_size(1, 1, 16) == 2048 and L.fp4_scales_size(128, 256, 16) == 2048
    assert L.fp4_codes_size(-1, 4) == 0 and L.fp4_scales_size(4, 4, 8) == 0
    assert L.layer_norm_backward_workspace_size(10, 0) == 0 and L.layer_norm_backward_workspace_size(10, 100) > 0


def quantize(L, x=at(20), dtype=muon.MUON_BF16, rows=100, cols=200, stride=200, along="default", across=None):
    along = matrix(rows=rows, cols=cols) if along == "default" else along
    return L.fp4_quantize(x, dtype, rows, cols, stride, along, across, 0, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"), (dict(stride=199), "INVALID_ARG"),
    (dict(along=None), "INVALID_ARG"), (dict(x=None), "INVALID_ARG"), (dict(x=at(20, 1)), "MISALIGNED"),
    (dict(along=matrix(rows=99)), "INVALID_ARG"), (dict(along=matrix(cols=201)), "INVALID_ARG"),
    (dict(along=matrix(block=8)), "INVALID_ARG"), (dict(along=matrix(reserved=1)), "INVALID_ARG"),
    (dict(along=matrix(block=16, scale=0)), "INVALID_ARG"), (dict(along=matrix(scale=at(2))), "INVALID_ARG"),
    (dict(along=matrix(codes=0)), "INVALID_ARG"), (dict(along=matrix(scales=0)), "INVALID_ARG"),
    (dict(along=matrix(codes=at(0, 8))), "MISALIGNED"), (dict(along=matrix(scales=at(1, 4))), "MISALIGNED"),
    (dict(along=matrix(block=16, scale=at(2, 2))), "MISALIGNED"),
    (dict(across=matrix(1)), "INVALID_ARG"),                                   # not the transpose's shape
    (dict(along=matrix(block=16), across=matrix(1, 200, 100)), "INVALID_ARG"),  # other blocks
    (dict(along=matrix(block=16), across=matrix(1, 200, 100, 16)), "INVALID_ARG"),  # other scale arrays
    (dict(along=matrix(codes=at(20))), "ALIASING"), (dict(along=matrix(scales=at(0, 64))), "ALIASING"),
    (dict(across=matrix(1, 200, 100, codes=at(0, 256))), "ALIASING"),
    (dict(stride=(1 << 32) + 8), "TOO_LARGE"), (dict(rows=1 << 31, along=matrix(rows=1 << 31)), "TOO_LARGE"),
])
def test_quantize_refuses(L, kw, want):
    assert quantize(L, **kw) == code(want)


def test_nothing_to_do(L):
    assert quantize(L, rows=0, x=None) == muon.MUON_OK
    assert quantize(L, cols=0, stride=0, x=None) == muon.MUON_OK
    assert L.fp4_values(matrix(rows=0), None, 0, 200, None) == muon.MUON_OK
    assert L.fp4_mm(matrix(rows=0), matrix(1), None, 0, 100, None, 0, None) == muon.MUON_OK
    assert norm(L, rows=0) == muon.MUON_OK


@pytest.mark.parametrize("kw,want", [
    (dict(q=matrix(block=4)), "INVALID_ARG"), (dict(dtype=5), "INVALID_ARG"), (dict(stride=100), "INVALID_ARG"),
    (dict(out=None), "INVALID_ARG"), (dict(out=at(9, 1)), "MISALIGNED"), (dict(out=at(0, 64)), "ALIASING"),
    (dict(stride=1 << 33), "TOO_LARGE"),
])
def test_values_refuses(L, kw, want):
    a = dict(q=matrix(), out=at(9), dtype=muon.MUON_BF16, stride=200)
    a.update(kw)
    assert L.fp4_values(a["q"], a["out"], a["dtype"], a["stride"], None) == code(want)


@pytest.mark.parametrize("kw,want", [
    (dict(a=matrix(cols=201)), "INVALID_ARG"), (dict(a=matrix(block=16)), "INVALID_ARG"), (dict(dtype=3), "INVALID_ARG"),
    (dict(stride=49), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"),
    (dict(a=None), "INVALID_ARG"), (dict(b=matrix(1, -1)), "INVALID_ARG"),
    (dict(out=at(9, 2), dtype=muon.MUON_F32), "MISALIGNED"), (dict(ws=at(10, 128)), "MISALIGNED"),
    (dict(bytes=255), "WORKSPACE_TOO_SMALL"), (dict(out=at(0)), "ALIASING"), (dict(out=at(4, 16)), "ALIASING"),
    (dict(ws=at(3)), "ALIASING"), (dict(ws=at(9, 256)), "ALIASING"), (dict(stride=1 << 33), "TOO_LARGE"),
])
def test_product_refuses(L, kw, want):
    p = dict(a=matrix(), b=matrix(1, 50), out=at(9), dtype=muon.MUON_BF16, stride=50, ws=at(10), bytes=256)
    p.update(kw)
    assert L.fp4_mm(p["a"], p["b"], p["out"], p["dtype"], p["stride"], p["ws"], p["bytes"], None) == code(want)


def norm(L, **kw):
    p = dict(x=at(0), dtype=muon.MUON_BF16, rows=10, cols=100, sx=100, res=None, sr=0, w=at(2), b=at(3),
             wt=muon.MUON_F32, eps=1e-5, y=at(4), sy=100, sum=None, ss=0, mean=at(6), rstd=at(7))
    p.update(kw)
    return L.layer_norm(p["x"], p["dtype"], p["rows"], p["cols"], p["sx"], p["res"], p["sr"], p["w"], p["b"], p["wt"],
                        p["eps"], p["y"], p["sy"], p["sum"], p["ss"], p["mean"], p["rstd"], None)


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), "INVALID_ARG"), (dict(wt=-1), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"), (dict(cols=0), "INVALID_ARG"),
    (dict(sx=99), "INVALID_ARG"), (dict(sy=99), "INVALID_ARG"), (dict(eps=-1e-9), "INVALID_ARG"), (dict(eps=NAN), "INVALID_ARG"),
    (dict(eps=INF), "INVALID_ARG"), (dict(res=at(1), sr=100), "INVALID_ARG"), (dict(sum=at(1), ss=100), "INVALID_ARG"),
    (dict(res=at(1), sr=99, sum=at(5), ss=100), "INVALID_ARG"), (dict(res=at(1), sr=100, sum=at(5), ss=99), "INVALID_ARG"),
    (dict(x=None), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"), (dict(mean=None), "INVALID_ARG"), (dict(rstd=None), "INVALID_ARG"),
    (dict(x=at(0, 1)), "MISALIGNED"), (dict(y=at(4, 1)), "MISALIGNED"), (dict(w=at(2, 2)), "MISALIGNED"),
    (dict(b=at(3, 1), wt=muon.MUON_BF16), "MISALIGNED"), (dict(mean=at(6, 2)), "MISALIGNED"), (dict(rstd=at(7, 1)), "MISALIGNED"),
    (dict(y=at(0, 2)), "ALIASING"), (dict(y=at(0), sy=104), "ALIASING"), (dict(mean=at(7, 4)), "ALIASING"), (dict(y=at(2, 4)), "ALIASING"),
    (dict(res=at(1), sr=100, sum=at(5), ss=100, y=at(0)), "ALIASING"),  # the sum is normalised: x is not written
    (dict(res=at(1), sr=100, sum=at(0, 2), ss=100), "ALIASING"), (dict(res=at(1), sr=100, sum=at(4), ss=100), "ALIASING"),
    (dict(cols=(1 << 24) + 1, sx=1 << 25, sy=1 << 25), "TOO_LARGE"), (dict(sx=1 << 33), "TOO_LARGE"), (dict(rows=1 << 31), "TOO_LARGE"),
])
def test_layer_norm_refuses(L, kw, want):
    assert norm(L, **kw) == code(want)


def norm_backward(L, **kw):
    p = dict(g=at(0), sg=100, x=at(1), sx=100, dtype=muon.MUON_BF16, rows=10, cols=100, mean=at(2), rstd=at(3), w=at(4),
             wt=muon.MUON_F32, gs=None, sgs=0, gx=at(6), sgx=100, gw=at(7), gb=at(8), ws=at(9), bytes=1 << 27)
    p.update(kw)
    return L.layer_norm_backward(p["g"], p["sg"], p["x"], p["sx"], p["dtype"], p["rows"], p["cols"], p["mean"], p["rstd"], p["w"],
                                 p["wt"], p["gs"], p["sgs"], p["gx"], p["sgx"], p["gw"], p["gb"], p["ws"], p["bytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), "INVALID_ARG"), (dict(cols=0), "INVALID_ARG"), (dict(sg=99), "INVALID_ARG"), (dict(sx=99), "INVALID_ARG"),
    (dict(sgx=99), "INVALID_ARG"), (dict(gs=at(5), sgs=99), "INVALID_ARG"), (dict(g=None), "INVALID_ARG"), (dict(x=None), "INVALID_ARG"),
    (dict(mean=None), "INVALID_ARG"), (dict(rstd=None), "INVALID_ARG"), (dict(gx=None), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"),
    (dict(bytes=100), "WORKSPACE_TOO_SMALL"), (dict(ws=at(9, 16)), "MISALIGNED"), (dict(g=at(0, 1)), "MISALIGNED"),
    (dict(gx=at(6, 1)), "MISALIGNED"), (dict(gw=at(7, 2)), "MISALIGNED"), (dict(gb=at(8, 2)), "MISALIGNED"), (dict(gs=at(5, 1), sgs=100), "MISALIGNED"),
    (dict(gx=at(1)), "ALIASING"), (dict(gx=at(0, 2)), "ALIASING"), (dict(gx=at(0), sgx=101), "ALIASING"), (dict(gw=at(8, 4)), "ALIASING"),
    (dict(gb=at(9)), "ALIASING"), (dict(gs=at(6, 4), sgs=100), "ALIASING"), (dict(gw=at(4)), "ALIASING"),
    (dict(sg=1 << 33), "TOO_LARGE"),
])
def test_layer_norm_backward_refuses(L, kw, want):
    assert norm_backward(L, **kw) == code(want)


# ----------------------------------------------------------------- the binding
def test_binding_refuses():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        muon.layer_norm(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        muon.fp4_quantize(x)
    with pytest.raises(ValueError, match="block"):
        muon.fp4_quantize(x, block=8)
    with pytest.raises(ValueError, match="axis"):
        muon.fp4_quantize(x, axis=2)
    with pytest.raises(ValueError, match="2-D"):
        muon.fp4_quantize(torch.zeros(2, 4, 8))
    with pytest.raises(ValueError, match="contiguous rows"):
        muon.layer_norm(torch.zeros(8, 4).t(), w)
    with pytest.raises(TypeError):
        muon.layer_norm(x.half(), w)
    with pytest.raises(ValueError, match="one entry per column"):
        muon.layer_norm(x, torch.zeros(7))
    with pytest.raises(ValueError, match="same dtype"):
        muon.layer_norm(x, w, w.bfloat16())
    with pytest.raises(ValueError, match="shape and dtype"):
        muon.layer_norm_backward(x.bfloat16(), x, torch.zeros(4), torch.zeros(4), w)
    with pytest.raises(ValueError, match="one entry per row"):
        muon.layer_norm_backward(x, x, torch.zeros(3), torch.zeros(4), w)
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    for bad in (dict(codes=u8(47)), dict(scales=u8(1023)), dict(block=8), dict(scale=torch.zeros(2)), dict(rows=-3)):
        with pytest.raises(ValueError):
            muon.FP4(**{**dict(codes=u8(48), scales=u8(1024), rows=3, cols=5), **bad})
    with pytest.raises(ValueError, match="CUDA"):
        muon.FP4(u8(48), u8(1024), 3, 5)


def test_exports_of_the_operators(L):
    assert ctypes.sizeof(muon.fp4_matrix) == 48
