"""fp4_mm of matrices without columns: zeros in out's rows at any pitch, nothing beside them, and the status cleared."""

import pytest
import torch

from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32


def without_columns(rows, block=32):
    return muon.fp4_quantize(torch.zeros(rows, 0, device="cuda"), block=block)


@pytest.mark.parametrize("block", [32, 16])
@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("m,n,pad", [(1, 1, 0), (3, 5, 2), (5000, 33, 1), (7, 3000, 0)])
def test_zeros(m, n, pad, dtype, block):
    flat = torch.full((m * (n + pad) + 2,), 7.0, dtype=dtype, device="cuda")
    out = flat[1:1 + m * (n + pad)].view(m, n + pad)[:, :n]
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    muon.fp4_mm(without_columns(m, block), without_columns(n, block), out=out, workspace=ws)
    assert muon.muon_device_status(ws) == muon.MUON_OK and not out.any()
    out.fill_(7.0)
    assert (flat == 7.0).all()


@pytest.mark.parametrize("dtype,pitch", [(B, (1 << 30) + 8), (F, (1 << 29) + 3), (B, (1 << 32) - 5), (F, 1 << 32)])
def test_pitch_past_2_31_bytes(dtype, pitch):
    flat = torch.full((pitch + 9,), 7.0, dtype=dtype, device="cuda")
    out = flat.as_strided((2, 9), (pitch, 1))
    muon.fp4_mm(without_columns(2), without_columns(9), out=out)
    assert not out.any() and (flat[9:pitch] == 7.0).all()
    a, b = (muon.fp4_quantize(torch.ones(r, 32, device="cuda")) for r in (2, 9))
    muon.fp4_mm(a, b, out=out)
    assert (out == 32.0).all() and (flat[9:pitch] == 7.0).all()
