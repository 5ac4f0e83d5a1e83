"""AdamW where second moments are float32 subnormals and eps does not cover
them: against the oracle, at the tolerances of test_gpu_adamw.  And what the
object holds."""

import pytest
import torch

from newton_schulz_08_gb300 import muon
from tests.test_gpu_adamw import HP, Tensor, step_all

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-22, 1e-15, 1e-12, 1e-8])
def test_subnormal_second_moments(eps, bits, odd):
    """|g| from 1e-21 (a second moment of a few units of the least subnormal) to 1e-15."""
    t = Tensor(1024, "f32", "f32", bits, seed=6, warm=False, odd=odd)
    t.G.copy_(torch.logspace(-21, -15, 1024) * torch.tensor([1.0, -1.0]).repeat(512))
    t.snapshot()
    hp = dict(HP, eps=eps)
    step_all([t], 1, eps=eps, seed=2)
    t.check(1, 0, 2, hp=hp)
    assert bool(torch.isfinite(t.P).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_subnormal_eps(bits):
    """eps below 2^-126: elements without a gradient stay, those with one move."""
    t = Tensor(1000, "f32", "f32", bits, seed=8, warm=False)
    t.G[::3] = 0
    t.snapshot()
    hp = dict(HP, eps=2.0 ** -130)
    step_all([t], 1, eps=2.0 ** -130, seed=2)
    t.check(1, 0, 2, hp=hp)
    assert bool(torch.isfinite(t.P).all())


def test_the_object_keeps_its_tensors_memory():
    """A parameter given other data after the object was made: the memory that the object steps is not handed out again."""
    p, g = torch.nn.Parameter(torch.zeros(1 << 20, device="cuda")), torch.zeros(1 << 20, device="cuda")
    opt = muon.AdamW([p], grads=[g])
    old = {t.data_ptr() for t in (p, g)}
    p.data, g.data = torch.ones(4, device="cuda"), torch.ones(4, device="cuda")
    new = [torch.empty(1 << 20, device="cuda") for _ in range(8)]
    assert not old & {t.data_ptr() for t in new}
    del opt
