"""What a recorded fp4_quantize does: its seed is part of the launch, so that every replay has the eager call's bits."""

import pytest
import torch

from newton_schulz_08_gb300 import muon

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [32, 16])
def test_replays_repeat_the_bits_of_their_seed(block):
    x = torch.randn(300, 520, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    want = [t.clone() for seed in (7, 8) for t in muon._tensors(muon.fp4_quantize(x, block=block, axis="both", seed=seed))]
    assert not torch.equal(want[0], want[len(want) // 2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [muon.fp4_quantize(x, block=block, axis="both", seed=seed) for seed in (7, 8)]
    got = list(muon._tensors(held))
    for _ in range(2):
        for t in got:
            t.fill_(0)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
