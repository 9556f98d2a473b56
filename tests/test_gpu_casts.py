"""A rotary tagger cast to the type that it has: the same emissions."""
import pytest
import torch

from semi_markov_crf_zero_amd import tagger

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("memory", ["linear", "delta"])
def test_a_cast_to_float32_changes_nothing(memory):
    torch.manual_seed(0)
    model = tagger.SemiCRFTagger(24, 64, 8, 16, causal=True, memory=memory, rotary=True).to(DEV)
    x, lengths, _ = tagger.synthetic(3, 70, 24, 8, 16, seed=4)
    starts = torch.full((3,), 1 << 20, dtype=torch.int32, device=DEV)
    with torch.no_grad():
        want = model.emissions(x, lengths, starts=starts)[0]
        assert torch.equal(model.float().emissions(x, lengths, starts=starts)[0], want)
        assert torch.equal(model.to(DEV, torch.float32).emissions(x, lengths, starts=starts)[0], want)
        pool = model.stream_states(3)
        assert model.step(x[:, 0], pool, positions=starts).isfinite().all()
