"""The tagger as a module (no GPU): casts."""
import pytest
import torch
from torch import nn

from semi_markov_crf_zero_amd import encoder, tagger


def make(**kw):
    return tagger.SemiCRFTagger(24, 64, 8, 16, causal=True, memory="delta", rotary=True, **kw)


@pytest.mark.parametrize("cast", [lambda m: m.float(), lambda m: m.to(torch.float32), lambda m: m.half(),
                                  lambda m: m.bfloat16().float(), lambda m: m.to("cpu", torch.float16),
                                  lambda m: nn.Sequential(m).float()[0]])
def test_casts_leave_the_frequencies_as_they_are(cast):
    model = cast(make())
    assert torch.equal(model.frequencies, encoder.rotary_frequencies(16))
    assert model.frequencies.dtype == torch.float64 and "frequencies" in dict(model.named_buffers())
    assert "frequencies" not in model.state_dict()


def test_casts_keep_frequencies_that_were_set():
    model = make()
    model.frequencies = encoder.rotary_frequencies(16, stretch=8.0)
    assert torch.equal(model.float().frequencies, encoder.rotary_frequencies(16, stretch=8.0))


def test_other_devices_are_followed():
    model = make().to("meta", torch.float32)
    assert model.frequencies.device.type == "meta" and model.frequencies.dtype == torch.float64
    assert tagger.SemiCRFTagger(24, 64, 8, 16).float().frequencies is None


def test_a_model_without_memory_gets_its_frequencies():
    with torch.device("meta"):
        model = make()
    assert model.frequencies.is_meta
    model = model.to_empty(device="cpu")
    assert torch.equal(model.frequencies, encoder.rotary_frequencies(16))
    assert torch.equal(model.to("cpu").frequencies, encoder.rotary_frequencies(16))
