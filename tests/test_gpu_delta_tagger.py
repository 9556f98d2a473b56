"""The tagger with the gated delta rule, rotary positions and clipping: the
operators together, in training and position by position."""
import pytest
import torch

from semi_markov_crf_zero_amd import optim, tagger

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(dtype=torch.float32, memory="delta", rotary=True, causal=True):
    torch.manual_seed(0)
    return tagger.SemiCRFTagger(24, 64, 8, 16, causal=causal, dtype=dtype, memory=memory,
                                rotary=rotary).to(DEV)


@pytest.mark.parametrize("args", [["--memory", "delta"], ["--rotary"], ["--clip", "0.5"],
                                  ["--memory", "delta", "--rotary", "--clip", "1.0", "--bits", "8"],
                                  ["--memory", "delta", "--rotary", "--clip", "1.0", "--dtype", "bfloat16"]])
def test_the_command_runs(args):
    losses = tagger.main(["--steps", "4", *args])
    assert len(losses) == 4 and all(x == x and abs(x) < 100 for x in losses)


@pytest.mark.parametrize("memory,rotary", [("delta", False), ("delta", True), ("linear", True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_give_what_the_sequence_gives(dtype, memory, rotary):
    """float32: the same sums in another order, 1e-4 of the emissions' scale;
    bfloat16: every layer's results are rounded to 2^-8 on both ways and the
    two differ by a few of those roundings."""
    model = make(dtype, memory, rotary)
    x, _, _ = tagger.synthetic(3, 70, 24, 8, 16, seed=4)
    at = lambda n: torch.full((3,), n, dtype=torch.int32, device=DEV)  # noqa: E731
    with torch.no_grad():
        whole, states = model.emissions(x)
        first, mid = model.emissions(x[:, :33])
        rest, end = model.emissions(x[:, 33:], states=mid, starts=at(33))
    pool = model.stream_states(6)
    slots = torch.tensor([4, 0, 3], dtype=torch.int32, device=DEV)
    steps = torch.stack([model.step(x[:, t], pool, slots, positions=at(t)) for t in range(70)], 1)
    scale = float(whole.abs().max())
    tol = (1e-4 if dtype == torch.float32 else 6 * 2.0 ** -8) * scale
    assert float((torch.cat([first, rest], 1) - whole).abs().max()) <= tol
    assert float((steps - whole).abs().max()) <= tol
    for p, s, e in zip(pool, states, end):
        top = float(s.abs().max())
        assert float((p[slots.long()] - s).abs().max()) <= tol / scale * 4 * top
        assert float((e - s).abs().max()) <= tol / scale * 4 * top
        assert not p[[1, 2, 5]].any()


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 1e30])
@pytest.mark.parametrize("causal,dtype", [(False, torch.float32), (True, torch.float32),
                                          (True, torch.float16)])
def test_what_is_past_the_lengths_is_not_used(causal, dtype, fill):
    """The same loss and gradients whatever it holds."""
    model = make(dtype, causal=causal)
    x, lengths, gold = tagger.synthetic(5, 80, 24, 8, 16, seed=3)
    y = x.clone()
    for b, n in enumerate(lengths.tolist()):
        y[b, n:] = fill
    (a, want), (b, got) = (
        (loss, torch.autograd.grad(loss, list(model.parameters())))
        for loss in (model.loss(t, lengths, gold).sum() for t in (x, y)))
    assert torch.isfinite(a) and torch.allclose(a, b, rtol=1e-6, atol=0)
    for (n, _), g, w in zip(model.named_parameters(), got, want):
        unit = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -20
        assert w.isfinite().all() and g.isfinite().all(), n
        assert float((g - w).abs().max()) <= 8 * unit * float(w.abs().max()), n


def test_gradients_against_differences():
    """Of the loss along random directions of each parameter, by central differences of the
    float32 model: its rounding, 2^-20 of a loss of about 10^3, over a step of 2^-7 of the
    parameter's norm, and the step's square."""
    model = make(causal=False)
    x, lengths, gold = tagger.synthetic(4, 60, 24, 8, 16, seed=5)
    loss = model.loss(x, lengths, gold).sum()
    loss.backward()
    gen = torch.Generator(device=DEV).manual_seed(1)
    for name, p in model.named_parameters():
        way = torch.randn(p.shape, device=DEV, generator=gen)
        way /= way.norm()
        h = 2.0 ** -7 * max(1.0, float(p.detach().norm()))
        with torch.no_grad():
            values = []
            for sign in (1, -1):
                p += sign * h * way
                values.append(float(model.loss(x, lengths, gold).double().sum()))
                p -= sign * h * way
        want = (values[0] - values[1]) / (2 * h)
        got = float((p.grad * way).sum())
        bar = 2.0 ** -20 * abs(float(loss.detach())) / h + 2.0 ** -5 * float(p.grad.norm())
        assert abs(got - want) <= bar, (name, got, want, bar)


def test_clipping_in_place_and_in_the_step_agree():
    """A clipped gradient is rounded once more than one that the step scales: 2^-24 of it; AdamW's
    first step is lr g / (|g| + eps), which moves by as little."""
    models = [make() for _ in range(2)]
    x, lengths, gold = tagger.synthetic(4, 60, 24, 8, 16, seed=6)
    for i, model in enumerate(models):
        opt = optim.AdamW(model.parameters(), lr=1e-3)
        model.loss(x, lengths, gold).mean().backward()
        if i:
            norm, clip = optim.grad_norm(model.parameters(), max_norm=0.1)
            opt.step(grad_scale=clip)
        else:
            norm = optim.clip_grad_norm_(model.parameters(), 0.1)
            opt.step()
        assert float(norm) > 0.1
    for a, b in zip(*(m.parameters() for m in models)):
        assert float((a - b).abs().max()) <= 1e-6


def test_refusals():
    with pytest.raises(ValueError, match="memory"):
        tagger.SemiCRFTagger(24, 64, 8, 16, memory="other")
    model = make()
    x = torch.zeros((2, 5, 24), device=DEV)
    _, states = model.emissions(x)
    with pytest.raises(ValueError, match="starts"):
        model.emissions(x, states=states)
    with pytest.raises(ValueError, match="positions"):
        model.step(x[:, 0], model.stream_states(2))
