"""The tagger: encoder, semi-CRF loss and AdamW together, and its streaming
form."""
import pytest
import torch

from semi_markov_crf_zero_amd import optim, tagger

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_training_lowers_the_loss(bits, dtype):
    losses = tagger.main(["--steps", "40", "--bits", str(bits), "--dtype", dtype])
    assert all(x == x for x in losses)
    assert sum(losses[-5:]) / 5 < 0.6 * losses[0]


def test_padding_changes_nothing():
    """1e30 past the lengths: the same loss, gradients and segments."""
    torch.manual_seed(0)
    model = tagger.SemiCRFTagger(24, 64, 8, 16).to(DEV)
    x, lengths, gold = tagger.synthetic(5, 80, 24, 8, 16, seed=3)
    a = model.loss(x, lengths, gold).sum()
    want = torch.autograd.grad(a, list(model.parameters()))
    y = x.clone()
    for b, n in enumerate(lengths.tolist()):
        y[b, n:] = 1e30
    b = model.loss(y, lengths, gold).sum()
    got = torch.autograd.grad(b, list(model.parameters()))
    assert torch.equal(a, b)
    for (n, _), g, w in zip(model.named_parameters(), got, want):
        # the products of the linear layers run over the padding too (times
        # zeros): only their order of summation is the library's
        assert torch.allclose(g, w, rtol=1e-4, atol=1e-5 * float(w.abs().max())), n
    s, t = model.decode(x, lengths), model.decode(y, lengths)
    for k in s:
        assert torch.equal(s[k], t[k]), k


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_give_what_the_sequence_gives(dtype):
    """float32: the same sums in another order, 1e-4 of the emissions' scale;
    bfloat16: every layer's results are rounded to 2^-8 on both ways and the
    two differ by a few of those roundings."""
    torch.manual_seed(0)
    model = tagger.SemiCRFTagger(24, 64, 8, 16, causal=True, dtype=dtype).to(DEV)
    x, _, _ = tagger.synthetic(3, 70, 24, 8, 16, seed=4)
    with torch.no_grad():
        whole, states = model.emissions(x)
        first, mid = model.emissions(x[:, :33])
        rest, end = model.emissions(x[:, 33:], states=mid)
    pool = model.stream_states(6)
    slots = torch.tensor([4, 0, 3], dtype=torch.int32, device=DEV)
    steps = torch.stack([model.step(x[:, t], pool, slots) for t in range(70)], 1)
    scale = float(whole.abs().max())
    tol = (1e-4 if dtype == torch.float32 else 6 * 2.0 ** -8) * scale
    assert float((torch.cat([first, rest], 1) - whole).abs().max()) <= tol
    assert float((steps - whole).abs().max()) <= tol
    for p, s, e in zip(pool, states, end):
        top = float(s.abs().max())
        assert float((p[slots.long()] - s).abs().max()) <= tol / scale * 4 * top
        assert float((e - s).abs().max()) <= tol / scale * 4 * top
        assert not p[[1, 2, 5]].any()


def test_refusals():
    with pytest.raises(ValueError):
        tagger.SemiCRFTagger(24, 64, 8, 16, heads=5)
    model = tagger.SemiCRFTagger(24, 64, 8, 16).to(DEV)
    with pytest.raises(ValueError):
        model.step(torch.zeros((2, 24), device=DEV), model.stream_states(2))


def test_optimizer_follows_a_schedule():
    """torch schedulers change a group's learning rate between steps."""
    model = tagger.SemiCRFTagger(24, 64, 8, 16).to(DEV)
    opt = optim.AdamW(model.parameters(), lr=1e-2, weight_decay=0.0)
    sched = torch.optim.lr_scheduler.StepLR(opt, 1, gamma=0.0)
    for p in model.parameters():
        p.grad = torch.ones_like(p)
    opt.step()
    sched.step()
    before = [p.clone() for p in model.parameters()]
    opt.step()
    assert all(torch.equal(a, b) for a, b in zip(before, model.parameters()))


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 1e30])
@pytest.mark.parametrize("causal,dtype", [(False, torch.float32), (True, torch.float32),
                                          (True, torch.float16)])
def test_what_is_past_the_lengths_is_not_used(causal, dtype, fill):
    """The same loss, gradients and segments whatever it holds."""
    torch.manual_seed(0)
    model = tagger.SemiCRFTagger(24, 64, 8, 16, causal=causal, dtype=dtype).to(DEV)
    x, lengths, gold = tagger.synthetic(5, 80, 24, 8, 16, seed=3)
    y = x.clone()
    for b, n in enumerate(lengths.tolist()):
        y[b, n:] = fill
    (a, want), (b, got) = (
        (loss, torch.autograd.grad(loss, list(model.parameters())))
        for loss in (model.loss(t, lengths, gold).sum() for t in (x, y)))
    assert torch.isfinite(a) and torch.allclose(a, b, rtol=1e-6, atol=0)
    for (n, _), g, w in zip(model.named_parameters(), got, want):
        # 8 roundings of the linear layers' type in a sum of another order
        unit = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -20
        assert w.isfinite().all() and g.isfinite().all(), n
        assert float((g - w).abs().max()) <= 8 * unit * float(w.abs().max()), n
    s, t = model.decode(x, lengths), model.decode(y, lengths)
    for k in s:
        assert torch.equal(s[k], t[k]), k


def test_the_longest_sequence():
    """2^20 positions in one call and in three that continue each other: the
    same sums in another order, 1e-4 of the emissions' scale, and a loss over
    all of them with finite gradients."""
    torch.manual_seed(0)
    model = tagger.SemiCRFTagger(8, 32, 4, 8, heads=2, groups=4, causal=True).to(DEV)
    T = 1 << 20
    x = torch.randn((1, T, 8), device=DEV)
    with torch.no_grad():
        whole, end = model.emissions(x)
        parts, states = [], None
        for a, b in ((0, 300001), (300001, 999999), (999999, T)):
            o, states = model.emissions(x[:, a:b], states=states)
            parts.append(o)
    scale = float(whole.abs().max())
    assert float((torch.cat(parts, 1) - whole).abs().max()) <= 1e-4 * scale
    for s, e in zip(states, end):
        assert float((s - e).abs().max()) <= 1e-4 * float(e.abs().max())
    o, _ = model.emissions(x, torch.tensor([T - 5], dtype=torch.int32, device=DEV))
    o.square().mean().backward()
    assert all(p.grad is None or p.grad.isfinite().all() for p in model.parameters())
