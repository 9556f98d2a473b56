"""Forward-mode derivatives and traces of the operators' entry points: refused, whichever way a
call takes past autograd.  No GPU: launches are recorded and not made."""
import pytest
import torch
from torch.autograd import forward_ad
from torch.fx.experimental.proxy_tensor import make_fx

from semi_markov_crf_zero_amd import encoder, optim


@pytest.fixture
def launched(monkeypatch):
    made = []
    monkeypatch.setattr(encoder, "_check_device", lambda t: None)
    monkeypatch.setattr(encoder, "launch", lambda fn, dev, *args: made.append(fn.__name__))
    return made


def calls():
    gen = torch.Generator().manual_seed(0)
    q = torch.randn((2, 5, 2, 8), generator=gen)
    g, b = -torch.rand((2, 5, 2), generator=gen), torch.rand((2, 5, 2), generator=gen)
    f, decay = encoder.rotary_frequencies(8), torch.tensor([-0.1, -0.2])
    pool, state = torch.zeros((2, 2, 8, 8)), torch.ones((2, 2, 8, 8))
    return {
        "linear_attention": (lambda q, g, s: encoder.linear_attention(q, q, q, g, state=s), (q, decay, state)),
        "linear_attention_step": (lambda q, g, s: encoder.linear_attention_step(q, q, q, g, s),
                                  (q[:, 0], decay, pool)),
        "gated_delta": (lambda q, g, b, s: encoder.gated_delta(q, q, q, g, b, state=s), (q, g, b, state)),
        "gated_delta_step": (lambda q, g, b, s: encoder.gated_delta_step(q, q, q, g, b, s),
                             (q[:, 0], g[:, 0], b[:, 0], pool)),
        "rotary": (lambda q, f: encoder.rotary(q, None, f), (q, f)),
        "rotary of both": (lambda q, k: torch.cat(encoder.rotary(q, k, f)), (q, q + 1)),
    }


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("name", list(calls()))
def test_tangents_are_refused(name, grad, launched):
    fn, args = calls()[name]
    with torch.set_grad_enabled(grad):
        for i in range(len(args)):
            with forward_ad.dual_level():
                x = list(args)
                x[i] = forward_ad.make_dual(x[i], torch.ones_like(x[i]))
                with pytest.raises(NotImplementedError):
                    fn(*x)
    assert not launched
    with forward_ad.dual_level():  # a level without a tangent among the arguments
        fn(*args)
    assert len(launched) == 1


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("name", list(calls()))
def test_traces_are_refused(name, grad, launched):
    fn, args = calls()[name]
    with torch.set_grad_enabled(grad), pytest.raises(RuntimeError, match="cannot be traced"):
        torch.jit.trace(fn, args, check_trace=False)
    assert not launched


def test_gradients_with_tangents_are_not_clipped():
    p = torch.zeros(3, requires_grad=True)
    with forward_ad.dual_level():
        p.grad = forward_ad.make_dual(torch.ones(3), torch.ones(3))
        for fn in (optim.clip_grad_norm_, optim.grad_norm):
            with pytest.raises(NotImplementedError):
                fn([p], 1.0)


@pytest.mark.parametrize("name", ["linear_attention", "gated_delta", "rotary", "group_norm"])
def test_incoming_gradients_with_tangents_are_refused(name, launched):
    """A tangent that comes in behind the operator would be lost on its way back."""
    q = calls()["rotary"][1][0].requires_grad_(True)
    if name == "group_norm":
        y = encoder.group_norm(q.flatten(2), 4)
    else:
        fn, args = calls()[name]
        y = fn(q, *args[1:])
    forwards = len(launched)
    with forward_ad.dual_level():
        w = forward_ad.make_dual(torch.ones_like(y), torch.ones_like(y))
        with pytest.raises(NotImplementedError):
            torch.autograd.grad((y * w).sum(), q)
    assert len(launched) == forwards == 1


@pytest.mark.parametrize("mode", ["real", "fake"])
@pytest.mark.parametrize("name", [*calls(), "group_norm"])
def test_recorded_graphs_are_refused(name, mode, monkeypatch):
    """Graphs of torch's operators, from real tensors too: the launch itself says no."""
    monkeypatch.setattr(encoder, "_check_device", lambda t: None)
    fn, args = calls().get(name, (lambda x: encoder.group_norm(x, 4), (torch.randn(2, 5, 8),)))
    with pytest.raises(RuntimeError, match="cannot be traced" if mode == "real" else "data pointer"):
        make_fx(fn, tracing_mode=mode)(*args)
