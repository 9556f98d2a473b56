"""The gated delta rule where beta is 0 and gradients, or values, are small.

Gradients are linear in the incoming ones, and in the values together with the states: scaled by a
power of two they have the same digits.  Half a step of float32 each of 64 roundings in a row, 2^-18, of the
norm of what belongs to the positions in question."""
import pytest
import torch

from semi_markov_crf_zero_amd import encoder
from tests.test_gpu_delta import DEV, NAMES, draw

pytestmark = pytest.mark.gpu


def gradients(t, do=1.0, v=1.0):
    d = {n: x.to(DEV).requires_grad_(n in NAMES) for n, x in t.items()}
    o, last = encoder.gated_delta(d["q"], d["k"], d["v"] * v, d["g"], d["b"], state=d["state"] * v, return_state=True)
    out = torch.autograd.grad((o, last), [d[n] for n in NAMES], (d["do"] * do, d["ds"] * do))
    return dict(zip(NAMES, out))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [140, 900])
@pytest.mark.parametrize("betas", ["some", "all", "tiny"])
@pytest.mark.parametrize("small", [-20, -40, -50])
@pytest.mark.parametrize("which", ["do", "v"])
def test_gradients_of_betas_of_zero(which, small, betas, T, dtype):
    t = draw(31, 2, T, (2, 2, 2), 32, 48, dtype)
    t["b"][:, ::3] = 0.0
    if betas == "all":
        t["b"] *= 0.0
    elif betas == "tiny":
        t["b"][:, ::3] = 2.0 ** -80
    got, want = gradients(t, **{which: 2.0 ** small}), gradients(t)
    x, y = got["b"][:, ::3] * 2.0 ** -small, want["b"][:, ::3]
    assert float(y.norm()) > 0
    assert float((x - y).norm()) <= 2.0 ** -18 * float(y.norm())


def test_what_is_not_written_is_not_read():
    """All betas 0: the state decays, and nothing else is read but 2^-64 of each of 900 values below 2^3."""
    t = draw(32, 2, 900, (2, 2, 2), 32, 48, "f32")
    d = {n: x.to(DEV) for n, x in t.items()}
    o, last = encoder.gated_delta(d["q"], d["k"], d["v"], d["g"], d["b"] * 0, return_state=True)
    assert float(o.abs().max()) <= 2.0 ** -50 and float(last.abs().max()) <= 2.0 ** -50
    last = encoder.gated_delta(d["q"], d["k"], d["v"], d["g"], d["b"] * 0, state=d["state"], return_state=True)[1]
    want = d["state"].double() * d["g"].double().sum(1).exp()[..., None, None]
    assert float((last - want).abs().max()) <= 2.0 ** -18 * float(want.abs().max()) + 2.0 ** -50
