"""More of the layer's operators: states in many short sequences, gradients over infinities in what is
masked, rotary positions of sequences that lie apart."""
import math

import pytest
import torch

from semi_markov_crf_zero_amd import encoder
from tests.test_gpu_delta import DEV, NAMES, call, draw
from tests.test_gpu_rotary import run

pytestmark = pytest.mark.gpu


def test_many_short_sequences_with_a_state():
    """2^20 sequences and heads of one position, each from its own state, against the formula in
    float64.  Sums of D = 8 products in a chain of four: 64 roundings of 2^-24 of the
    products of norms."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    B, H, D = 1 << 18, 4, 8
    q, k, v = (torch.randn((B, 1, H, D), device=DEV, generator=gen) for _ in range(3))
    k = k / k.norm(dim=-1, keepdim=True)
    g, b = -torch.rand((B, 1, H), device=DEV, generator=gen), torch.rand((B, 1, H), device=DEV, generator=gen)
    state = torch.randn((B, H, D, D), device=DEV, generator=gen)
    o, last = encoder.gated_delta(q, k, v, g, b, state=state, return_state=True)
    Q, K, V = (t.double()[:, 0] for t in (q, k, v))
    S = state.double() * g.double()[:, 0].exp()[..., None, None]
    miss = V - (K[..., None] * S).sum(-2)
    S += b.double()[:, 0, :, None, None] * K[..., None] * miss[..., None, :]
    size = state.norm(dim=(-1, -2))[..., None] + v[:, 0].abs()
    want = D ** -0.5 * (Q[..., None] * S).sum(-2)
    assert ((o[:, 0] - want).abs() <= 64 * 2.0 ** -24 * q[:, 0].norm(dim=-1, keepdim=True) * size).all()
    assert ((last - S).abs() <= 64 * 2.0 ** -24 * size[..., None, :]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,lengths", [(80, [33, 64]), (900, [300, 7])])
def test_gradients_over_infinities_in_what_is_masked(T, lengths, dtype):
    """Queries, values, gates and gradients are infinite past the lengths, keys 0 or infinite."""
    t = draw(23, 2, T, (2, 2, 2), 32, 32, dtype)
    lt = torch.tensor(lengths, dtype=torch.int32, device=DEV)

    def both(d):
        d = {n: x.clone().requires_grad_(n in NAMES) for n, x in d.items()}
        o, last = call(d, lt)
        return o, last, *torch.autograd.grad((o, last), [d[n] for n in NAMES], (d["do"], d["ds"]))
    d = {n: x.to(DEV) for n, x in t.items()}
    want = both(d)
    for key in (0.0, math.inf):
        for b, n in enumerate(lengths):
            for name, x in dict(q=math.inf, k=key, v=-math.inf, do=math.inf, g=math.inf, b=-math.inf).items():
                d[name][b, n:] = x
        assert all(torch.equal(x, y) for x, y in zip(both(d), want))
    assert all(x.isfinite().all() for x in want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_of_sequences_that_lie_apart(layout, dtype):
    """Every other sequence, position or head of a tensor."""
    for dim in (0, 1, 2):
        run(3, 33, (4, 2), 32, 24, layout, "sequence", dtype,
            view=lambda x: x.repeat_interleave(2, dim)[(slice(None),) * dim + (slice(None, None, 2),)])
