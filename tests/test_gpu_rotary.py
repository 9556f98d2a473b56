"""Rotary positions against complex products in float64.

Bars: a turned element is f c - g s with c, s within 4 * 2^-24 of the cosine and sine
(half a turn's float32 part, sincospi's own error, the rest of the angle and the scale),
three roundings more: 8 * 2^-24 (|f| + |g|) |scale|, and the output's rounding.  The angle in
float64 is off by 2^-52 of itself, up to 2^21 radians: 2^-31."""
import math

import numpy as np
import pytest
import torch

from semi_markov_crf_zero_amd import encoder

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def reference(x, f, at, layout, scale, inverse=False):
    """x [B, T, heads, D], at [B, T] float64."""
    n = len(f)
    a, b = (np.arange(n), np.arange(n) + n) if layout == "half" else (2 * np.arange(n), 2 * np.arange(n) + 1)
    z = np.exp((-1j if inverse else 1j) * at[..., None] * f)[:, :, None] * scale
    y, size = x.copy(), np.zeros_like(x)
    w = (x[..., a] + 1j * x[..., b]) * z
    y[..., a], y[..., b] = w.real, w.imag
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(scale)
    return y, size


def check(got, want, size, dtype):
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape
    tol = (8 * 2.0 ** -24 + 2.0 ** -31) * size + ULP[dtype] * np.abs(want) + (2.0 ** -25 if dtype == "f16" else 0)
    off = np.abs(got - want)
    assert np.all(off <= tol), (off - tol).max()


def positions_of(kind, B, T, gen):
    if kind == "none":
        return None, np.broadcast_to(np.arange(T, dtype=np.float64), (B, T))
    if kind == "sequence":
        p = torch.randint(-5, 1 << 20, (B,), generator=gen, dtype=torch.int32)
        return p.to(DEV), p.double().numpy()[:, None] + np.arange(T)
    p = torch.randint(-(1 << 20), 1 << 20, (B, T), generator=gen, dtype=torch.int32)
    return p.to(DEV), p.double().numpy()


def run(B, T, heads, D, turn, layout, kind, dtype, scale=1.0, view=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = [torch.randn((B, T, h, D), generator=gen).to(TYPES[dtype]) for h in heads]
    d = [torch.randn((B, T, h, D), generator=gen).to(TYPES[dtype]) for h in heads]
    f = encoder.rotary_frequencies(turn, device=DEV)
    p, at = positions_of(kind, B, T, gen)
    dev = [t.to(DEV) if view is None else view(t.to(DEV)) for t in x]
    for t in dev:
        t.requires_grad_(True)
    out = encoder.rotary(dev[0], dev[1] if len(dev) > 1 else None, f, positions=p, layout=layout, scale=scale)
    out = out if len(dev) > 1 else (out,)
    grads = torch.autograd.grad(out, dev, [t.to(DEV) for t in d])
    for y, g, a, b in zip(out, grads, x, d):
        assert y.is_contiguous() and y.dtype == TYPES[dtype]
        check(y, *reference(a.double().numpy(), f.cpu().numpy(), at, layout, scale), dtype)
        check(g, *reference(b.double().numpy(), f.cpu().numpy(), at, layout, scale, True), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,turn", [(64, 64), (64, 32), (40, 36), (72, 72), (128, 128), (2, 2), (7, 6), (33, 2),
                                    (10, 4), (256, 100)])
def test_widths(D, turn, layout, dtype):
    run(2, 50, (4, 2), D, turn, layout, "none", dtype)


@pytest.mark.parametrize("kind", ["none", "sequence", "each"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (1, 1000), (5, 77), (300, 1)])
def test_positions(B, T, layout, kind):
    run(B, T, (2, 1), 32, 32, layout, kind, "f32", scale=1.25)


@pytest.mark.parametrize("heads", [(1,), (5,), (3, 7), (16, 16), (1, 130)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_heads(heads, dtype):
    run(2, 9, heads, 16, 16, "half", "sequence", dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_views(layout, dtype):
    def odd(x):
        y = torch.zeros((*x.shape[:-1], x.shape[-1] + 3), dtype=x.dtype, device=DEV)
        y[..., 1:-2] = x
        return y[..., 1:-2]

    def heads_first(x):
        return x.transpose(1, 2).contiguous().transpose(1, 2)

    def by_element(x):
        return x.transpose(1, 3).contiguous().transpose(1, 3)

    def reversed_batch(x):
        return x.flip(0).as_strided(x.shape, x.stride()) if x.shape[0] == 1 else x.repeat(2, 1, 1, 1)[::2]
    for view in (odd, heads_first, by_element):
        run(2, 33, (4, 2), 32, 24, layout, "sequence", dtype, view=view)


def test_widest_row():
    run(1, 3, (1, 1), 8192, 8192, "half", "sequence", "f32")
    run(1, 3, (1, 1), 8192, 8190, "interleaved", "none", "bf16")


@pytest.mark.parametrize("scaling", ["linear", "base", "bands"])
def test_stretched_frequencies(scaling):
    plain = encoder.rotary_frequencies(32)
    f = encoder.rotary_frequencies(32, stretch=8.0, scaling=scaling)
    assert f.dtype == torch.float64 and f.shape == (16,)
    share = (plain / f).numpy()
    if scaling == "linear":
        np.testing.assert_allclose(share, 8.0, rtol=1e-12)
    else:
        assert share[0] == pytest.approx(1.0) and share[-1] == pytest.approx(8.0, rel=1e-9)
        assert np.all(np.diff(share) > -1e-9)


def test_scores_depend_on_distances():
    """Turned queries and keys have the products of their distance."""
    gen = torch.Generator().manual_seed(3)
    q, k = (torch.randn((1, 1, 1, 64), generator=gen).to(DEV) for _ in range(2))
    f = encoder.rotary_frequencies(64, device=DEV)
    at = lambda p: torch.tensor([p], dtype=torch.int32, device=DEV)  # noqa: E731
    score = lambda i, j: float((encoder.rotary(q, None, f, at(i)) * encoder.rotary(k, None, f, at(j))).sum())  # noqa: E731
    for i in (0, 17, 1000, 1 << 20):
        assert score(i + 9, i) == pytest.approx(score(9, 0), abs=64 * 16 * 2.0 ** -24 * 64)


def test_single_positions():
    gen = torch.Generator().manual_seed(4)
    q, k = (torch.randn((6, h, 32), generator=gen).to(DEV) for h in (4, 2))
    p = torch.tensor([5, 0, 1 << 20, 77, 3, -2], dtype=torch.int32, device=DEV)
    f = encoder.rotary_frequencies(32, device=DEV)
    one = encoder.rotary(q, k, f, positions=p)
    whole = encoder.rotary(q[:, None], k[:, None], f, positions=p[:, None].contiguous())
    for x, y in zip(one, whole):
        assert torch.equal(x, y[:, 0])
    assert torch.equal(encoder.rotary(q, None, f, positions=p), one[0])


def test_empty_calls():
    f = encoder.rotary_frequencies(8, device=DEV)
    for shape in ((0, 3, 2, 8), (2, 0, 2, 8), (2, 3, 0, 8)):
        q = torch.zeros(shape, device=DEV, requires_grad=True)
        y, z = encoder.rotary(q, q, f)
        assert y.shape == shape and z.shape == shape
        (y.sum() + z.sum()).backward()
    q, k = torch.zeros((2, 3, 0, 8), device=DEV), torch.randn((2, 3, 2, 8), device=DEV)
    assert torch.equal(encoder.rotary(q, k, f)[1], encoder.rotary(k, None, f))
    assert torch.equal(encoder.rotary(k, q, f)[0], encoder.rotary(k, None, f))


def test_padding_is_turned_alone():
    """NaN in one row stays in it."""
    x = torch.randn((1, 40, 2, 16), device=DEV)
    f = encoder.rotary_frequencies(16, device=DEV)
    want = encoder.rotary(x, None, f)
    x[0, 30:] = math.nan
    got = encoder.rotary(x, None, f)
    assert torch.equal(got[:, :30], want[:, :30]) and got[:, 30:].isnan().all()


def test_other_stream_and_graph():
    q, k = (torch.randn((2, 100, 2, 64), device=DEV, dtype=torch.bfloat16) for _ in range(2))
    f = encoder.rotary_frequencies(64, device=DEV)
    p = torch.tensor([3, 9], dtype=torch.int32, device=DEV)
    want = encoder.rotary(q, k, f, positions=p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = encoder.rotary(q, k, f, positions=p)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = encoder.rotary(q, k, f, positions=p)
    for i in range(3):
        q.copy_(torch.randn_like(q))
        p.add_(100)
        want = encoder.rotary(q, k, f, positions=p)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), i


def test_offsets_past_32_bits():
    far = (1 << 32) + 64
    big = torch.empty(far + 70 * 2 * 16, dtype=torch.bfloat16, device=DEV)
    x = big.as_strided((2, 70, 2, 16), (far, 32, 16, 1))
    x.copy_(torch.randn((2, 70, 2, 16), device=DEV))
    f = encoder.rotary_frequencies(16, device=DEV)
    assert torch.equal(encoder.rotary(x, None, f), encoder.rotary(x.contiguous(), None, f))
    del big, x
    torch.cuda.empty_cache()


def test_second_derivatives_are_refused():
    x = torch.randn((1, 4, 1, 8), device=DEV, requires_grad=True)
    y = encoder.rotary(x, None, encoder.rotary_frequencies(8, device=DEV))
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.square().sum().backward()


def test_refusals():
    q, k = torch.zeros((2, 5, 2, 8), device=DEV), torch.zeros((2, 5, 1, 8), device=DEV)
    f = encoder.rotary_frequencies(8, device=DEV)
    at = torch.zeros(2, dtype=torch.int32, device=DEV)
    for args, kw in (((q, k[:, :4], f), {}), ((q, k.half(), f), {}), ((q, k[..., :6], f), {}),
                     ((q, k, f.float()), {}), ((q, k, f.cpu()), {}), ((q[..., :6], k[..., :6], f), {}),
                     ((q, k, f), dict(layout="other")), ((q, k, f), dict(positions=at.long())),
                     ((q, k, f), dict(positions=at[:1])), ((q[:, 0], k[:, 0], f), {}), ((q[0, 0], None, f), {}),
                     ((q, k, f.clone().requires_grad_(True)), {}), ((q.double(), None, f), {})):
        with pytest.raises(ValueError):
            encoder.rotary(*args, **kw)
