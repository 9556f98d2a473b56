"""The norm of many gradients and clipping against float64.

Bars: the sum is in float64 (n 2^-53), the norm is rounded once: 2^-23 of it.  A clipped
element is the product with the float32 coefficient (off by 2^-24 for its rounding and 2^-23
for the norm's), rounded to float32 and to its type."""
import math

import pytest
import torch

from semi_markov_crf_zero_amd import optim

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
INF = math.inf


def params(sizes, dtypes, scale=1.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        p = torch.zeros(n, dtype=dtypes[i % len(dtypes)], device=DEV, requires_grad=True)
        p.grad = (torch.randn(n, generator=gen) * scale).to(p.dtype).to(DEV)
        out.append(p)
    return out


def norm_of(ps, order):
    g = torch.cat([p.grad.double().flatten() for p in ps if p.grad is not None])
    return float(torch.linalg.vector_norm(g, order)) if g.numel() else 0.0


def compare(ps, order, max_norm):
    want = norm_of(ps, order)
    before = [None if p.grad is None else p.grad.clone() for p in ps]
    norm = optim.grad_norm(ps, norm_type=order)
    assert norm.shape == () and norm.dtype == torch.float32
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    both = optim.grad_norm(ps, max_norm=max_norm, norm_type=order)
    c = min(1.0, max_norm / (want + 1e-6))
    assert float(both[0]) == float(norm) and abs(float(both[1]) - c) <= 2.0 ** -22 * c
    got = optim.clip_grad_norm_(ps, max_norm, norm_type=order)
    assert float(got) == float(norm)
    for p, b in zip(ps, before):
        if b is None:
            assert p.grad is None
            continue
        x = b.double() * c
        tiny = 2.0 ** -25 if p.dtype == torch.float16 else 2.0 ** -149
        assert ((p.grad.double() - x).abs() <= (2.0 ** -22 + ULP[p.dtype]) * x.abs() + tiny).all()
        if max_norm > want * 1.001:
            assert torch.equal(p.grad, b)


@pytest.mark.parametrize("order", [2.0, 1.0, INF])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes", [[1], [7], [4095], [4096], [4097], [100000], [0, 5, 0], [3, 8192, 1, 12289, 64]])
def test_sizes(sizes, dtype, order):
    compare(params(sizes, [dtype]), order, 0.5)


@pytest.mark.parametrize("order", [2.0, INF])
@pytest.mark.parametrize("max_norm", [0.0, 1e-3, 1.0, 1e9])
def test_coefficients(max_norm, order):
    compare(params([1000, 33], [torch.float32, torch.bfloat16]), order, max_norm)


@pytest.mark.parametrize("order", [2.0, 1.0, INF])
@pytest.mark.parametrize("count", [2, 255, 256, 257, 700])
def test_many_tensors_of_several_types(count, order):
    """More than one launch's."""
    gen = torch.Generator().manual_seed(count)
    sizes = torch.randint(0, 9000, (count,), generator=gen).tolist()
    compare(params(sizes, [torch.float32, torch.bfloat16, torch.float16]), order, 2.0)


def test_more_blocks_than_workgroups():
    compare(params([20_000_003, 5], [torch.float32]), 2.0, 1.0)
    compare(params([30_000_001], [torch.bfloat16]), INF, 1.0)


@pytest.mark.parametrize("scale", [1e-30, 1e25, 1e30])
def test_magnitudes_whose_squares_leave_float32(scale):
    ps = params([5000, 77], [torch.float32], scale)
    compare(ps, 2.0, scale)


@pytest.mark.parametrize("order", [2.0, 1.0, INF])
def test_nan_and_infinity(order):
    ps = params([5000, 77], [torch.float32])
    ps[1].grad[3] = math.nan
    ps[0].grad[9] = math.inf
    norm, c = optim.grad_norm(ps, max_norm=1.0, norm_type=order)
    assert math.isnan(norm) and math.isnan(c)
    ps[1].grad[3] = -math.inf
    norm, c = optim.grad_norm(ps, max_norm=1.0, norm_type=order)
    assert float(norm) == math.inf and float(c) == 0.0
    optim.clip_grad_norm_(ps, 1.0, norm_type=order)
    assert ps[0].grad[9].isnan() and ps[0].grad[8] == 0


def test_unaligned_and_missing_gradients():
    flat = torch.randn(20011, device=DEV)
    for dtype in ULP:
        ps = []
        for a, b in ((1, 5000), (5001, 5004), (5007, 20011)):
            p = torch.zeros(b - a, dtype=dtype, device=DEV, requires_grad=True)
            p.grad = flat.to(dtype)[a:b]
            ps.append(p)
        ps.insert(1, torch.zeros(5, device=DEV, requires_grad=True))
        compare(ps, 2.0, 1.0)


def test_neighbours_are_left_alone():
    flat = torch.randn(9001, device=DEV)
    before = flat.clone()
    p = torch.zeros(4103, device=DEV, requires_grad=True)
    p.grad = flat[3:4106]
    optim.clip_grad_norm_([p], 1e-3)
    assert torch.equal(flat[:3], before[:3]) and torch.equal(flat[4106:], before[4106:])


def test_gradients_that_are_not_contiguous():
    p = torch.zeros((30, 50), device=DEV, requires_grad=True)
    p.grad = torch.randn((50, 30), device=DEV).t()
    q = torch.zeros((4, 6), device=DEV, requires_grad=True)
    q.grad = torch.randn((8, 6), device=DEV)[::2]
    compare([p, q], 2.0, 1.0)


def test_no_gradients():
    p = torch.zeros(4, device=DEV, requires_grad=True)
    assert float(optim.grad_norm([p])) == 0.0 and float(optim.clip_grad_norm_([p], 1.0)) == 0.0
    p.grad = torch.zeros(4, device=DEV)
    assert float(optim.clip_grad_norm_(p, 1.0)) == 0.0 and not p.grad.any()
    e = torch.zeros(0, device=DEV, requires_grad=True)
    e.grad = torch.zeros(0, device=DEV)
    norm, c = optim.grad_norm([e], max_norm=1.0)
    assert float(norm) == 0.0 and float(c) == 1.0
    assert float(optim.clip_grad_norm_([e], 1.0)) == 0.0


def test_shared_memory_is_refused():
    p, q = (torch.zeros(100, device=DEV, requires_grad=True) for _ in range(2))
    flat = torch.ones(150, device=DEV)
    p.grad, q.grad = flat[:100], flat[50:]
    with pytest.raises(ValueError, match="twice"):
        optim.clip_grad_norm_([p, q], 1.0)
    with pytest.raises(ValueError, match="twice"):
        optim.clip_grad_norm_([p, p], 1.0)
    w = torch.zeros((4, 4), device=DEV, requires_grad=True)
    w.grad = torch.ones((1, 4), device=DEV).expand(4, 4)
    with pytest.raises(ValueError, match="twice"):
        optim.clip_grad_norm_([w], 1.0)
    assert (flat == 1).all() and (w.grad == 1).all()
    assert float(optim.grad_norm([p, q])) == pytest.approx(math.sqrt(200))


def test_the_step_takes_the_coefficient():
    """Clipping in place and the coefficient alone move the parameters alike: a coefficient that is a
    power of two, and a norm of gradients of powers of two."""
    def make():
        p = torch.linspace(-1, 1, 64, device=DEV).requires_grad_(True)
        p.grad = torch.full((64,), 0.5, device=DEV)
        return p, optim.AdamW([p], lr=0.1)
    a, first = make()
    b, second = make()
    c = optim.grad_norm([b], max_norm=1.0)[1]
    optim.clip_grad_norm_([a], 1.0)
    first.step()
    second.step(grad_scale=c)
    assert torch.equal(a, b)


def test_other_stream_and_graph():
    ps = params([5000, 3, 77777], [torch.float32, torch.bfloat16])
    want = optim.grad_norm(ps)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = optim.grad_norm(ps)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    keep = [p.grad.clone() for p in ps]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = optim.clip_grad_norm_(ps, 1.0)
    held = [p.grad for p in ps]
    for i in range(3):
        fresh = [torch.randn_like(k) * (i + 1) for k in keep]
        for h, f in zip(held, fresh):
            h.copy_(f)
        others = [torch.zeros_like(f, requires_grad=True) for f in fresh]
        for p, f in zip(others, fresh):
            p.grad = f
        want = optim.clip_grad_norm_(others, 1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all(torch.equal(h, f) for h, f in zip(held, fresh)), i


def test_clipping_is_seen_by_autograd():
    p = torch.ones(4, device=DEV, requires_grad=True)
    p.grad = torch.ones(4, device=DEV)
    w = torch.ones(4, device=DEV, requires_grad=True)
    y = (w * p.grad).sum()
    optim.clip_grad_norm_([p], 0.5)
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.backward()


def test_refusals():
    p = torch.zeros(4, device=DEV, requires_grad=True, dtype=torch.float64)
    p.grad = torch.zeros(4, device=DEV, dtype=torch.float64)
    q = torch.zeros(4, device=DEV, requires_grad=True)
    q.grad = torch.zeros(4, device=DEV)
    cpu = torch.zeros(4, requires_grad=True)
    cpu.grad = torch.zeros(4)
    for params in ([p], [q, p], [q, cpu]):
        with pytest.raises(ValueError):
            optim.grad_norm(params)
    with pytest.raises(ValueError):
        optim.grad_norm([q], norm_type=0.5)
