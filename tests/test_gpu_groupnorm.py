"""Group norm with an activation against its formula in float64 (numpy).

Bars, with e = 2^-24.  mean is rounded once to float32 (e |mean| rstd in h),
x - mean and the product with rstd each once more; z = h w + b adds two, the
activation about 8 e (1 + |z|) of itself (an exponential or the error
function, and the products around it): |dz| <= e (|w| (6 |h| + 2 |mean| rstd)
+ 4 |b| + 2 |z|), and y within 1.2 |dz| + 16 e (1 + |z|)^2, plus the output's
rounding.  Sums over n values with magnitudes summing to S: float32 partials
of at most 64 rows, then float64: 80 e S.  The gradients' parts are products
of at most eight rounded factors; act' moves by at most its own error and
1.2 |dz|."""
import math

import numpy as np
import pytest
import torch

from semi_markov_crf_zero_amd import encoder

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
E = 2.0 ** -24
erf = np.vectorize(math.erf)


def act(z, name):
    if name == "silu":
        with np.errstate(over="ignore"):
            s = 1 / (1 + np.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        c = 0.5 * (1 + erf(z / math.sqrt(2)))
        return z * c, c + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "relu":
        return np.maximum(z, 0), (z > 0).astype(float)
    return z, np.ones_like(z)


def reference(x, w, b, lengths, G, eps, name, dy=None):
    """Outputs and their bars, without the roundings of the outputs' types."""
    B, T, C = x.shape
    out = {n: np.zeros(x.shape) for n in ("y", "dx")}
    tol = {n: np.zeros(x.shape) for n in ("y", "dx")}
    for n in ("dw", "db"):
        out[n], tol[n] = np.zeros(C), np.zeros(C)
    Cg = C // G
    for i in range(B):
        L = lengths[i]
        if not L:
            continue
        u = x[i, :L].reshape(L, G, Cg)
        mean = u.mean((0, 2), keepdims=True)
        rstd = 1 / np.sqrt(((u - mean) ** 2).mean((0, 2), keepdims=True) + eps)
        h = ((u - mean) * rstd).reshape(L, C)
        z = h * w + b
        off = np.broadcast_to(np.abs(mean) * rstd, u.shape).reshape(L, C)
        dh = E * (6 * np.abs(h) + 2 * off)
        dz_ = np.abs(w) * dh + E * (4 * np.abs(b) + 2 * np.abs(z))
        out["y"][i, :L], slope = act(z, name)
        tol["y"][i, :L] = 1.2 * dz_ + 16 * E * (1 + np.abs(z)) ** 2
        if dy is None:
            continue
        d = dy[i, :L]
        # act' near a kink of relu may go either way: the tests keep away from it
        ds = (0 if name == "none" else 1.2 * dz_ + 24 * E * (1 + np.abs(z)) ** 2)
        if name == "relu":
            ds = 0
        g, gt = d * slope, np.abs(d) * (ds + 2 * E)
        a, at = g * h, gt * np.abs(h) + np.abs(g) * dh + E * np.abs(g * h)
        out["db"] += g.sum(0)
        tol["db"] += gt.sum(0) + 80 * E * np.abs(g).sum(0)
        out["dw"] += a.sum(0)
        tol["dw"] += at.sum(0) + 80 * E * np.abs(a).sum(0)

        def group(v):
            return np.broadcast_to(v.reshape(L, G, Cg).mean((0, 2), keepdims=True),
                                   u.shape).reshape(L, C)
        aw = np.abs(w)
        m1, m2 = group(g * w), group(a * w)
        t1 = group(gt * aw) + 84 * E * group(np.abs(g) * aw)
        t2 = group(at * aw) + 84 * E * group(np.abs(a) * aw)
        r = np.broadcast_to(rstd, u.shape).reshape(L, C)
        out["dx"][i, :L] = r * (g * w - m1 - h * m2)
        tol["dx"][i, :L] = r * (gt * aw + t1 + np.abs(h) * t2 + np.abs(m2) * dh + 6 * E * (
            np.abs(g * w) + np.abs(m1) + np.abs(h * m2)))
    return out, tol


def compare(B, T, C, G, dtype, name="silu", lengths=None, offset=0.0, spread=1.0, affine=True,
            eps=1e-5, seed=0, poison=False):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((B, T, C), generator=gen) * spread + offset).to(TYPES[dtype])
    dy = torch.randn((B, T, C), generator=gen).to(TYPES[dtype])
    w = 1 + 0.3 * torch.randn(C, generator=gen) if affine else None
    b = 0.5 * torch.randn(C, generator=gen) if affine else None
    lens = [T] * B if lengths is None else lengths
    want, tol = reference(x.double().numpy(), w.double().numpy() if affine else np.ones(C),
                          b.double().numpy() if affine else np.zeros(C), lens, G, eps, name,
                          dy.double().numpy())
    xd, dyd = x.to(DEV), dy.to(DEV)
    if poison:
        for i, L in enumerate(lens):
            xd[i, L:] = float("nan")
            dyd[i, L:] = float("nan")
    xd.requires_grad_(True)
    wd, bd_ = (t.to(DEV).requires_grad_(True) if affine else None for t in (w, b))
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    y = encoder.group_norm(xd, G, wd, bd_, lengths=lt, eps=eps, activation=name)
    assert y.dtype == TYPES[dtype]
    grads = torch.autograd.grad(y, [t for t in (xd, wd, bd_) if t is not None], dyd)
    got = dict(zip(("y", "dx", "dw", "db"), (y.detach(), *grads)))
    for n, g in got.items():
        g = g.float().cpu().double().numpy()
        u = ULP[dtype] if n in ("y", "dx") else E
        off = np.abs(g - want[n]) - (tol[n] + u * np.abs(want[n]) + 2.0 ** -25)
        assert np.all(off <= 0), (n, float(np.nanmax(off)), np.argwhere(~(off <= 0))[:4].tolist())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,T,C,G", [(1, 1, 1, 1), (3, 1, 64, 8), (2, 5, 12, 3), (2, 33, 250, 10),
                                     (1, 700, 64, 1), (4, 100, 256, 32), (2, 9, 3, 3),
                                     (1, 17, 1030, 5), (1, 5, 4096, 4), (300, 1, 40, 5),
                                     (1, 3000, 16, 2), (70, 2, 24, 24), (2, 260, 7, 1)])
def test_shapes(B, T, C, G, dtype):
    # a group of one value is h = 0: covered with its rstd of 1/sqrt(eps)
    compare(B, T, C, G, dtype, seed=C + T)


@pytest.mark.parametrize("name", ["none", "silu", "gelu", "relu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_activations(name, dtype):
    compare(3, 50, 48, 6, dtype, name=name, lengths=[50, 31, 7], seed=5)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C,G", [(64, 8), (30, 10), (256, 32)])
def test_ragged_lengths_and_nan_past_them(C, G, dtype):
    compare(6, 150, C, G, dtype, lengths=[150, 0, 1, 64, 149, 2], poison=True, seed=6)


def test_long_and_ragged():
    compare(2, 9000, 32, 4, "f32", lengths=[9000, 4321], seed=7)
    compare(2, 9000, 32, 4, "bf16", lengths=[8999, 17], seed=8)


def test_offsets_and_scales():
    compare(2, 400, 32, 4, "f32", offset=1000.0, seed=9)
    compare(2, 400, 32, 4, "f32", spread=1e-6, eps=1e-12, seed=10)
    compare(2, 400, 32, 4, "f32", spread=1e6, seed=11)
    compare(2, 64, 32, 4, "f32", spread=0.0, offset=3.0, name="none", seed=12)  # constant groups


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_weight_and_bias(dtype):
    compare(2, 40, 24, 3, dtype, affine=False, seed=13)


def test_invalid_lengths():
    x = torch.randn((4, 20, 16), device=DEV).requires_grad_(True)
    w = torch.ones(16, device=DEV).requires_grad_(True)
    lengths = torch.tensor([20, -1, 21, 5], dtype=torch.int32, device=DEV)
    y = encoder.group_norm(x, 4, w, None, lengths=lengths, activation="silu")
    assert y[1:3].isnan().all() and y[[0, 3]].isfinite().all()
    dx, dw = torch.autograd.grad(y, (x, w), torch.ones_like(y))
    assert (dx[1:3] == 0).all() and dx.isfinite().all() and dw.isfinite().all()


def test_many_sequences():
    """More sequences than a grid's second dimension holds, each of one position."""
    x = torch.randn((70001, 1, 8), device=DEV)
    y = encoder.group_norm(x, 2)
    u = x.double().view(-1, 2, 4)
    want = (u - u.mean(2, keepdim=True)) / torch.sqrt(u.var(2, unbiased=False, keepdim=True) + 1e-5)
    # |h| <= sqrt(3) in a group of four; mean and rstd rounded once each
    bound = E * (8 * want.abs() + 4 * u.abs().amax(2, keepdim=True) / torch.sqrt(
        u.var(2, unbiased=False, keepdim=True) + 1e-5))
    assert ((y.double().view_as(u) - want).abs() <= bound + 1e-7 * want.abs()).all()


def test_layouts():
    """Images channels last, a tensor that is not contiguous, an odd start."""
    x = torch.randn((2, 6, 5, 32), device=DEV)
    y = encoder.group_norm(x, 4, activation="gelu")
    assert torch.equal(y, encoder.group_norm(x.view(2, 30, 32), 4, activation="gelu").view_as(x))
    t = torch.randn((2, 32, 30), device=DEV).transpose(1, 2)
    assert torch.equal(encoder.group_norm(t, 4), encoder.group_norm(t.contiguous(), 4))
    for dtype in TYPES.values():
        s = torch.zeros(2 * 30 * 32 + 1, device=DEV, dtype=dtype)[1:].view(2, 30, 32)
        s.copy_(x.view(2, 30, 32))
        a, b = encoder.group_norm(s, 4), encoder.group_norm(x.view(2, 30, 32).to(dtype), 4)
        # another order of the sums: float64, so the statistics agree to a rounding or two
        assert ((a.double() - b.double()).abs() <= (ULP["f32"] if dtype == torch.float32 else
                ULP["bf16" if dtype == torch.bfloat16 else "f16"]) * 4 * (1 + b.double().abs())).all()


def test_gradient_against_differences():
    """Central differences in float64 of the float32 outputs.  With step s the
    truncation is s^2 / 6 times a third derivative, of the order of the loss
    over the spread cubed; the outputs' error e |y| enters divided by s."""
    torch.manual_seed(3)
    x, w, b = (torch.randn(s, device=DEV) for s in ((2, 12, 16), (16,), (16,)))
    dy = torch.randn((2, 12, 16), device=DEV)
    lengths = torch.tensor([12, 7], dtype=torch.int32, device=DEV)

    def loss(x, w, b):
        y = encoder.group_norm(x, 4, w, b, lengths=lengths, activation="silu")
        return float((y.double() * dy.double()).sum())

    t = [v.clone().requires_grad_(True) for v in (x, w, b)]
    grads = torch.autograd.grad(encoder.group_norm(t[0], 4, t[1], t[2], lengths=lengths,
                                                   activation="silu"), t, dy)
    s = 2.0 ** -7
    for i in range(3):
        u = (torch.randint(0, 2, (x, w, b)[i].shape, device=DEV) * 2 - 1).float() * s
        up, down = [x, w, b], [x, w, b]
        up[i], down[i] = up[i] + u, down[i] - u
        num = (loss(*up) - loss(*down)) / (2 * s)
        ana = float((grads[i].double() * u.double()).sum()) / s
        # 304 outputs of size about 1, each within about 32 e, divided by s; third derivatives
        # of each output along u below about 8: 304 * 8 s^2 / 6
        assert abs(num - ana) <= 304 * (32 * E / s + 8 * s * s / 6), i


def test_stream_and_graph():
    x = torch.randn((2, 3000, 64), device=DEV, dtype=torch.bfloat16)
    want = encoder.group_norm(x, 8, activation="silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = encoder.group_norm(x, 8, activation="silu")
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = encoder.group_norm(x, 8, activation="silu")
    for i in range(3):
        x.copy_(torch.randn_like(x))
        want = encoder.group_norm(x, 8, activation="silu")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), i


def test_empty_and_refusals():
    assert encoder.group_norm(torch.zeros((0, 5, 8), device=DEV), 2).shape == (0, 5, 8)
    assert encoder.group_norm(torch.zeros((2, 0, 8), device=DEV), 2).shape == (2, 0, 8)
    x = torch.zeros((2, 5, 8), device=DEV)
    w = torch.ones(8, device=DEV)
    for args, kw in (((x, 3), {}), ((x, 0), {}), ((x.double(), 2), {}), ((x[0, 0], 2), {}),
                     ((x, 2, w[:7]), {}), ((x, 2, w.half()), {}), ((x, 2, w, w.cpu()), {}),
                     ((x, 2), dict(activation="tanh")), ((x, 2), dict(eps=-1.0)),
                     ((x, 2), dict(lengths=torch.zeros(2, device=DEV))),
                     ((x[:, None], 2), dict(lengths=torch.zeros(2, dtype=torch.int32, device=DEV)))):
        with pytest.raises(ValueError):
            encoder.group_norm(*args, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C,G", [(96, 32), (24, 24), (40, 8), (12, 1), (50, 2), (72, 8)])
def test_vectors_that_groups_part(C, G, dtype):
    """Long sequences whose groups are not whole vectors of channels."""
    compare(2, 1500, C, G, dtype, lengths=[1500, 901], poison=True, seed=C)


def test_many_rows_of_partials():
    """Parameters' gradients over more workgroups than one reduction takes."""
    compare(9000, 1, 520, 8, "bf16", name="none", seed=21)


def test_second_derivatives_are_refused():
    """A penalty on a gradient would lack the terms through the operator."""
    x = torch.randn((2, 5, 8), device=DEV, requires_grad=True)
    y = encoder.group_norm(x, 2, activation="silu")
    dx, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.square().sum().backward()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(0, 5, 8), (2, 0, 8)])
def test_empty_calls_carry_gradients(shape, dtype):
    x = torch.zeros(shape, device=DEV, dtype=TYPES[dtype])
    w, b = (torch.ones(8, device=DEV, requires_grad=True) for _ in range(2))
    y = encoder.group_norm(x, 2, w, b, activation="silu")
    assert y.shape == shape and y.dtype == x.dtype
    y.float().sum().backward()
    assert torch.equal(w.grad, torch.zeros_like(w)) and torch.equal(b.grad, torch.zeros_like(b))


@pytest.mark.parametrize("B,T,C,G", [(1, 65536, 16, 1), (1, 30000, 30, 3), (300, 1, 512, 1)])
def test_a_first_element_far_from_the_others(B, T, C, G):
    """The others, 0.02 to 0.025, are less than half of the first one's last
    place: a float32 difference from it would be the same for all of them,
    and move the mean by 0.02 where the deviation is 10^6 / sqrt(n)."""
    x = 0.02 + 0.005 * torch.rand((B, T, C), generator=torch.Generator().manual_seed(4))
    x[:, 0, ::C // G] = 1e6
    want, tol = reference(x.double().numpy(), np.ones(C), np.zeros(C), [T] * B, G, 1e-5, "none")
    y = encoder.group_norm(x.to(DEV), G).cpu().double().numpy()
    assert np.all(np.abs(y - want["y"]) <= tol["y"] + E * np.abs(want["y"]))


@pytest.mark.parametrize("T,C,G", [(900, 64, 8), (2, 64, 8)])
@pytest.mark.parametrize("spread", [1e25, 1e-25])
def test_variances_past_float32(T, C, G, spread):
    compare(2, T, C, G, "f32", name="none", spread=spread, eps=0.0, seed=14)


@pytest.mark.parametrize("B,C,G,dtype,act", [(1 << 20, 64, 4, "f32", "none"),
                                             ((1 << 20) + 3, 32, 4, "bf16", "silu"),
                                             (270001, 4096, 8, "bf16", "none")])
def test_positions_of_the_longest_sequences(B, C, G, dtype, act):
    """A norm of each position by itself for as many positions as the head
    takes, and of wide ones (a workgroup each).  Rows at both ends against
    float64, with the bars of `reference`; the parameters' gradients against
    float64 sums over all of them: 80 e of the magnitudes, and what the parts
    themselves are off by (16 e of each: |h| and |dy| are within about 6)."""
    gen = torch.Generator(device=DEV).manual_seed(C)
    x = torch.randn((B, 1, C), device=DEV, generator=gen, dtype=TYPES[dtype])
    dy = torch.randn((B, 1, C), device=DEV, generator=gen, dtype=TYPES[dtype])
    w, b = 1 + 0.3 * torch.randn((2, C), device=DEV, generator=gen)
    x.requires_grad_(True), w.requires_grad_(True), b.requires_grad_(True)
    y = encoder.group_norm(x, G, w, b, activation=act)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy)
    wn, bn = (t.detach().cpu().double().numpy() for t in (w, b))
    for rows in (slice(0, 300), slice(B - 300, B)):
        xr, dyr = (t.detach()[rows].cpu().double().numpy() for t in (x, dy))
        want, tol = reference(xr, wn, bn, [1] * 300, G, 1e-5, act, dyr)
        for n, got in (("y", y), ("dx", dx)):
            got = got.detach()[rows].cpu().double().numpy()
            assert np.all(np.abs(got - want[n]) <= tol[n] + ULP[dtype] * np.abs(want[n])
                          + 2.0 ** -25), n
    sums = torch.zeros((4, C), dtype=torch.float64, device=DEV)
    for xr, dyr in zip(x.detach().split(1 << 15), dy.split(1 << 15)):
        u = xr.double().view(-1, G, C // G)
        h = ((u - u.mean(2, keepdim=True)) / torch.sqrt(
            u.var(2, unbiased=False, keepdim=True) + 1e-5)).view(-1, C)
        z = h * w.detach().double() + b.detach().double()
        s = torch.sigmoid(z)
        dz = dyr.double().view(-1, C) * (s * (1 + z * (1 - s)) if act == "silu" else 1.0)
        for i, t in enumerate((dz * h, dz)):
            sums[i] += t.sum(0)
            sums[2 + i] += t.abs().sum(0)
    for got, want, size in ((dw, sums[0], sums[2]), (db, sums[1], sums[3])):
        assert ((got.double() - want).abs() <= (80 + 16 * 6) * E * size).all()


def test_sums_over_many_positions():
    """A thread sums 512 positions of dz here.  dy = 1 + 2^-16 - 2^-23: from
    256 on a float32 sum drops 2^-16 of it at every position, 128 e in the end.
    db and mean(d) are within 80 e, and dx = rstd (d - mean(d) - h mean(d h))
    within 96 e rstd of its exact 0 (the sum of h is 0)."""
    T, C, c = 1 << 24, 64, 1 + 2.0 ** -16 - 2.0 ** -23
    x = torch.randn((1, T, C), device=DEV, requires_grad=True)
    b = torch.zeros(C, device=DEV, requires_grad=True)
    dy = torch.full((1, T, C), c, device=DEV)
    dx, db = torch.autograd.grad(encoder.group_norm(x, 8, None, b), (x, b), dy)
    assert ((db.double() / (T * c) - 1).abs() <= 80 * E).all(), db
    # rstd is 1 to 1e-3: 2^24 * 8 values of a variance of 1
    assert float(dx.abs().max()) <= 97 * E


@pytest.mark.parametrize("way", ["backward", "grad"])
def test_second_derivatives_are_refused_beside_others(way):
    """The gradient of a plain sum: what comes in asks for no gradient, and
    the penalty also depends on w by a way that is known."""
    w = torch.full((2, 5, 8), 2.0, device=DEV, requires_grad=True)
    a = torch.randn((2, 5, 8), device=DEV, requires_grad=True)
    y = encoder.group_norm(w * a, 2, activation="silu")
    g, = torch.autograd.grad(y.sum(), a, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        if way == "grad":
            torch.autograd.grad(g.square().sum(), w)
        else:
            g.square().sum().backward()


@pytest.mark.parametrize("shape,dtype", [((2, 3000, 64), "bf16"), ((300, 1, 40), "f32")])
def test_gradients_on_another_stream_and_in_a_graph(shape, dtype):
    x, dy = torch.randn((2, *shape), device=DEV).to(TYPES[dtype]).unbind(0)
    x, dy = x.clone().requires_grad_(True), dy.clone()
    w, b = (torch.randn(shape[2], device=DEV, requires_grad=True) for _ in range(2))

    def call():
        y = encoder.group_norm(x, 8, w, b, activation="silu")
        return (y.detach(), *torch.autograd.grad(y, (x, w, b), dy))
    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, e) for a, e in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(4):
        with torch.no_grad():
            x.copy_(torch.randn_like(x))
            dy.copy_(torch.randn_like(dy))
        want = call()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(got, want)), i
