"""The AdamW step against its definition.

The header gives every operation and its rounding to float32, so the states
and float32 parameters are compared bit by bit with numpy's float32
operations in that order, and the 8-bit codes with a search over the 256
values.  Against the formula in float64: m and v are sums of two products
(4 e |terms|), the update a quotient of them (12 e of itself), e = 2^-24."""
import copy
import math

import numpy as np
import pytest
import torch

from semi_markov_crf_zero_amd import optim

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F = np.float32
E = 2.0 ** -24
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.98, eps=1e-8, weight_decay=0.1)

# magnitudes of the 8-bit forms, in order of their codes
SIGNED = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                   for e in range(16) for m in range(8)][:127])
ROOT = np.array([(m / 16 if e == 0 else 1 + m / 16) * 2.0 ** (max(e, 1) - 7)
                 for e in range(16) for m in range(16)])


def nearest(x, table):
    """Code of the nearest value, ties to the even code."""
    i = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo, hi = x - table[i - 1], table[i] - x
    return np.where((lo < hi) | ((lo == hi) & (i % 2 == 1)), i - 1, i)


def blocks(x):
    n = -(-len(x) // 256) * 256
    return np.concatenate([x, np.zeros(n - len(x), x.dtype)]).reshape(-1, 256)


def encode(x, table, most):
    n = len(x)
    x = blocks(x)
    top = np.abs(x).max(1, keepdims=True).astype(F)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.where(top > F(2.0 ** -100), (F(1) / top) * F(most), F(0)).astype(F)
    y = (x * inv).astype(F)
    code = nearest(np.abs(y).astype(np.float64), table)
    return code.reshape(-1)[:n], np.signbit(y).reshape(-1)[:n], (top * F(1 / most)).reshape(-1).astype(F)


def decode8(code, neg, scale, table):
    x = blocks(np.where(neg, -table[code], table[code]).astype(F)) * scale[:, None]
    return x.astype(F).reshape(-1)[:len(code)]


def step(p, g, m, v, t, hy, gs=None):
    """One step in float32, each operation by itself."""
    b1, b2 = hy["beta1"], hy["beta2"]
    g = g.astype(F)
    if gs is not None:
        g = g * F(gs)
    m = m * F(b1) + F(1 - b1) * g
    v = v * F(b2) + (F(1 - b2) * g) * g
    root = np.sqrt(v)
    down = root * F(1 / math.sqrt(1 - b2 ** t)) + F(hy["eps"])
    p = p * F(1 - hy["lr"] * hy["weight_decay"]) - (m / down) * F(hy["lr"] / (1 - b1 ** t))
    return p.astype(F), m.astype(F), v.astype(F), root.astype(F)


def tensors(seed, sizes, dtype, grad, offset=0):
    """Parameters and gradients, each `offset` elements past an aligned start."""
    gen = torch.Generator().manual_seed(seed)

    def one(n, dt, std):
        t = (torch.randn(n, generator=gen) * std).to(dt)
        d = torch.zeros(n + offset, dtype=dt, device=DEV)[offset:]
        d.copy_(t)
        return d
    return [one(n, TYPES[dtype], 0.5) for n in sizes], [one(n, TYPES[grad], 0.01) for n in sizes]


def host(ts):
    return [t.detach().float().cpu().numpy() for t in ts]


SIZES = [1, 3, 255, 256, 257, 4095, 4096, 4097, 0, 20000, 64]


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"),
                                        ("bf16", "f32"), ("f16", "f16")])
def test_states_in_32_bits(dtype, grad, offset):
    p, g = tensors(1, SIZES, dtype, grad, offset)
    plan = optim.AdamWPlan(p)
    P, G = host(p), host(g)
    M, V = [np.zeros(n, F) for n in SIZES], [np.zeros(n, F) for n in SIZES]
    for t in range(1, 4):
        plan.run(g, t, **HYPER)
        for i in range(len(SIZES)):
            P[i], M[i], V[i], _ = step(P[i], G[i], M[i], V[i], t, HYPER)
            if dtype != "f32":
                P[i] = torch.from_numpy(P[i]).to(TYPES[dtype]).float().numpy()
        for got, want in ((host(p), P), (host(plan.exp_avg), M), (host(plan.exp_avg_sq), V)):
            for a, b in zip(got, want):
                assert np.array_equal(a, b), t


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_states_in_8_bits(dtype, grad, offset):
    p, g = tensors(2, SIZES, dtype, grad, offset)
    plan = optim.AdamWPlan(p, bits=8)
    P, G = host(p), host(g)
    M, V = [np.zeros(n, F) for n in SIZES], [np.zeros(n, F) for n in SIZES]
    for t in range(1, 5):
        plan.run(g, t, **HYPER)
        for i, n in enumerate(SIZES):
            if not n:
                continue
            P[i], m, _, root = step(P[i], G[i], M[i], V[i], t, HYPER)
            if dtype != "f32":
                P[i] = torch.from_numpy(P[i]).to(TYPES[dtype]).float().numpy()
            cm, neg, sm = encode(m, SIGNED, 448)
            cr, _, sr = encode(root, ROOT, 496)
            M[i] = decode8(cm, neg, sm, SIGNED)
            r = decode8(cr, np.zeros(n, bool), sr, ROOT)
            V[i] = (r * r).astype(F)
            (gm, gsm), (gr, gsr) = plan.exp_avg[i], plan.exp_avg_sq[i]
            raw = gm.view(torch.uint8).cpu().numpy()
            assert np.array_equal(raw & 127, cm) and np.array_equal(raw >> 7, neg), (t, n)
            assert np.array_equal(gr.cpu().numpy(), cr), (t, n)
            assert np.array_equal(gsm.cpu().numpy(), sm) and np.array_equal(gsr.cpu().numpy(), sr)
            assert np.array_equal(optim.moment_values(gm, gsm).cpu().numpy(), M[i])
            assert np.array_equal(optim.moment_values(gr, gsr).cpu().numpy(), V[i])
            assert np.array_equal(host(p[i:i + 1])[0], P[i]), (t, n)


def test_against_the_formula_in_64_bits():
    p, g = tensors(3, [10000], "f32", "f32")
    plan = optim.AdamWPlan(p)
    x, gg = host(p)[0].astype(np.float64), host(g)[0].astype(np.float64)
    m = v = 0.0
    for t in range(1, 6):
        plan.run(g, t, **HYPER)
        m = 0.9 * m + 0.1 * gg
        v = 0.98 * v + 0.02 * gg * gg
        up = HYPER["lr"] * (m / (1 - 0.9 ** t)) / (np.sqrt(v / (1 - 0.98 ** t)) + 1e-8)
        x = x * (1 - HYPER["lr"] * 0.1) - up
        # gradients of one sign in every step: no cancellation in m
        assert np.all(np.abs(host(plan.exp_avg)[0] - m) <= 5 * t * E * np.abs(m))
        assert np.all(np.abs(host(plan.exp_avg_sq)[0] - v) <= 6 * t * E * v)
        assert np.all(np.abs(host(p)[0] - x) <= t * E * (4 * np.abs(x) + 40 * np.abs(up) + 0.02))


def test_masters_scale_and_missing_gradients():
    p, g = tensors(4, [500, 300, 700], "bf16", "bf16")
    masters = [t.float() + 1e-4 for t in p]
    plan = optim.AdamWPlan(p, masters=masters)
    P, G, W = host(p), host(g), host(masters)
    scale = torch.tensor([0.37], device=DEV)
    plan.run([g[0], None, g[2]], 1, grad_scale=scale, **HYPER)
    for i in (0, 2):
        W[i], m, v, _ = step(W[i], G[i], np.zeros_like(W[i]), np.zeros_like(W[i]), 1, HYPER, 0.37)
        assert np.array_equal(host(masters)[i], W[i])
        assert np.array_equal(host(p)[i], torch.from_numpy(W[i]).bfloat16().float().numpy())
        assert np.array_equal(host(plan.exp_avg)[i], m)
    assert np.array_equal(host(p)[1], P[1]) and not host(plan.exp_avg)[1].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """More than one launch holds."""
    sizes = [1 + (i * 37) % 600 for i in range(1000)]
    p, g = tensors(5, sizes, "f32", "f32")
    plan = optim.AdamWPlan(p, bits=bits)
    P, G = host(p), host(g)
    g[417] = None
    plan.run(g, 1, **HYPER)
    for i in range(1000):
        if i != 417:
            P[i] = step(P[i], G[i], np.zeros(sizes[i], F), np.zeros(sizes[i], F), 1, HYPER)[0]
    for a, b in zip(host(p), P):
        assert np.array_equal(a, b)


def test_non_finite_gradients_stay_where_they_are():
    for bits in (32, 8):
        p, g = tensors(6, [1024], "f32", "f32")
        plan = optim.AdamWPlan(p, bits=bits)
        g[0][300], g[0][800] = float("nan"), float("inf")
        plan.run(g, 1, **HYPER)
        bad = ~host(p)[0].astype(np.float64).__abs__().__lt__(1e30)
        assert bad[300] and bad[800] and bad.sum() == 2
        m = plan.exp_avg[0] if bits == 32 else optim.moment_values(*plan.exp_avg[0])
        fine = np.isfinite(host([m])[0])
        if bits == 32:
            assert fine.sum() == 1022
        else:  # their blocks of 256 and no others
            assert fine[:256].all() and fine[512:768].all()
            assert not fine[256:512].any() and not fine[800]


def test_states_that_decay_to_nothing():
    """Blocks whose moments pass below 2^-100 hold zeros, not NaN."""
    p, g = tensors(7, [512], "f32", "f32")
    plan = optim.AdamWPlan(p, bits=8)
    plan.run(g, 1, **HYPER)
    zero = [torch.zeros_like(g[0])]
    for t in range(2, 1500):
        plan.run(zero, t, lr=0.0, beta1=0.9, beta2=0.9, eps=1e-8, weight_decay=0.0)
    m, v = optim.moment_values(*plan.exp_avg[0]), optim.moment_values(*plan.exp_avg_sq[0])
    assert (m == 0).all() and plan.exp_avg[0][1].isfinite().all()
    # v stops at float32's last subnormals (0.9 times 4 of them rounds to 4),
    # whose root is far above 2^-100
    assert (v >= 0).all() and (v <= 16 * 2.0 ** -149).all()


def test_optimizer_matches_torch_and_resumes():
    """AdamW as a torch optimizer: torch's own AdamW on the same gradients
    (the same formula in another order: 64 e of the parameter and the moves)."""
    torch.manual_seed(0)
    net = torch.nn.Sequential(torch.nn.Linear(33, 65), torch.nn.Linear(65, 7)).to(DEV)
    other = torch.nn.Sequential(torch.nn.Linear(33, 65), torch.nn.Linear(65, 7)).to(DEV)
    other.load_state_dict(net.state_dict())
    kw = dict(lr=1e-2, betas=(0.9, 0.98), weight_decay=0.05)
    a, b = optim.AdamW(net.parameters(), **kw), torch.optim.AdamW(other.parameters(), **kw)
    for i in range(5):
        for x, y in zip(net.parameters(), other.parameters()):
            x.grad = torch.randn_like(x)
            y.grad = x.grad.clone()
        a.step()
        b.step()
    for x, y in zip(net.parameters(), other.parameters()):
        assert ((x - y).abs() <= 64 * E * (y.abs() + 5e-2)).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_state_dict(bits):
    def make():
        torch.manual_seed(1)
        net = torch.nn.Linear(40, 30).to(DEV).bfloat16()
        return net, optim.AdamW(net.parameters(), lr=1e-2, bits=bits, masters=True)

    def steps(net, opt, lo, hi):
        for i in range(lo, hi):
            gen = torch.Generator(device=DEV).manual_seed(i)
            for p in net.parameters():
                p.grad = torch.randn(p.shape, device=DEV, generator=gen).bfloat16()
            opt.step()

    net, opt = make()
    steps(net, opt, 0, 3)
    saved = [t.clone() for t in net.parameters()], opt.state_dict()
    saved = (saved[0], {"state": {k: {n: t.clone() if isinstance(t, torch.Tensor) else t
                                      for n, t in s.items()} for k, s in saved[1]["state"].items()},
                        "param_groups": saved[1]["param_groups"]})
    steps(net, opt, 3, 6)
    net2, opt2 = make()
    with torch.no_grad():
        for p, t in zip(net2.parameters(), saved[0]):
            p.copy_(t)
    opt2.load_state_dict(saved[1])
    steps(net2, opt2, 3, 6)
    for x, y in zip(net.parameters(), net2.parameters()):
        assert torch.equal(x, y)


def test_refusals():
    p = torch.zeros(10, device=DEV)
    for args, kw in ((([p.double()],), {}), (([p[::2]],), {}), (([p],), dict(bits=16)),
                     (([p],), dict(exp_avg=[])), (([p],), dict(exp_avg=[p[:9]])),
                     (([p],), dict(masters=[p.half()])),
                     (([p],), dict(bits=8, exp_avg=[(p.to(torch.uint8), p[:1])])),
                     (([p],), dict(bits=8, exp_avg_sq=[(p.to(torch.uint8), p[:2])]))):
        with pytest.raises(ValueError):
            optim.AdamWPlan(*args, **kw)
    plan = optim.AdamWPlan([p])
    for grads, kw in (([], {}), ([p[:9]], {}), ([p.double()], {}), ([p.cpu()], {}),
                      ([torch.zeros(20, device=DEV)[::2]], {}), ([p], dict(grad_scale=p))):
        with pytest.raises(ValueError):
            plan.run(grads, 1, **kw)
    with pytest.raises(RuntimeError):
        plan.run([p], 0)
    with pytest.raises(ValueError):
        optim.moment_values(torch.zeros(300, dtype=torch.uint8, device=DEV), p[:1])
    with pytest.raises(ValueError):
        optim.moment_values(p, p[:1])


def test_a_step_is_seen_by_autograd():
    """A backward pass over weights that a step has moved since must not run;
    one over weights without a gradient may."""
    a, b = (torch.nn.Parameter(torch.ones(4, device=DEV)) for _ in range(2))
    opt = optim.AdamW([a, b])
    x = torch.ones(4, device=DEV, requires_grad=True)
    over_a, over_b = (x * a).sum(), (x * b).sum()
    a.grad = torch.ones_like(a)
    opt.step()
    over_b.backward()
    with pytest.raises(RuntimeError, match="inplace operation"):
        over_a.backward()


def test_a_parameter_twice():
    p = torch.ones(300, device=DEV)
    with pytest.raises(ValueError, match="twice"):
        optim.AdamWPlan([p, p.view(30, 10)])
    optim.AdamWPlan([p, torch.empty(0, device=DEV), torch.empty(0, device=DEV)])


@pytest.mark.parametrize("bits", [32, 8])
def test_a_copied_optimizer_steps(bits):
    """A deep copy of a model's parameters with their optimizer goes on as
    the original does."""
    p = torch.nn.Parameter(torch.linspace(-1, 1, 300, device=DEV))
    opt = optim.AdamW([p], bits=bits)
    p.grad = torch.linspace(2, -1, 300, device=DEV)
    opt.step()
    other = copy.deepcopy(opt)
    twin, = other.param_groups[0]["params"]
    assert twin.data_ptr() != p.data_ptr()
    twin.grad = p.grad.clone()
    opt.step()
    after = p.detach().clone()
    other.step()
    assert torch.equal(twin, after) and torch.equal(p, after)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_parameter_that_changes_its_layout(bits):
    """The same storage in another order, type or size is another parameter."""
    hy = dict(lr=1e-2, weight_decay=0.0, bits=bits)
    p = torch.nn.Parameter(torch.linspace(-1, 1, 300, device=DEV).view(15, 20))
    opt = optim.AdamW([p], **hy)
    p.grad = torch.linspace(-2, 1, 300, device=DEV).view(15, 20)
    opt.step()
    before = p.detach().clone()
    p.data = p.data.t()
    p.grad = torch.ones_like(p)
    with pytest.raises(ValueError, match="contiguous"):
        opt.step()
    assert torch.equal(p.detach().t(), before)
    # contiguous again: goes on, from the states of its elements in their order
    p.data = p.data.t()
    p.grad = torch.ones_like(p)
    opt.step()
    assert not torch.equal(p, before) and p.isfinite().all()
    # another shape of the same elements is the same parameter
    p.data = p.data.view(10, 30)
    p.grad = torch.ones_like(p)
    opt.step()

    q = torch.nn.Parameter(torch.ones(256, device=DEV, dtype=torch.bfloat16))
    opt = optim.AdamW([q], **hy)
    q.grad = torch.ones_like(q)
    opt.step()
    q.data = q.data.view(torch.float16)  # the bits of 1 - 0.01 in bfloat16
    start = q.detach().clone()
    q.grad = torch.ones_like(q)
    opt.step()
    # a step with one sign moves a float16 by its learning rate, 1e-2, up to
    # the roundings of float16 near 2 and of the 8-bit states (2^-4)
    assert ((start - q).float() - 1e-2).abs().max() <= 2.0 ** -10 + 1e-2 * 2.0 ** -3


def test_a_refused_step_does_not_count():
    """What goes on after a refusal goes on as if it had not been tried."""
    def make():
        p = torch.nn.Parameter(torch.linspace(-1, 1, 300, device=DEV))
        p.grad = torch.linspace(2, -1, 300, device=DEV)
        return p, optim.AdamW([p], lr=1e-2)
    (p, opt), (q, other) = make(), make()
    opt.step()
    other.step()
    with pytest.raises(ValueError, match="grad_scale"):
        opt.step(grad_scale=torch.ones(2, device=DEV))
    assert opt.state[p]["step"] == 1
    opt.step()
    other.step()
    assert opt.state[p]["step"] == 2 and torch.equal(p, q)


def test_parameters_that_overlap():
    """A part of a parameter beside it; neighbours in one buffer are two."""
    flat = torch.ones(512, device=DEV)
    for params in ([flat, flat[256:]], [flat[100:], flat[:101]], [flat, flat[3:4]],
                   [flat.view(torch.bfloat16)[:600], flat[299:]]):
        with pytest.raises(ValueError, match="twice"):
            optim.AdamWPlan(params)
    a, b, m = torch.zeros((3, 64), device=DEV)
    for kw in (dict(exp_avg=[m, m]), dict(exp_avg=[m, a], exp_avg_sq=[torch.zeros_like(m), m])):
        with pytest.raises(ValueError, match="state"):
            optim.AdamWPlan([a, b], **kw)
    optim.AdamWPlan([a, b], masters=[a, None])  # float32: its own master copy
    plan = optim.AdamWPlan([flat[256:], flat[:256], flat[256:256]])
    plan.run([torch.ones(256, device=DEV), None, None], 1, lr=1e-2)
    assert (flat[256:] < 1).all() and (flat[:256] == 1).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_on_another_stream_and_in_a_graph(bits):
    """Replays of a captured run step the parameters on, as the same calls do
    (the step's number is the captured one)."""
    def make():
        p, g = tensors(8, [300, 4097, 64], "f32", "f32")
        return p, g, optim.AdamWPlan(p, bits=bits)
    (p, g, plan), (q, h, other), (r, k, graphed) = make(), make(), make()
    plan.run(g, 5, **HYPER)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other.run(h, 5, **HYPER)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(p, q))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.run(k, 5, **HYPER)
    for i in range(4):
        if i:
            for a, b in zip(g, k):
                a.copy_(torch.randn_like(a))
                b.copy_(a)
            plan.run(g, 5, **HYPER)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(p, r)), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_masters_follow_parameters_that_are_loaded(dtype):
    """Weights that are put back between steps are stepped from there; those
    that were not touched keep their masters' last bits."""
    hy = dict(lr=1e-3, weight_decay=0.0, masters=True)
    p, q = (torch.nn.Parameter(torch.linspace(-1, 1, 300, device=DEV).to(dtype)) for _ in range(2))
    opt = optim.AdamW([p, q], **hy)
    best = p.detach().clone()
    for _ in range(3):
        p.grad, q.grad = torch.ones_like(p), torch.ones_like(q)
        opt.step()
    kept = opt.state[q]["master"].clone()
    with torch.no_grad():
        p.copy_(best)
        p[100:200] = q[100:200]  # these are their masters' roundings as before
        q.copy_(q.clone())       # a new version, the same values
    old = opt.state[p]["master"].clone()
    same = old.to(dtype) == best  # moved by less than the type shows: still its rounding
    assert not same.all()
    start = torch.where(same, old, best.float())
    start[100:200] = old[100:200]
    opt.step()
    # steps of one sign move by the learning rate, to 2^-20 of 1
    assert float((opt.state[p]["master"] - (start - 1e-3)).abs().max()) <= 2.0 ** -20
    assert float((opt.state[q]["master"] - (kept - 1e-3)).abs().max()) <= 2.0 ** -20
    assert torch.equal(p, opt.state[p]["master"].to(dtype))
    # a state that is loaded goes with the weights it was saved with, in either order
    saved, weights = copy.deepcopy(opt.state_dict()), [t.detach().clone() for t in (p, q)]
    opt.step()
    after = [t.detach().clone() for t in (p, q)]
    opt.step()
    opt.load_state_dict(saved)
    with torch.no_grad():
        for t, w in zip((p, q), weights):
            t.copy_(w)
    opt.step()
    assert torch.equal(p, after[0]) and torch.equal(q, after[1])


def test_a_plan_that_goes_while_another_stream_uses_it():
    """Its table and states are not handed out again before that stream has
    passed the step."""
    p, g = tensors(9, [5000, 300], "f32", "f32")
    plan = optim.AdamWPlan(p)
    sizes = [plan.table.numel(), 4 * 5000, 4 * 300]
    held = {t.data_ptr() for t in (plan.table, *plan.exp_avg, *plan.exp_avg_sq)}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        plan.run(g, 1, **HYPER)
    del plan
    new = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
    assert not s.query()  # else the check below says nothing
    assert not held & {t.data_ptr() for t in new}
    s.synchronize()
    want, other = tensors(9, [5000, 300], "f32", "f32")
    optim.AdamWPlan(want).run(other, 1, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(p, want))
