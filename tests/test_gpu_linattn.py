"""Linear attention with a decay for each head against its recurrence in
float64 (numpy, one position at a time).

Bars.  Every output is a sum of products; its error is bounded by the
roundings times the same sum over magnitudes, computed beside it (`size`).
Float32: a product of Dk terms, a sum over a chunk, over the chunks and the
decays e^{g n} (their exponents |g n| up to about 30 where a term still
counts): (Dk + 160 + T/16) 2^-24 size.  bfloat16 and float16 inputs are
exact; the working values keep at least 16 bits (2^-16 size), and the output
rounds once more, by 2^-8 or 2^-11 of itself (float16: by 2^-25 near 0)."""
import math

import numpy as np
import pytest
import torch

from semi_markov_crf_zero_amd import encoder

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def bar(value, size, dtype, D, T):
    work = 2.0 ** -16 if dtype != "f32" else 0.0
    return ((D + 160 + T / 16) * 2.0 ** -24 + work) * size + ULP[dtype] * np.abs(value) + 2.0 ** -25


def bar32(size, D, T):
    """Float32 outputs whatever the inputs: products of exact inputs."""
    return (D + 160 + T / 16) * 2.0 ** -24 * size + 1e-30


def reference(q, k, v, g, lengths, state, scale, do=None, ds=None):
    """Outputs and the same with every term's magnitude.  q, k, v [B, T, heads, D] float64."""
    B, T = q.shape[:2]
    H = len(g)
    rep = [H // t.shape[2] for t in (q, k, v)]
    Q, K, V = (np.repeat(t, r, axis=2) for t, r in zip((q, k, v), rep))
    Dk, Dv = Q.shape[3], V.shape[3]
    e = np.exp(g)
    out = []
    for mag in (False, True):
        f = np.abs if mag else (lambda x: x)
        sc = abs(scale) if mag else scale
        o = np.zeros((B, T, H, Dv))
        last = np.zeros((B, H, Dk, Dv))
        r = dict(o=o, last=last)
        if do is not None:
            r.update(q=np.zeros(Q.shape), k=np.zeros(K.shape), v=np.zeros(V.shape),
                     state=np.zeros((B, H, Dk, Dv)))
        for b in range(B):
            S = f(state[b]).copy() if state is not None else np.zeros((H, Dk, Dv))
            for t in range(lengths[b]):
                S = e[:, None, None] * S + f(K[b, t])[:, :, None] * f(V[b, t])[:, None, :]
                o[b, t] = sc * np.einsum("hij,hi->hj", S, f(Q[b, t]))
                if do is not None:
                    r["q"][b, t] = sc * np.einsum("hij,hj->hi", S, f(do[b, t]))
            last[b] = S
            if do is not None:
                G = f(ds[b]).copy() if ds is not None else np.zeros((H, Dk, Dv))
                for t in reversed(range(lengths[b])):
                    G = G + sc * f(Q[b, t])[:, :, None] * f(do[b, t])[:, None, :]
                    r["k"][b, t] = np.einsum("hij,hj->hi", G, f(V[b, t]))
                    r["v"][b, t] = np.einsum("hij,hi->hj", G, f(K[b, t]))
                    G = e[:, None, None] * G
                r["state"][b] = G
        if do is not None:
            for n, x, s in (("q", q, rep[0]), ("k", k, rep[1]), ("v", v, rep[2])):
                r[n] = r[n].reshape(B, T, x.shape[2], s, -1).sum(3)
        out.append(r)
    return out


def draw(seed, B, T, heads, Dk, Dv, dtype, state, decay=None):
    gen = torch.Generator().manual_seed(seed)
    H = max(heads)
    t = {n: torch.randn((B, T, h, d), generator=gen).to(TYPES[dtype])
         for n, h, d in (("q", heads[0], Dk), ("k", heads[1], Dk), ("v", heads[2], Dv),
                         ("do", H, Dv))}
    t["state"] = torch.randn((B, H, Dk, Dv), generator=gen) if state else None
    t["ds"] = torch.randn((B, H, Dk, Dv), generator=gen)
    t["g"] = (-torch.exp2(-torch.linspace(0.0, 9.0, H)) if decay is None
              else torch.tensor(decay, dtype=torch.float32))
    return t


def check(name, got, want, size, tol):
    got = got.detach().float().cpu().double().numpy()
    assert got.shape == want.shape, name
    off = np.abs(got - want) - tol
    assert np.all(off <= 0), (name, float(np.nanmax(off)), np.argwhere(~(off <= 0))[:4].tolist())


def compare(t, dtype, lengths=None, backward=True, views=None, scale=None):
    B, T, _, Dk = t["q"].shape
    Dv = t["v"].shape[3]
    d = {n: None if x is None else x.to(DEV) for n, x in t.items()}
    if views is not None:
        d.update(views(d))
    lens = [T] * B if lengths is None else lengths
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    wrt = [n for n in ("q", "k", "v", "state") if d[n] is not None]
    if backward:
        for n in wrt:
            d[n].requires_grad_(True)
    o, last = encoder.linear_attention(d["q"], d["k"], d["v"], d["g"], lengths=lt,
                                       state=d["state"], scale=scale, return_state=True)
    f64 = {n: None if t[n] is None else t[n].double().numpy() for n in t}
    want, size = reference(f64["q"], f64["k"], f64["v"], f64["g"], lens, f64["state"],
                           Dk ** -0.5 if scale is None else scale,
                           f64["do"] if backward else None, f64["ds"])
    check("o", o, want["o"], size["o"], bar(want["o"], size["o"], dtype, Dk, T))
    check("last", last, want["last"], size["last"], bar32(size["last"], Dk, T))
    assert o.dtype == TYPES[dtype] and last.dtype == torch.float32
    if backward:
        grads = torch.autograd.grad((o, last), [d[n] for n in wrt], (d["do"], d["ds"]))
        for n, gr in zip(wrt, grads):
            tol = (bar32(size[n], Dv, T) if n == "state"
                   else bar(want[n], size[n], dtype, max(Dk, Dv), T))
            check("grad " + n, gr, want[n], size[n], tol)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [1, 2, 31, 63, 64, 65, 130, 257])
def test_lengths_of_a_sequence(T, dtype):
    compare(draw(T, 2, T, (2, 2, 2), 64, 64, dtype, True), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Dk,Dv", [(1, 1), (3, 5), (16, 32), (33, 64), (64, 33), (40, 72),
                                   (96, 128), (128, 16), (130, 65), (200, 256), (256, 200)])
def test_widths(Dk, Dv, dtype):
    compare(draw(Dk, 2, 100, (2, 2, 2), Dk, Dv, dtype, True), dtype, lengths=[100, 71])


@pytest.mark.parametrize("heads", [(1, 1, 1), (4, 2, 2), (4, 1, 4), (2, 2, 6), (1, 3, 3),
                                   (6, 2, 3), (5, 5, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_heads(heads, dtype):
    compare(draw(7, 2, 90, heads, 24, 40, dtype, True), dtype, lengths=[90, 66])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_ragged_lengths_and_nan_past_them(dtype):
    t = draw(3, 6, 150, (2, 2, 2), 32, 48, dtype, True)
    lengths = [150, 0, 1, 64, 65, 128]

    def views(d):
        out = {}
        for n in ("q", "k", "v", "do"):
            x = d[n].clone()
            for b, L in enumerate(lengths):
                x[b, L:] = float("nan")
            out[n] = x
        return out
    compare(t, dtype, lengths=lengths, views=views)


def test_invalid_lengths():
    t = draw(4, 4, 70, (2, 2, 2), 16, 16, "f32", True)
    d = {n: x.to(DEV) for n, x in t.items()}
    lengths = torch.tensor([70, -1, 71, 30], dtype=torch.int32, device=DEV)
    for n in ("q", "k", "v", "state"):
        d[n].requires_grad_(True)
    o, last = encoder.linear_attention(d["q"], d["k"], d["v"], d["g"], lengths=lengths,
                                       state=d["state"], return_state=True)
    grads = torch.autograd.grad((o, last), [d[n] for n in ("q", "k", "v", "state")],
                                (d["do"], d["ds"]))
    assert o[1:3].isnan().all() and last[1:3].isnan().all()
    assert o[[0, 3]].isfinite().all() and last[[0, 3]].isfinite().all()
    for g in grads:
        assert (g[1:3] == 0).all() and g.isfinite().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [[0.0, 0.0], [-float("inf"), -1e-6], [-200.0, -0.5],
                                   [-1e-9, -88.0]])
def test_extreme_decays(decay, dtype):
    compare(draw(5, 2, 200, (2, 2, 2), 32, 32, dtype, True, decay), dtype, lengths=[200, 133])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_strided_inputs(dtype):
    """q, k and v as slices of one projection, [B, T, 3 H D] and [T, B, ...]."""
    t = draw(6, 2, 77, (3, 3, 3), 40, 40, dtype, False)

    def fused(d):
        x = torch.cat([d[n].flatten(2) for n in "qkv"], dim=2)
        return {n: x[..., 120 * i:120 * (i + 1)].unflatten(2, (3, 40)) for i, n in enumerate("qkv")}

    def time_first(d):
        return {n: d[n].permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3) for n in "qkv"}

    def heads_first(d):
        return {n: d[n].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for n in "qkv"}

    def odd_start(d):  # one element past an aligned address, and odd row strides
        out = {}
        for n in "qkv":
            x = torch.zeros((2, 77, 3, 43), dtype=d[n].dtype, device=DEV)
            x[..., 1:41] = d[n]
            out[n] = x[..., 1:41]
        return out

    def columns(d):  # rows that are not contiguous are copied
        return {n: d[n].transpose(2, 3).contiguous().transpose(2, 3) for n in "qkv"}
    for views in (fused, time_first, heads_first, odd_start, columns):
        compare(t, dtype, lengths=[77, 50], views=lambda d: {
            n: x.detach() for n, x in views(d).items()})


def test_broadcast_inputs():
    """A key expanded over the batch: its gradient is the sum over the batch."""
    t = draw(8, 3, 70, (2, 2, 2), 16, 24, "f32", False)
    t["k"] = t["k"][:1].expand(3, -1, -1, -1).contiguous()
    d = {n: None if x is None else x.to(DEV) for n, x in t.items()}
    k1 = d["k"][:1].clone().requires_grad_(True)
    o = encoder.linear_attention(d["q"], k1.expand(3, -1, -1, -1), d["v"], d["g"])
    got, = torch.autograd.grad(o, k1, d["do"])
    f64 = {n: None if t[n] is None else t[n].double().numpy() for n in t}
    want, size = reference(f64["q"], f64["k"], f64["v"], f64["g"], [70] * 3, None, 0.25,
                           f64["do"], None)
    check("k", got, want["k"].sum(0, keepdims=True), None,
          bar(want["k"].sum(0), size["k"].sum(0), "f32", 24, 70)[None])


@pytest.mark.parametrize("dtype,T,B", [("f32", 5000, 1), ("bf16", 5000, 1), ("bf16", 2300, 2),
                                       ("f16", 3001, 1)])
def test_long_sequences(dtype, T, B):
    """Sequences split over workgroups; ragged so that splits end early."""
    t = draw(9, B, T, (2, 2, 2), 32, 32, dtype, True)
    compare(t, dtype, lengths=[T - 17, T // 3][:B])


def test_pieces_equal_the_whole():
    """The state after a piece continues the next one."""
    t = draw(10, 2, 210, (2, 2, 2), 48, 64, "f32", False)
    d = {n: None if x is None else x.to(DEV) for n, x in t.items()}
    whole, end = encoder.linear_attention(d["q"], d["k"], d["v"], d["g"], return_state=True)
    state, parts = None, []
    for a, b in ((0, 1), (1, 65), (65, 66), (66, 210)):
        o, state = encoder.linear_attention(d["q"][:, a:b], d["k"][:, a:b], d["v"][:, a:b], d["g"],
                                            state=state, return_state=True)
        parts.append(o)
    f64 = {n: None if t[n] is None else t[n].double().numpy() for n in t}
    _, size = reference(f64["q"], f64["k"], f64["v"], f64["g"], [210] * 2, None, 48 ** -0.5)
    tol = 2 * bar32(size["o"], 48, 210)
    assert np.all((torch.cat(parts, 1) - whole).abs().cpu().double().numpy() <= tol)
    assert np.all((state - end).abs().cpu().double().numpy() <= 2 * bar32(size["last"], 48, 210))


def test_gradients_against_differences():
    """o and the last state are linear in each of q, k, v and state alone, so
    a central difference of any step is the derivative; the loss is summed in
    float64 and its error is the outputs' bar."""
    t = draw(11, 2, 100, (2, 1, 2), 20, 28, "f32", True)
    d = {n: x.to(DEV) for n, x in t.items()}
    lengths = torch.tensor([100, 67], dtype=torch.int32, device=DEV)
    names = ("q", "k", "v", "state")

    def loss(x):
        o, last = encoder.linear_attention(x["q"], x["k"], x["v"], x["g"], lengths=lengths,
                                           state=x["state"], return_state=True)
        return float((o.double() * x["do"].double()).sum() + (last.double() * x["ds"].double()).sum())

    x = {n: v.clone().requires_grad_(n in names) for n, v in d.items()}
    o, last = encoder.linear_attention(x["q"], x["k"], x["v"], x["g"], lengths=lengths,
                                       state=x["state"], return_state=True)
    grads = torch.autograd.grad((o, last), [x[n] for n in names], (d["do"], d["ds"]))
    f64 = {n: t[n].double().numpy() for n in t}
    _, size = reference(f64["q"], f64["k"], f64["v"], f64["g"], [100, 67], f64["state"], 20 ** -0.5)
    whole = float((np.abs(f64["do"]) * size["o"]).sum() + (np.abs(f64["ds"]) * size["last"]).sum())
    for i, n in enumerate(names):
        # a direction that is exact in float32: +-1 times a power of two
        gen = torch.Generator().manual_seed(20 + i)
        u = (torch.randint(0, 2, t[n].shape, generator=gen) * 2 - 1).float().to(DEV)
        up, down = dict(d), dict(d)
        up[n], down[n] = d[n] + u, d[n] - u
        num = (loss(up) - loss(down)) / 2
        ana = float((grads[i].double() * u.double()).sum())
        # magnitudes grow by at most 1 + 1/mean|x| ~ 3 under the shift
        assert abs(num - ana) <= 3 * (28 + 160 + 7) * 2.0 ** -24 * whole, n


def test_only_what_is_asked_for():
    t = draw(12, 2, 70, (2, 2, 2), 16, 16, "bf16", True)
    d = {n: x.to(DEV) for n, x in t.items()}
    v = d["v"].clone().requires_grad_(True)
    o = encoder.linear_attention(d["q"], d["k"], v, d["g"])
    o.backward(d["do"])
    assert v.grad.isfinite().all()
    state = d["state"].clone().requires_grad_(True)
    _, last = encoder.linear_attention(d["q"], d["k"], d["v"], d["g"], state=state,
                                       return_state=True)
    g, = torch.autograd.grad(last, state, d["ds"])  # o unused: its gradient is 0
    want = np.exp(70 * t["g"].double().numpy())[None, :, None, None] * t["ds"].double().numpy()
    assert np.all(np.abs(g.cpu().double().numpy() - want) <= (16 + 165) * 2.0 ** -24 * np.abs(want) + 1e-30)


def test_empty_calls():
    g = torch.zeros(2, device=DEV)
    q = torch.zeros((2, 0, 2, 8), device=DEV)
    s = torch.ones((2, 2, 8, 8), device=DEV)
    o, last = encoder.linear_attention(q, q, q, g, state=s, return_state=True)
    assert o.shape == (2, 0, 2, 8) and torch.equal(last, s) and last.data_ptr() != s.data_ptr()
    q = torch.zeros((0, 5, 2, 8), device=DEV)
    assert encoder.linear_attention(q, q, q, g).shape == (0, 5, 2, 8)


def test_other_stream_and_graph():
    """A call on a stream of its own, and captured: replays follow the inputs."""
    t = draw(13, 2, 3000, (2, 2, 2), 64, 64, "bf16", True)
    d = {n: x.to(DEV) for n, x in t.items()}
    call = lambda: encoder.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["state"],  # noqa: E731
                                            return_state=True)
    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(3):
        d["v"].copy_(torch.randn_like(d["v"]))
        want = call()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i


def test_offsets_past_32_bits():
    """Batch rows 2^32 elements apart."""
    far = (1 << 32) + 64
    big = torch.empty(far + 70 * 2 * 16, dtype=torch.bfloat16, device=DEV)
    t = draw(14, 2, 70, (2, 2, 2), 16, 16, "bf16", False)

    def views(d):
        v = big.as_strided((2, 70, 2, 16), (far, 32, 16, 1))
        v.copy_(d["v"])
        return {"v": v}
    compare(t, "bf16", backward=False, views=views)
    del big
    torch.cuda.empty_cache()


# ---- single positions ------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,Dk,Dv", [((4, 4, 4), 64, 64), ((2, 2, 2), 128, 128),
                                         ((4, 2, 2), 40, 72), ((1, 3, 3), 5, 7),
                                         ((2, 2, 2), 256, 256), ((2, 2, 2), 33, 130)])
def test_step(heads, Dk, Dv, dtype):
    B, N, H = 5, 9, max(heads)
    t = draw(15, B, 1, heads, Dk, Dv, dtype, False)
    gen = torch.Generator().manual_seed(1)
    pool = torch.randn((N, H, Dk, Dv), generator=gen)
    slots = [7, -1, 0, 9, 3]  # the second and the fourth are idle
    d = {n: x[:, 0].to(DEV) for n, x in t.items() if n in "qkv"}
    state = pool.to(DEV)
    o = encoder.linear_attention_step(d["q"], d["k"], d["v"], t["g"].to(DEV), state,
                                      slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    for b, s in enumerate(slots):
        if not 0 <= s < N:
            assert (o[b] == 0).all()
            continue
        f = {n: t[n][b:b + 1].double().numpy() for n in "qkv"}
        want, size = reference(f["q"], f["k"], f["v"], t["g"].double().numpy(), [1],
                               pool[s:s + 1].double().numpy(), Dk ** -0.5)
        check("o", o[b:b + 1, None], want["o"], None, bar(want["o"], size["o"], dtype, Dk, 1))
        check("state", state[s:s + 1], want["last"], None, bar32(size["last"], 0, 1))
    others = [i for i in range(N) if i not in slots]
    assert torch.equal(state[others].cpu(), pool[others])


def test_steps_follow_the_whole_sequence():
    t = draw(16, 3, 20, (2, 2, 2), 32, 48, "bf16", True)
    d = {n: x.to(DEV) for n, x in t.items()}
    whole, end = encoder.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["state"],
                                          return_state=True)
    state = d["state"].clone()
    f = {n: t[n].double().numpy() for n in t}
    want, size = reference(f["q"], f["k"], f["v"], f["g"], [20] * 3, f["state"], 32 ** -0.5)
    for i in range(20):
        # rows of a fused [B, heads, D] slice: strided
        o = encoder.linear_attention_step(d["q"][:, i], d["k"][:, i], d["v"][:, i], d["g"], state)
        check("o", o, want["o"][:, i], None, bar(want["o"], size["o"], "bf16", 32, 20)[:, i])
    check("state", state, want["last"], None, bar32(size["last"], 32, 20))
    check("state", end, want["last"], None, bar32(size["last"], 32, 20))


def test_refusals():
    q = torch.zeros((2, 5, 4, 8), device=DEV)
    g = torch.zeros(4, device=DEV)
    la = encoder.linear_attention
    for args, kw in (((q, q[:, :4], q, g), {}), ((q, q.half(), q, g), {}),
                     ((q, q[..., :7], q, g), {}), ((q, q[:, :, :3], q, g), {}),
                     ((q, q, q, g[:3]), {}), ((q, q, q, g.double()), {}), ((q[0], q, q, g), {}),
                     ((q.double(), q.double(), q.double(), g), {}),
                     ((q, q, q, g.clone().requires_grad_(True)), {}),
                     ((q, q, q, g), dict(lengths=torch.zeros(2, device=DEV))),
                     ((q, q, q, g), dict(lengths=torch.zeros(3, dtype=torch.int32, device=DEV))),
                     ((q, q, q, g), dict(state=torch.zeros((2, 4, 8, 7), device=DEV))),
                     ((torch.zeros((1, 1, 1, 257), device=DEV),) * 3 + (g[:1],), {})):
        with pytest.raises(ValueError):
            la(*args, **kw)
    x, s = q[:, 0], torch.zeros((3, 4, 8, 8), device=DEV)
    for args, kw in (((q, q, q, g, s), {}), ((x, x, x, g, s[:, :3]), {}),
                     ((x, x, x, g, s.half()), {}), ((x, x, x, g, s[:0]), {}),
                     ((x, x, x, g, s), dict(slots=torch.zeros(2, dtype=torch.int64, device=DEV))),
                     ((x, x, x, g, s.transpose(2, 3)), {})):
        with pytest.raises(ValueError):
            encoder.linear_attention_step(*args, **kw)


def test_backward_without_the_forward_call():
    """semicrf_linattn_bwd with no states left by a forward call computes them."""
    import ctypes
    t = draw(17, 1, 3000, (2, 2, 2), 32, 48, "bf16", True)
    d = {n: x.to(DEV) for n, x in t.items()}
    for n in ("q", "k", "v", "state"):
        d[n].requires_grad_(True)
    o, last = encoder.linear_attention(d["q"], d["k"], d["v"], d["g"], state=d["state"],
                                       return_state=True)
    want = torch.autograd.grad((o, last), [d[n] for n in ("q", "k", "v", "state")],
                               (d["do"], d["ds"]))
    fields = (1, 3000, 2, 2, 2, 2, 32, 48, 1, 32 ** -0.5,
              *(d[n].stride()[:3] for n in ("q", "k", "v")))
    ws, n = encoder._workspace("semicrf_linattn_workspace_size", encoder._LinattnShape, fields, 1,
                               o.device)
    got = [torch.empty_like(x) for x in want]
    encoder.launch(encoder.load().semicrf_linattn_bwd, o.device,
                   ctypes.byref(encoder._LinattnShape(*fields)),
                   *(d[n].data_ptr() for n in ("q", "k", "v", "g")), None, d["state"].data_ptr(),
                   None, d["do"].data_ptr(), d["ds"].data_ptr(), *(x.data_ptr() for x in got),
                   ws.data_ptr(), n)
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(1 << 18, 1), (40000, 160)])
def test_slow_decays_over_long_sequences(T, H, dtype):
    """k = v = 1: every element of the state is sum_j e^{g j}, a closed form.
    Each chunk (and segment) rounds it once, without a sign: 4 sqrt(n) 2^-24 of
    it for the n roundings; e^{g 64} used as one float32 would put its own
    rounding in thousands of times with one sign.  T = 40000 over 160 heads is
    one segment or few."""
    g = float(np.float32(-1.5 / T))
    k = torch.ones((1, T, H, 16), dtype=TYPES[dtype], device=DEV)
    _, last = encoder.linear_attention(k, k, k, torch.full((H,), g, device=DEV), return_state=True)
    want = np.expm1(g * T) / np.expm1(g)
    off = np.abs(last.cpu().double().numpy() / want - 1).max()
    assert off <= 4 * np.sqrt(T / 32 + 64) * 2.0 ** -24, off


def test_second_derivatives_are_refused():
    """A penalty on a gradient would lack the terms through the operator."""
    q, k, v = (torch.randn((1, 5, 2, 4), device=DEV, requires_grad=True) for _ in range(3))
    g = torch.full((2,), -0.1, device=DEV)
    o = encoder.linear_attention(q, k, v, g)
    grads = torch.autograd.grad(o.square().sum(), (q, k, v), create_graph=True)
    first = torch.autograd.grad(encoder.linear_attention(q, k, v, g).square().sum(), (q, k, v))
    for a, b in zip(grads, first):
        assert torch.equal(a, b)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        sum(t.square().sum() for t in grads).backward()


def test_a_step_is_seen_by_autograd():
    """A backward pass over states that a step has moved since must not run."""
    q, k, v = (torch.randn((1, 5, 2, 4), device=DEV, requires_grad=True) for _ in range(3))
    g = torch.full((2,), -0.1, device=DEV)
    pool = torch.zeros((1, 2, 4, 4), device=DEV)
    o = encoder.linear_attention(q, k, v, g, state=pool)
    with torch.no_grad():
        encoder.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g, pool)
    with pytest.raises(RuntimeError, match="inplace operation"):
        o.sum().backward()


def test_empty_calls_carry_gradients():
    g = torch.zeros(2, device=DEV)
    q = torch.zeros((2, 0, 2, 8), device=DEV, dtype=torch.bfloat16, requires_grad=True)
    o, last = encoder.linear_attention(q, q, q, g, return_state=True)
    assert o.shape == (2, 0, 2, 8) and last.shape == (2, 2, 8, 8) and not last.any()
    assert o.dtype == torch.bfloat16 and last.dtype == torch.float32
    (o.float().sum() + last.sum()).backward()
    assert q.grad.shape == q.shape
    s = torch.ones((2, 2, 8, 8), device=DEV, requires_grad=True)
    encoder.linear_attention(q, q, q, g, state=s, return_state=True)[1].sum().backward()
    assert torch.equal(s.grad, torch.ones_like(s))


def test_slow_decays_over_many_steps():
    """A state that is only read: S_n = e^{g n} S_0.  A step rounds it twice at
    most, by 2^-24 of it, without a sign over the 64 elements and 12 decays: 6
    sqrt(2 n) 2^-24 of it.  e^g used as one float32, up to 2^-25 off, would
    add up to n 2^-25, 7 times that at n = 5000.  An infinite element stays
    infinite."""
    n, H = 5000, 12
    g = torch.tensor([-1.0 / (700 + 100 * i) for i in range(H)])
    s0 = 1 + torch.rand((1, H, 8, 8), generator=torch.Generator().manual_seed(3))
    q = torch.zeros((1, H, 8), device=DEV)
    state, gd = s0.to(DEV), g.to(DEV)
    for _ in range(n):
        encoder.linear_attention_step(q, q, q, gd, state)
    want = np.exp(g.double().numpy() * n)[None, :, None, None] * s0.double().numpy()
    off = np.abs(state.cpu().double().numpy() / want - 1).max()
    assert off <= 6 * np.sqrt(2 * n) * 2.0 ** -24, off
    state[0, 0, 0, 0] = math.inf
    encoder.linear_attention_step(q, q, q, gd, state)
    assert state[0, 0, 0, 0] == math.inf


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_what_is_left_where_terms_cancel(dtype):
    """a = 1 + 2^-9 + 2^-18 and b = 1 + 2^-9 are neighbours to 16 bits, and
    float32 knows them apart.  They meet as elements of a state and as products
    of two rows, for every output; with g = 0 and a scale of 1 every other
    operation is exact.  A handful of roundings of values up to 2: 8 * 2^-24."""
    a, b, left, bar8 = 1 + 2.0 ** -9 + 2.0 ** -18, 1 + 2.0 ** -9, 2.0 ** -18, 8 * 2.0 ** -24
    g = torch.zeros(1, device=DEV)

    def call(q, k, v, state):
        t = [x.clone().to(TYPES[dtype]).requires_grad_(True) for x in (q, k, v)]
        return t, encoder.linear_attention(*t, g, state=state, scale=1.0, return_state=True)

    def near(x, want):
        assert abs(x.item() - want) <= bar8, (x.item(), want)

    def rows(T, **at):  # [1, T, 1, 32], rows t0.. as given
        x = torch.zeros((1, T, 1, 32), device=DEV)
        for t, row in at.items():
            x[0, int(t[1:]), 0, :3] = torch.tensor(row, device=DEV)
        return x

    # elements of a state: S = G = [[a, b], [b, a]], rows (1, -1)
    S = torch.zeros((1, 1, 32, 32), device=DEV)
    S[0, 0, :2, :2] = torch.tensor([[a, b], [b, a]], device=DEV)
    one, none = rows(1, t0=[1.0, -1.0, 0.0]), rows(1)
    (q, _, _), (o, _) = call(one, none, none, S)
    near(o[0, 0, 0, 0], left)
    dq, = torch.autograd.grad(o, q, one.to(o.dtype))
    near(dq[0, 0, 0, 0], left)
    (_, k, v), (_, last) = call(none, one, one, None)
    dk, dv = torch.autograd.grad(last, (k, v), S)
    near(dk[0, 0, 0, 0], left)
    near(dv[0, 0, 0, 0], left)

    # products of rows
    ones, minus = [1.0, 1.0, 1.0], [-1.0, -1.0, -1.0]
    far, near_ = [1.0, 2.0 ** -9, 2.0 ** -18], [1.0, 2.0 ** -9, 0.0]
    _, (o, _) = call(rows(3, t2=ones), rows(3, t0=far, t1=near_), rows(3, t0=ones, t1=minus), None)
    near(o[0, 2, 0, 0], left)
    (q, _, _), (o, _) = call(rows(3), rows(3, t0=ones, t1=minus), rows(3, t0=far, t1=near_), None)
    dq, = torch.autograd.grad(o, q, rows(3, t2=ones).to(o.dtype))
    near(dq[0, 2, 0, 0], left)
    (_, k, _), (o, _) = call(rows(3, t1=ones, t2=minus), rows(3), rows(3, t0=ones), None)
    dk, = torch.autograd.grad(o, k, rows(3, t1=far, t2=near_).to(o.dtype))
    near(dk[0, 0, 0, 0], left)
    (_, _, v), (o, _) = call(rows(3, t1=far, t2=near_), rows(3, t0=ones), rows(3), None)
    dv, = torch.autograd.grad(o, v, rows(3, t1=ones, t2=minus).to(o.dtype))
    near(dv[0, 0, 0, 0], left)


def test_sizes_past_31_bits_are_refused():
    """The library's sizes are ints: 2^32 + 1 streams would be one there."""
    x = torch.zeros((1, 1, 1), device=DEV).expand((1 << 32) + 1, 1, 1)
    g = torch.zeros(1, device=DEV)
    with pytest.raises(ValueError, match="sizes"):
        encoder.linear_attention_step(x, x, x, g, torch.zeros((1, 1, 1, 1), device=DEV))
    with pytest.raises(ValueError, match="sizes"):
        encoder.linear_attention(x[:, None], x[:, None], x[:, None], g)


@pytest.mark.parametrize("way", ["backward", "grad"])
def test_second_derivatives_are_refused_beside_others(way):
    """The gradient of a plain sum: what comes in asks for no gradient, and
    the penalty also depends on w by a way that is known."""
    w = torch.full((1, 5, 2, 4), 2.0, device=DEV, requires_grad=True)
    a = torch.randn((1, 5, 2, 4), device=DEV, requires_grad=True)
    q = w * a
    o = encoder.linear_attention(q, q, q, torch.full((2,), -0.1, device=DEV))
    g, = torch.autograd.grad(o.sum(), a, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        if way == "grad":
            torch.autograd.grad(g.square().sum(), w)
        else:
            g.square().sum().backward()


def test_a_step_s_missing_gradients_are_noticed():
    """The result of a step has none: a backward pass through it fails and does
    not leave q, k and v out; a state that wants one is not moved."""
    g = torch.full((2,), -0.1, device=DEV)
    for i in range(3):
        x = [torch.randn((3, 2, 4), device=DEV) for _ in range(3)]
        pool = torch.zeros((3, 2, 4, 4), device=DEV)
        want = encoder.linear_attention_step(*x, g, pool.clone())
        assert not want.requires_grad
        x[i].requires_grad_(True)
        o = encoder.linear_attention_step(*x, g, pool)
        assert torch.equal(o, want)
        with pytest.raises(RuntimeError, match="no gradients"):
            (o.sum() + x[i].sum()).backward()
        with pytest.raises(RuntimeError, match="no gradients"):
            torch.autograd.grad(o.sum() + x[i].sum(), x[i])
        with torch.no_grad():
            assert not encoder.linear_attention_step(*x, g, pool).requires_grad
    pool = torch.zeros((3, 2, 4, 4), device=DEV, requires_grad=True)
    with pytest.raises(ValueError, match="in place"):
        encoder.linear_attention_step(*x, g, pool)
    assert not pool.detach().any()
    with torch.no_grad():
        encoder.linear_attention_step(*x, g, pool)
    assert pool.detach().any()


def test_more_heads_than_two_million():
    """2^21 + 5 sequences of two positions, written out, and as many streams.
    `bar32`'s constants; T = 2."""
    B, D, e = (1 << 21) + 5, 4, math.exp(-0.5)
    g = torch.full((1,), -0.5, device=DEV)
    q, k, v, do = (torch.randn((B, 2, 1, D), device=DEV) for _ in range(4))
    v.requires_grad_(True)
    o, last = encoder.linear_attention(q, k, v, g, scale=1.0, return_state=True)
    dv, = torch.autograd.grad(o, v, do)
    state = torch.zeros((B, 1, D, D), device=DEV)
    v = v.detach()
    steps = [encoder.linear_attention_step(q[:, t], k[:, t], v[:, t], g, state, scale=1.0)
             for t in range(2)]
    off = []
    for f in (lambda x: x, torch.abs):
        (q0, q1), (k0, k1), (v0, v1), (d0, d1) = (f(x.double()).unbind(1) for x in (q, k, v, do))
        dot = lambda a, b: (a * b).sum(-1, keepdim=True)  # noqa: E731
        off.append((torch.stack([dot(q0, k0) * v0, e * dot(q1, k0) * v0 + dot(q1, k1) * v1], 1),
                    e * k0[..., None] * v0[..., None, :] + k1[..., None] * v1[..., None, :],
                    torch.stack([dot(k0, q0) * d0 + e * dot(k0, q1) * d1, dot(k1, q1) * d1], 1)))
    c = (D + 160 + 1) * 2.0 ** -24
    for got, want, size in zip((o, last, dv), *off):
        assert ((got.double() - want).abs() <= c * size + 1e-30).all()
    for got, i in ((torch.stack(steps, 1), 0), (state, 1)):
        assert ((got.double() - off[0][i]).abs() <= c * off[1][i] + 1e-30).all()


def test_invalid_lengths_of_empty_calls():
    q = torch.zeros((3, 0, 2, 8), device=DEV)
    state = torch.ones((3, 2, 8, 8), device=DEV, requires_grad=True)
    lengths = torch.tensor([0, 1, -1], dtype=torch.int32, device=DEV)
    _, last = encoder.linear_attention(q, q, q, torch.zeros(2, device=DEV), lengths=lengths,
                                       state=state, return_state=True)
    assert torch.equal(last[0], state[0]) and last[1:].isnan().all()
    g, = torch.autograd.grad(last, state, torch.ones_like(last))
    assert (g[0] == 1).all() and (g[1:] == 0).all()


def segments_of(t):
    """How many segments the sequences are cut into, by the states kept."""
    B, T, Hq, Dk = t["q"].shape
    Hk, Hv, Dv = t["k"].shape[2], *t["v"].shape[2:]
    H = max(Hq, Hk, Hv)
    n = encoder._workspace_bytes("semicrf_linattn_workspace_size", encoder._LinattnShape,
                                 (B, T, H, Hq, Hk, Hv, Dk, Dv, encoder.DTYPES[t["q"].dtype], 1.0,
                                  (0, 0, 0), (0, 0, 0), (0, 0, 0)), 0)
    return 1 + n // (4 * B * H * Dk * Dv)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Dk,Dv", [(40, 72), (33, 65), (96, 128), (128, 24), (130, 200), (256, 256),
                                   (8, 96)])
def test_widths_over_segments(Dk, Dv, dtype):
    """Both passes over segments whose states are not square, and whose ends
    the lengths part."""
    t = draw(Dk + Dv, 2, 1500, (1, 1, 1), Dk, Dv, dtype, True, decay=[-1.0 / 512])
    assert segments_of(t) > 1
    compare(t, dtype, lengths=[1500, 777])


@pytest.mark.parametrize("heads", [(4, 2, 2), (1, 3, 3), (2, 2, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_heads_over_segments(heads, dtype):
    t = draw(31, 2, 1400, heads, 24, 40, dtype, True)
    assert segments_of(t) > 1
    compare(t, dtype, lengths=[1400, 513])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Dk,Dv", [(40, 72), (136, 48)])
def test_rows_read_by_element_over_segments(Dk, Dv, dtype):
    """One element past an aligned address, odd strides; NaN past the lengths."""
    t = draw(32, 2, 1300, (1, 1, 1), Dk, Dv, dtype, True, decay=[-1.0 / 300])
    assert segments_of(t) > 1
    lengths = [1300, 640]

    def odd_start(d):
        out = {}
        for n in "qkv":
            x = torch.zeros((2, 1300, 1, d[n].shape[3] + 3), dtype=d[n].dtype, device=DEV)
            x[..., 1:-2] = d[n]
            for b, L in enumerate(lengths):
                x[b, L:] = float("nan")
            out[n] = x[..., 1:-2]
        return out
    compare(t, dtype, lengths=lengths, views=odd_start)


def test_steps_on_another_stream_and_in_a_graph():
    """Replays move the pool on, as the same calls do."""
    gen = torch.Generator(device=DEV).manual_seed(33)
    q, k, v = (torch.randn((5, 2, 40), device=DEV, generator=gen, dtype=torch.bfloat16)
               for _ in range(3))
    g = torch.tensor([-0.1, -0.01], device=DEV)
    slots = torch.tensor([7, 3, -1, 0, 5], dtype=torch.int32, device=DEV)
    pool = torch.randn((8, 2, 40, 40), device=DEV, generator=gen)
    other, graphed = pool.clone(), pool.clone()
    want = encoder.linear_attention_step(q, k, v, g, pool, slots=slots)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = encoder.linear_attention_step(q, k, v, g, other, slots=slots)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want) and torch.equal(other, pool)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = encoder.linear_attention_step(q, k, v, g, graphed, slots=slots)
    for i in range(4):
        if i:
            q.copy_(torch.randn_like(q))
            slots.copy_(slots.roll(1))
            want = encoder.linear_attention_step(q, k, v, g, pool, slots=slots)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(graphed, pool), i


def test_decays_that_ask_for_gradients_nobody_records():
    """Refused while gradients are recorded (there is none to give), taken
    where they are not."""
    g = torch.full((2,), -0.1, device=DEV, requires_grad=True)
    q = torch.randn((1, 5, 2, 4), device=DEV)
    with torch.no_grad():
        o = encoder.linear_attention(q, q, q, g)
        s = encoder.linear_attention_step(q[:, 0], q[:, 0], q[:, 0], g,
                                          torch.zeros((1, 2, 4, 4), device=DEV))
    assert torch.equal(o, encoder.linear_attention(q, q, q, g.detach()))
    assert s.shape == (1, 2, 4)
    with pytest.raises(ValueError, match="log_decay"):
        encoder.linear_attention(q, q, q, g)
