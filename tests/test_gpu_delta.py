"""The gated delta rule against its recurrence in float64 (numpy, one position
at a time).

Bars.  With keys of length 1 and beta in [0, 2] a step is a contraction of every
column of the state, so an error put in at position t is at most its own size
later, times the decays since.  The reference carries beside each column's norm
|S_c| the sum m_c of what has gone into it, decayed: m <- a m + (1 + b) |S| + b |v|,
and the same (n_c) for the gradient of the state.  A working value is a sum of up
to D + 2 L products (L = 64 positions of a chunk at most) in a chunk's chain of
five products; each position rounds its share: w = (D + 128) 2^-24, of
    o_c      scale |q| (m_c + |S_c|)
    dq       scale sum_c |do_c| (m_c + |S_c|)
    dv_c     b n_c
    dk       sum_c (n_c (|S_c| + |v_c|) + |D_c| (m_c + |v_c|)) (1 + b) + dq's share
    db       the same
    dg       sums of dk's and dq's over the chunk.
16-bit inputs are exact, working values are float32 whatever the inputs are;
16-bit outputs round once more.  Beside this bound on each element, which counts every
rounding with one sign, the whole of an output is off by no more than 2^-18 of its
norm (64 roundings of 2^-24 of it in a row) and its own rounding."""
import math

import numpy as np
import pytest
import torch

from semi_markov_crf_zero_amd import encoder

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
NAMES = ("q", "k", "v", "g", "b", "state")


def norm(x, axis=-1):
    return np.sqrt((x * x).sum(axis))


def reference(q, k, v, g, b, lengths, state, scale, do=None, ds=None):
    """Outputs and the bars' shares, by name.  q, k, v [B, T, heads, D], g, b [B, T, H] float64."""
    B, T = q.shape[:2]
    H = g.shape[2]
    rep = [H // t.shape[2] for t in (q, k, v)]
    Q, K, V = (np.repeat(t, r, axis=2) for t, r in zip((q, k, v), rep))
    Dk, Dv = Q.shape[3], V.shape[3]
    out = {n: np.zeros(s) for n, s in dict(o=V.shape, q=Q.shape, k=K.shape, v=V.shape, g=g.shape, b=g.shape,
                                           last=(B, H, Dk, Dv), state=(B, H, Dk, Dv)).items()}
    bar = {n: np.zeros(x.shape) for n, x in out.items()}
    for i in range(B):
        n = lengths[i]
        S = np.zeros((n + 1, H, Dk, Dv))
        m = np.zeros((n + 1, H, Dv))
        if state is not None:
            S[0] = state[i]
        a = np.exp(g[i])
        for t in range(n):
            old = a[t, :, None, None] * S[t]
            miss = V[i, t] - np.einsum("hi,hij->hj", K[i, t], old)
            S[t + 1] = old + b[i, t, :, None, None] * K[i, t][:, :, None] * miss[:, None, :]
            bt = np.abs(b[i, t, :, None])
            m[t + 1] = a[t, :, None] * (m[t] + (1 + bt) * norm(S[t], 1)) + bt * np.abs(V[i, t])
            out["o"][i, t] = scale * np.einsum("hi,hij->hj", Q[i, t], S[t + 1])
            bar["o"][i, t] = scale * norm(Q[i, t])[:, None] * (m[t + 1] + norm(S[t + 1], 1))
        out["last"][i], bar["last"][i] = S[n], (m[n] + norm(S[n], 1))[:, None, :]
        if do is None:
            continue
        D = ds[i].copy() if ds is not None else np.zeros((H, Dk, Dv))
        nn = np.zeros((H, Dv))
        for t in reversed(range(n)):
            w = scale * do[i, t]
            D = D + Q[i, t][:, :, None] * w[:, None, :]
            nn = nn + norm(D, 1) + norm(Q[i, t])[:, None] * np.abs(w)
            bt, kt = b[i, t, :, None], K[i, t]
            old = a[t, :, None, None] * S[t]
            miss = V[i, t] - np.einsum("hi,hij->hj", kt, old)
            said = np.einsum("hij,hj->hi", D, miss)
            dv = bt * np.einsum("hi,hij->hj", kt, D)
            out["q"][i, t] = np.einsum("hij,hj->hi", S[t + 1], w)
            out["k"][i, t] = bt * said - np.einsum("hij,hj->hi", old, dv)
            out["v"][i, t] = dv
            out["b"][i, t] = (kt * said).sum(-1)
            P = D - kt[:, :, None] * dv[:, None, :]
            out["g"][i, t] = (P * old).sum((1, 2))
            s, d, vv, mm = norm(S[t], 1), norm(D, 1), np.abs(V[i, t]), m[t] + m[t + 1]
            at = (nn * (s + vv) + d * (mm + s + vv)).sum(-1) * (1 + np.abs(b[i, t]))
            mine = (np.abs(w) * (mm + norm(S[t + 1], 1))).sum(-1)
            bar["q"][i, t] = mine[:, None]
            bar["k"][i, t] = (at + mine)[:, None]
            bar["v"][i, t] = np.abs(bt) * (nn + d)
            bar["b"][i, t] = at
            bar["g"][i, t] = at + mine
            D = a[t, :, None, None] * P
            nn = a[t, :, None] * (nn + (1 + np.abs(bt)) * d)
        for t0 in range(0, n, 64):
            bar["g"][i, t0:t0 + 64] = bar["g"][i, t0:t0 + 64].sum(0)
        out["g"][i][g[i] < -104] = 0
        out["state"][i], bar["state"][i] = D, (nn + norm(D, 1))[:, None, :]
    for r in (out, bar):
        for name, x, s in (("q", q, rep[0]), ("k", k, rep[1]), ("v", v, rep[2])):
            r[name] = r[name].reshape(B, T, x.shape[2], s, -1).sum(3)
    return out, bar


def draw(seed, B, T, heads, Dk, Dv, dtype, state=True):
    gen = torch.Generator().manual_seed(seed)
    H = max(heads)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    t = {"q": unit(torch.randn((B, T, heads[0], Dk), generator=gen)),
         "k": unit(torch.randn((B, T, heads[1], Dk), generator=gen)),
         "v": torch.randn((B, T, heads[2], Dv), generator=gen), "do": torch.randn((B, T, H, Dv), generator=gen)}
    t = {n: x.to(TYPES[dtype]) for n, x in t.items()}
    # the rounded keys may be a little longer than 1: no matter at beta below 1.9
    t["g"] = -torch.exp2(-9 * torch.rand((B, T, H), generator=gen))
    t["b"] = torch.sigmoid(torch.randn((B, T, H), generator=gen))
    t["state"] = torch.randn((B, H, Dk, Dv), generator=gen) if state else None
    t["ds"] = torch.randn((B, H, Dk, Dv), generator=gen)
    return t


def check(name, got, want, share, dtype, D):
    got = got.detach().float().cpu().double().numpy()
    assert got.shape == want.shape, name
    ulp = ULP[dtype] if name in ("o", "q", "k", "v") else ULP["f32"]
    off = np.abs(got - want)
    over = off - ((D + 128) * 2.0 ** -24 * share + ulp * np.abs(want) + 2.0 ** -25)
    assert np.all(over <= 0), (name, float(np.nanmax(over)), np.argwhere(~(over <= 0))[:4].tolist())
    size = np.linalg.norm(want)
    # of sums that cancel (a gradient of a shared head, a decay's) the norm says nothing
    if size > 1e-3 * np.linalg.norm(share):
        assert np.linalg.norm(got - want) <= (2.0 ** -18 + ulp) * size + 2.0 ** -25 * math.sqrt(want.size), (
            name, np.linalg.norm(got - want) / size)


def call(d, lt, scale=None):
    return encoder.gated_delta(d["q"], d["k"], d["v"], d["g"], d["b"], lengths=lt, state=d["state"],
                               scale=scale, return_state=True)


def compare(t, dtype, lengths=None, backward=True, views=None, scale=None):
    B, T, _, Dk = t["q"].shape
    d = {n: None if x is None else x.to(DEV) for n, x in t.items()}
    if views is not None:
        d.update(views(d))
    lens = [T] * B if lengths is None else lengths
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    wrt = [n for n in NAMES if d[n] is not None]
    if backward:
        for n in wrt:
            d[n].requires_grad_(True)
    o, last = call(d, lt, scale)
    assert o.dtype == TYPES[dtype] and last.dtype == torch.float32
    f = {n: None if x is None else x.double().numpy() for n, x in t.items()}
    want, bar = reference(f["q"], f["k"], f["v"], f["g"], f["b"], lens, f["state"],
                          Dk ** -0.5 if scale is None else scale, f["do"] if backward else None, f["ds"])
    got = dict(o=o, last=last)
    if backward:
        got.update(zip(wrt, torch.autograd.grad((o, last), [d[n] for n in wrt], (d["do"], d["ds"]))))
    D = max(Dk, t["v"].shape[3])
    for n, x in got.items():
        check(n, x, want[n], bar[n], dtype, D)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 97, 128, 130, 257])
def test_lengths_of_a_sequence(T, dtype):
    compare(draw(T, 2, T, (2, 2, 2), 64, 64, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Dk,Dv", [(1, 1), (3, 5), (16, 32), (33, 64), (64, 33), (40, 72), (96, 128),
                                   (128, 16), (128, 128), (8, 128), (65, 127)])
def test_widths(Dk, Dv, dtype):
    compare(draw(Dk, 2, 100, (2, 2, 2), Dk, Dv, dtype), dtype, lengths=[100, 71])


@pytest.mark.parametrize("heads", [(1, 1, 1), (4, 2, 2), (4, 1, 4), (2, 2, 6), (1, 3, 3), (6, 2, 3),
                                   (5, 5, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_heads(heads, dtype):
    compare(draw(3, 2, 70, heads, 24, 40, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_ragged_lengths_and_nan_past_them(dtype):
    B, T = 6, 150
    lengths = [150, 0, 1, 64, 65, 97]
    t = draw(5, B, T, (2, 2, 2), 32, 48, dtype)
    for b, n in enumerate(lengths):
        for name in ("q", "k", "v", "do", "g", "b"):
            t[name][b, n:] = 0
    compare(t, dtype, lengths=lengths)
    d = {n: x.to(DEV) for n, x in t.items()}
    lt = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    for n in NAMES:
        d[n].requires_grad_(True)
    first = call(d, lt)
    grads = torch.autograd.grad(first, [d[n] for n in NAMES], (d["do"], d["ds"]))
    with torch.no_grad():
        for b, n in enumerate(lengths):
            for name in ("q", "k", "v", "do", "g", "b"):
                d[name][b, n:] = math.nan
    again = call(d, lt)
    for x, y in zip((*first, *grads), (*again, *torch.autograd.grad(again, [d[n] for n in NAMES],
                                                                    (d["do"], d["ds"])))):
        assert torch.equal(x, y)
    for x in (again[0], *grads[:5]):
        for b, n in enumerate(lengths):
            assert not x[b, n:].any()


def test_invalid_lengths():
    t = draw(6, 3, 40, (2, 2, 2), 16, 16, "f32")
    d = {n: x.to(DEV) for n, x in t.items()}
    for n in NAMES:
        d[n].requires_grad_(True)
    lt = torch.tensor([41, 40, -1], dtype=torch.int32, device=DEV)
    o, last = call(d, lt)
    grads = torch.autograd.grad((o, last), [d[n] for n in NAMES], (d["do"], d["ds"]))
    alone = {n: x.detach()[1:2].clone().requires_grad_(n in NAMES) for n, x in d.items()}
    o1, last1 = call(alone, None)
    want = torch.autograd.grad((o1, last1), [alone[n] for n in NAMES], (alone["do"], alone["ds"]))
    for b in (0, 2):
        assert o[b].isnan().all() and last[b].isnan().all()
        assert all(not x[b].any() for x in grads)
    assert torch.equal(o[1:2], o1) and torch.equal(last[1:2], last1)
    assert all(torch.equal(x[1:2], y) for x, y in zip(grads, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gates", ["keep", "forget", "far", "none written", "all written", "reflected", "negative"])
def test_gates_at_their_ends(gates, dtype):
    """Decays of 1, 0 and below float32's range, writes of nothing, of everything (the state
    then says the value for the key) and past it."""
    t = draw(7, 2, 140, (2, 2, 2), 32, 32, dtype)
    if gates == "keep":
        t["g"] = torch.zeros_like(t["g"])
    elif gates == "forget":
        t["g"][:, ::7] = -math.inf
        t["g"][0, 64:70] = -math.inf
    elif gates == "far":
        t["g"][:, ::5] = -103.0
        t["g"][:, 2::5] = -1e30
    elif gates == "none written":
        t["b"][:, ::3] = 0.0
        t["b"][1] = 0.0
    elif gates == "all written":
        t["b"] = torch.ones_like(t["b"])
    elif gates == "reflected":
        t["b"] = torch.full_like(t["b"], 1.9)
    else:
        t["b"][:, ::2] *= -0.05
    compare(t, dtype)


def test_a_full_write_is_read_back():
    """beta = 1, no decay: right after its write a key reads its value."""
    gen = torch.Generator().manual_seed(2)
    k = torch.randn((1, 100, 1, 64), generator=gen)
    k = (k / k.norm(dim=-1, keepdim=True)).to(DEV)
    v = torch.randn((1, 100, 1, 64), generator=gen).to(DEV)
    ones = torch.ones((1, 100, 1), device=DEV)
    o = encoder.gated_delta(k, k, v, ones * 0, ones, scale=1.0)
    assert (o - v).abs().max() < 2.0 ** -16  # |k|^2 is off by 64 roundings, |S k| below 16


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_strided_inputs(dtype):
    """Slices of one packed tensor, rows of odd offsets, transposed heads."""
    B, T, H, D = 2, 75, 3, 40
    t = draw(8, B, T, (H, H, H), D, D, dtype)

    def packed(d):
        x = torch.cat([d[n] for n in "qkv"], dim=2)
        return dict(zip("qkv", x.split(H, dim=2)))

    def odd(d):
        x = torch.zeros((B, T, 3 * H, D + 3), dtype=TYPES[dtype], device=DEV)
        for i, n in enumerate("qkv"):
            x[:, :, i * H:(i + 1) * H, 1:D + 1] = d[n]
        return {n: x[:, :, i * H:(i + 1) * H, 1:D + 1] for i, n in enumerate("qkv")}

    def heads_first(d):
        return {n: d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "qkv"}

    def by_element(d):
        return {n: d[n].transpose(1, 3).contiguous().transpose(1, 3) for n in "qkv"}

    def gates(d):
        return {n: d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "gb"}
    for views in (packed, odd, heads_first, by_element, gates):
        compare(t, dtype, views=views)


def test_broadcast_inputs():
    """Expanded keys and queries: stride 0, gradients summed by autograd."""
    t = draw(9, 2, 50, (2, 2, 2), 16, 16, "f32")
    t["k"] = t["k"][:1, :, :1].expand(2, 50, 2, 16)
    k = t["k"][:1, :, :1].to(DEV).requires_grad_(True)
    d = {n: x.to(DEV) for n, x in t.items()}
    d["k"] = k.expand(2, 50, 2, 16)
    o, last = call(d, None)
    got, = torch.autograd.grad((o, last), k, (d["do"], d["ds"]))
    full = t["k"].contiguous().to(DEV).requires_grad_(True)
    d["k"] = full
    o1, last1 = call(d, None)
    want, = torch.autograd.grad((o1, last1), full, (d["do"], d["ds"]))
    assert torch.equal(o, o1) and torch.equal(last, last1)
    assert torch.allclose(got, want.sum((0, 2), keepdim=True), rtol=1e-6, atol=1e-6)


def recurrence(t, lengths=None):
    """o and the last state by torch on the GPU in float64, for long sequences."""
    q, k, v, g, b = (t[n].to(DEV).double() for n in ("q", "k", "v", "g", "b"))
    B, T, H = g.shape
    S = torch.zeros((B, H, q.shape[3], v.shape[3]), dtype=torch.float64, device=DEV)
    if t["state"] is not None:
        S = t["state"].to(DEV).double()
    a = g.exp()
    o = torch.empty((B, T, H, v.shape[3]), dtype=torch.float64, device=DEV)
    for i in range(T):
        S = S * a[:, i, :, None, None]
        miss = v[:, i] - (k[:, i, :, None] @ S)[:, :, 0]
        S = S + (b[:, i, :, None] * k[:, i])[..., None] * miss[:, :, None]
        o[:, i] = (q[:, i, :, None] @ S)[:, :, 0] * q.shape[3] ** -0.5
    return o, S


@pytest.mark.parametrize("dtype,B,T,D", [("f32", 1, 6000, 64), ("bf16", 1, 6000, 64), ("bf16", 3, 2300, 32),
                                         ("f16", 1, 4111, 128)])
def test_long_sequences(dtype, B, T, D):
    t = draw(10, B, T, (2, 2, 2), D, D, dtype)
    t["g"] = t["g"] * 0.02  # a memory of up to 25000 positions
    o, last = call({n: x.to(DEV) for n, x in t.items()}, None)
    want, state = recurrence(t)
    err = lambda x, y: float((x.double() - y).norm() / y.norm())  # noqa: E731
    assert err(o, want) < ULP[dtype] + 2.0 ** -18
    assert err(last, state) < 2.0 ** -18


def test_pieces_equal_the_whole():
    """A sequence in two calls with the state between them, forward and backward."""
    t = draw(11, 2, 200, (2, 2, 2), 32, 40, "f32")
    d = {n: x.to(DEV) for n, x in t.items()}
    for n in NAMES:
        d[n].requires_grad_(True)
    o, last = call(d, None)
    want = torch.autograd.grad((o, last), [d[n] for n in NAMES], (d["do"], d["ds"]))
    for cut in (1, 64, 77, 199):
        one = {n: x[:, :cut] if n not in ("state", "ds") else x for n, x in d.items()}
        two = {n: x[:, cut:] if n not in ("state", "ds") else x for n, x in d.items()}
        o1, s1 = call(one, None)
        o2, s2 = call({**two, "state": s1}, None)
        got = torch.autograd.grad((torch.cat((o1, o2), 1), s2), [d[n] for n in NAMES], (d["do"], d["ds"]))
        for x, y in zip((torch.cat((o1, o2), 1), s2, *got), (o, last, *want)):
            assert (x - y).norm() <= 2.0 ** -18 * y.norm(), cut


def test_gradients_against_differences():
    """Central differences of the float64 recurrence along random directions: the
    difference's own error is below 1e-8, so the float32 gradients' bar is 2^-18 of the product
    of norms."""
    t = draw(12, 1, 45, (2, 1, 2), 12, 20, "f32")
    f = {n: x.double().numpy() for n, x in t.items()}

    def loss(x):
        out, _ = reference(*(x[n] for n in ("q", "k", "v", "g", "b")), [45], x["state"], 12 ** -0.5)
        return (out["o"] * f["do"]).sum() + (out["last"] * f["ds"]).sum()
    d = {n: x.to(DEV) for n, x in t.items()}
    for n in NAMES:
        d[n].requires_grad_(True)
    o, last = call(d, None)
    grads = dict(zip(NAMES, torch.autograd.grad((o, last), [d[n] for n in NAMES], (d["do"], d["ds"]))))
    rng = np.random.default_rng(0)
    for n in NAMES:
        way = rng.standard_normal(f[n].shape)
        h = 1e-5
        want = (loss({**f, n: f[n] + h * way}) - loss({**f, n: f[n] - h * way})) / (2 * h)
        got = grads[n].double().cpu().numpy()
        assert abs((got * way).sum() - want) <= 2.0 ** -18 * np.linalg.norm(got) * np.linalg.norm(way) + 1e-6, n


def test_only_what_is_asked_for():
    t = draw(13, 2, 70, (2, 1, 2), 16, 24, "bf16")
    d = {n: x.to(DEV) for n, x in t.items()}
    full = {n: x.clone().requires_grad_(n in NAMES) for n, x in d.items()}
    o, last = call(full, None)
    want = dict(zip(NAMES, torch.autograd.grad((o, last), [full[n] for n in NAMES], (d["do"], d["ds"]))))
    for n in NAMES:
        some = {m: x.clone().requires_grad_(m == n) for m, x in d.items()}
        o, last = call(some, None)
        got, = torch.autograd.grad((o, last), some[n], (d["do"], d["ds"]))
        assert torch.equal(got, want[n]), n
    some = {m: x.clone().requires_grad_(m in NAMES) for m, x in d.items()}
    o, last = call(some, None)
    by_state = torch.autograd.grad(last, [some[n] for n in NAMES], d["ds"], retain_graph=True)
    by_o = torch.autograd.grad(o, [some[n] for n in NAMES], d["do"])
    for n, x, y in zip(NAMES, by_state, by_o):
        assert (x.float() + y.float() - want[n].float()).norm() <= 2.0 ** -7 * (x.float().norm() + y.float().norm()), n


def test_empty_calls_carry_gradients():
    q = torch.zeros((2, 0, 2, 8), device=DEV, dtype=torch.bfloat16, requires_grad=True)
    g = torch.zeros((2, 0, 2), device=DEV, requires_grad=True)
    o, last = encoder.gated_delta(q, q, q, g, g, return_state=True)
    assert o.shape == (2, 0, 2, 8) and last.shape == (2, 2, 8, 8) and not last.any()
    (o.float().sum() + last.sum()).backward()
    assert q.grad.shape == q.shape and g.grad.shape == g.shape
    s = torch.ones((2, 2, 8, 8), device=DEV, requires_grad=True)
    lt = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    last = encoder.gated_delta(q, q, q, g, g, state=s, lengths=lt, return_state=True)[1]
    assert last[1].isnan().all() and (last[0] == 1).all()
    none = torch.zeros((0, 4, 2, 8), device=DEV)
    assert encoder.gated_delta(none, none, none, none[..., 0], none[..., 0]).shape == (0, 4, 2, 8)


def test_other_stream_and_graph():
    """A call on a stream of its own, and forward and backward captured: replays follow the inputs."""
    t = draw(14, 2, 300, (2, 2, 2), 64, 64, "bf16")
    d = {n: x.to(DEV) for n, x in t.items()}
    want = call(d, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call(d, None)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

    def step(d):
        leaves = {n: d[n].detach().requires_grad_(True) for n in NAMES}
        o, last = call({**d, **leaves}, None)
        return o.detach(), last.detach(), *torch.autograd.grad((o, last), list(leaves.values()), (d["do"], d["ds"]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(d)
    for i in range(3):
        d["v"].copy_(torch.randn_like(d["v"]))
        d["do"].copy_(torch.randn_like(d["do"]))
        want = step({n: x.clone() for n, x in d.items()})
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), i


def test_two_captured_graphs_do_not_share_memory():
    t = [draw(15 + i, 2, 200, (2, 2, 2), 32, 32, "f32") for i in range(2)]
    d = [{n: x.to(DEV) for n, x in s.items()} for s in t]
    want = [call(x, None) for x in d]
    graphs, got = [], []
    for x in d:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(call(x, None))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_the_same_result_every_time():
    t = draw(17, 3, 500, (4, 2, 1), 64, 64, "bf16")
    d = {n: x.to(DEV) for n, x in t.items()}
    for n in NAMES:
        d[n].requires_grad_(True)
    runs = []
    for _ in range(3):
        o, last = call(d, None)
        runs.append((o, last, *torch.autograd.grad((o, last), [d[n] for n in NAMES], (d["do"], d["ds"]))))
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, runs[0]))


def test_offsets_past_32_bits():
    """Batch rows 2^32 elements apart."""
    far = (1 << 32) + 64
    big = torch.empty(far + 70 * 2 * 16, dtype=torch.bfloat16, device=DEV)
    t = draw(18, 2, 70, (2, 2, 2), 16, 16, "bf16")

    def views(d):
        v = big.as_strided((2, 70, 2, 16), (far, 32, 16, 1))
        v.copy_(d["v"])
        return {"v": v}
    compare(t, "bf16", backward=False, views=views)
    del big
    torch.cuda.empty_cache()


def test_second_derivatives_are_refused():
    t = draw(19, 1, 20, (1, 1, 1), 8, 8, "f32")
    d = {n: x.to(DEV).requires_grad_(n in NAMES) for n, x in t.items()}
    o, _ = call(d, None)
    g, = torch.autograd.grad(o.square().sum(), d["k"], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.square().sum().backward()


# ---- single positions ------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,Dk,Dv", [((4, 4, 4), 64, 64), ((2, 2, 2), 128, 128), ((4, 2, 2), 40, 72),
                                         ((1, 3, 3), 5, 7), ((2, 2, 2), 128, 127), ((2, 2, 2), 33, 4),
                                         ((1, 1, 1), 1, 1), ((2, 2, 2), 127, 1)])
def test_step(heads, Dk, Dv, dtype):
    B, N, H = 5, 9, max(heads)
    t = draw(20, B, 1, heads, Dk, Dv, dtype, False)
    pool = torch.randn((N, H, Dk, Dv), generator=torch.Generator().manual_seed(1))
    slots = [7, -1, 0, 9, 3]  # the second and the fourth are idle
    d = {n: x[:, 0].to(DEV) for n, x in t.items() if n in "qkvgb"}
    state = pool.to(DEV)
    o = encoder.gated_delta_step(d["q"], d["k"], d["v"], d["g"], d["b"], state,
                                 slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    for b, s in enumerate(slots):
        if not 0 <= s < N:
            assert (o[b] == 0).all()
            continue
        f = [t[n][b:b + 1].double().numpy() for n in "qkvgb"]
        want, bar = reference(*f, [1], pool[s:s + 1].double().numpy(), Dk ** -0.5)
        check("o", o[b:b + 1, None], want["o"], bar["o"], dtype, max(Dk, Dv))
        check("last", state[s:s + 1], want["last"], bar["last"], dtype, max(Dk, Dv))
    others = [i for i in range(N) if i not in slots]
    assert torch.equal(state[others].cpu(), pool[others])


def test_steps_follow_the_whole_sequence():
    t = draw(21, 3, 90, (2, 2, 2), 32, 48, "f32", False)
    d = {n: x.to(DEV) for n, x in t.items() if x is not None}
    o, last = encoder.gated_delta(d["q"], d["k"], d["v"], d["g"], d["b"], return_state=True)
    state = torch.zeros((3, 2, 32, 48), device=DEV)
    for i in range(90):
        x = encoder.gated_delta_step(*(d[n][:, i] for n in "qkvgb"), state)
        assert (x - o[:, i]).norm() <= 2.0 ** -18 * o[:, i].norm(), i
    assert (state - last).norm() <= 2.0 ** -18 * last.norm()


def test_slow_decays_over_many_steps():
    """A state that is only read: S_n = e^{g n} S_0.  Two roundings of 2^-24 a step without a sign: 6
    sqrt(2 n) 2^-24 of it; e^g as one float32 would add up to n 2^-25."""
    n, H = 5000, 12
    g = torch.tensor([[-1.0 / (700 + 100 * i) for i in range(H)]])
    s0 = 1 + torch.rand((1, H, 8, 8), generator=torch.Generator().manual_seed(3))
    q = torch.zeros((1, H, 8), device=DEV)
    state, gd = s0.to(DEV), g.to(DEV)
    for _ in range(n):
        encoder.gated_delta_step(q, q, q, gd, gd * 0, state)
    want = s0.double() * torch.exp(g.double() * n)[..., None, None]
    assert ((state.cpu().double() - want).abs() <= 6 * math.sqrt(2 * n) * 2.0 ** -24 * want).all()


def test_slow_decays_over_a_long_sequence():
    """The same over the chunks of one sequence."""
    T = 1 << 17
    g = torch.full((1, T, 2), -1.0 / (1 << 15))
    g[..., 1] = -1.0 / 50000
    s0 = 1 + torch.rand((1, 2, 8, 8), generator=torch.Generator().manual_seed(4))
    q = torch.zeros((1, T, 2, 8), device=DEV)
    last = encoder.gated_delta(q, q, q, g.to(DEV), torch.zeros_like(g).to(DEV), state=s0.to(DEV),
                               return_state=True)[1]
    want = s0.double() * torch.exp(g.double().sum(1))[..., None, None]
    # two roundings a chunk of 32 positions
    assert ((last.cpu().double() - want).abs() <= 6 * math.sqrt(2 * T / 32) * 2.0 ** -24 * want).all()


def test_a_step_is_seen_by_autograd():
    q, k, v = (torch.randn((1, 5, 2, 4), device=DEV, requires_grad=True) for _ in range(3))
    gate = torch.full((1, 5, 2), -0.1, device=DEV, requires_grad=True)
    pool = torch.zeros((1, 2, 4, 4), device=DEV)
    read = q[:, 0].detach()[..., None].requires_grad_(True) * pool
    with torch.no_grad():
        encoder.gated_delta_step(q[:, 0], k[:, 0], v[:, 0], gate[:, 0], -gate[:, 0], pool)
    with pytest.raises(RuntimeError, match="inplace operation"):
        read.sum().backward()
    for t in (q, gate):
        args = [x.detach() for x in (q[:, 0], k[:, 0], v[:, 0], gate[:, 0], -gate[:, 0])]
        args[0 if t is q else 3] = t[:, 0]
        with pytest.raises(RuntimeError, match="no gradients"):
            encoder.gated_delta_step(*args, pool).sum().backward()


def test_steps_on_another_stream_and_in_a_graph():
    t = draw(22, 4, 1, (2, 2, 2), 64, 64, "bf16", False)
    d = {n: t[n][:, 0].to(DEV) for n in "qkvgb"}
    pool = torch.randn((4, 2, 64, 64), device=DEV)
    want_pool = pool.clone()
    want = encoder.gated_delta_step(*(d[n] for n in "qkvgb"), want_pool)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got_pool = pool.clone()
        got = encoder.gated_delta_step(*(d[n] for n in "qkvgb"), got_pool)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want) and torch.equal(got_pool, want_pool)
    held = pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = encoder.gated_delta_step(*(d[n] for n in "qkvgb"), held)
    held.copy_(pool)
    for i in range(3):
        want = encoder.gated_delta_step(*(d[n] for n in "qkvgb"), pool)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(held, pool), i


def test_many_short_sequences():
    """2^20 sequences and heads of one position: o = scale (q . k) b v, and a state in."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    B, H, D = 1 << 18, 4, 8
    q, k, v = (torch.randn((B, 1, H, D), device=DEV, generator=gen) for _ in range(3))
    k = k / k.norm(dim=-1, keepdim=True)
    g, b = -torch.rand((B, 1, H), device=DEV, generator=gen), torch.rand((B, 1, H), device=DEV, generator=gen)
    o, last = encoder.gated_delta(q, k, v, g, b, return_state=True)
    d = [t.double() for t in (q, k, v, b)]
    want = D ** -0.5 * (d[0] * d[1]).sum(-1, keepdim=True) * d[3][..., None] * d[2]
    assert ((o - want).abs() <= 64 * 2.0 ** -24 * (q.norm(dim=-1, keepdim=True) * v.abs())).all()
    want = d[3][:, 0, :, None, None] * d[1][:, 0, :, :, None] * d[2][:, 0, :, None, :]
    assert ((last - want).abs() <= 8 * 2.0 ** -24 * want.abs() + 2.0 ** -40).all()


def test_infinities_in_what_is_masked():
    """Infinite values past the lengths, and keys of 0 with infinite queries there."""
    t = draw(23, 2, 80, (2, 2, 2), 32, 32, "bf16")
    d = {n: x.to(DEV) for n, x in t.items()}
    lt = torch.tensor([33, 64], dtype=torch.int32, device=DEV)
    want = call(d, lt)
    for b, n in enumerate([33, 64]):
        for name in ("q", "k", "v"):
            d[name][b, n:] = math.inf
        d["g"][b, n:], d["b"][b, n:] = math.inf, -math.inf
    got = call(d, lt)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_over_segments(dtype):
    """One sequence of few heads, cut into segments on the way: against the same in pieces of
    64 positions, one segment each, tied by autograd."""
    t = draw(24, 1, 1500, (1, 1, 1), 48, 40, dtype)
    d = {n: x.to(DEV) for n, x in t.items()}
    for n in NAMES:
        d[n].requires_grad_(True)
    o, last = call(d, None)
    got = torch.autograd.grad((o, last), [d[n] for n in NAMES], (d["do"], d["ds"]))
    parts, s = [], d["state"]
    for i in range(0, 1500, 64):
        x, s = call({**{n: y if n in ("state", "ds") else y[:, i:i + 64] for n, y in d.items()}, "state": s}, None)
        parts.append(x)
    x = torch.cat(parts, 1)
    want = torch.autograd.grad((x, s), [d[n] for n in NAMES], (d["do"], d["ds"]))
    tol = 2.0 ** -18 if dtype == "f32" else 2.0 ** -18 + 2 * ULP["bf16"]
    for n, a, b in zip(("o", "last", *NAMES), (o, last, *got), (x, s, *want)):
        assert (a.float() - b.float()).norm() <= tol * b.float().norm(), n


def test_refusals():
    x = torch.zeros((2, 5, 2, 8), device=DEV)
    g = torch.zeros((2, 5, 2), device=DEV)
    wide = torch.zeros((2, 5, 2, 129), device=DEV)
    for args, kw in (((x, x, wide, g, g), {}), ((wide, wide, x, g, g), {}), ((x, x[:, :4], x, g, g), {}),
                     ((x, x.half(), x, g, g), {}), ((x, x, x, g[..., :1], g), {}), ((x, x, x, g, g.half()), {}),
                     ((x, x, x, g.cpu(), g), {}), ((x.double(), x.double(), x.double(), g, g), {}),
                     ((x, x, x[:, :, :1].expand(2, 5, 3, 8), g, g), {}),
                     ((x, x, x, g, g), dict(state=torch.zeros((2, 2, 8, 7), device=DEV))),
                     ((x, x, x, g, g), dict(lengths=torch.zeros(2, device=DEV)))):
        with pytest.raises(ValueError):
            encoder.gated_delta(*args, **kw)
    pool = torch.zeros((3, 2, 8, 8), device=DEV)
    one = x[:, 0], x[:, 0], x[:, 0], g[:, 0], g[:, 0]
    for args, kw in (((*one, pool[:, :1]), {}), ((*one, pool.half()), {}), ((*one, pool.transpose(2, 3)), {}),
                     ((*one[:4], g, pool), {}), ((*one, pool), dict(slots=torch.zeros(2, device=DEV))),
                     ((*one, pool.clone().requires_grad_(True)), {})):
        with pytest.raises(ValueError):
            encoder.gated_delta_step(*args, **kw)
    assert not pool.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("beta", [1.0, 1.95])
def test_the_same_key_all_along(dtype, beta):
    """Writes that undo each other: the triangles' inverses have entries that alternate
    with hardly a decay."""
    t = draw(25, 1, 200, (2, 2, 2), 32, 32, dtype)
    t["k"] = t["k"][:, :1].expand(1, 200, 2, 32).contiguous()
    t["g"] = t["g"] * 1e-3
    t["b"] = torch.full_like(t["b"], beta)
    compare(t, dtype)
