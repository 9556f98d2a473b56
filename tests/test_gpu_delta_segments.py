"""The gated delta rule over segments: shapes that the library does cut, as the size of its workspace
shows, against the recurrence in float64.

Bars as in test_gpu_delta.py, with one thing more: what a segment makes of the state before it is a
product with a Dk x Dk matrix phi.  Each column of phi is walked like a column of a state of norm 1
and is off by w m, so phi S is off by w m sum_j |S_j| <= w m sqrt(Dk) |S|: each element's bar is
1 + sqrt(Dk) times the walk's.  The bar of a whole output stays: 2^-18 of its norm and its
rounding."""
import ctypes
import math

import numpy as np
import pytest
import torch

from semi_markov_crf_zero_amd import encoder
from tests.test_gpu_delta import DEV, NAMES, TYPES, ULP, call, draw, reference

pytestmark = pytest.mark.gpu


def cut(t, dtype):
    """Segments, and positions of one: from the parts of the workspace that a call in one segment
    lacks."""
    B, T, H = t["g"].shape
    dims = (B, T, H, *(t[n].shape[2] for n in "qkv"), t["k"].shape[3], t["v"].shape[3])
    n = ctypes.c_size_t(0)
    s = encoder._LinattnShape(*dims, encoder.DTYPES[TYPES[dtype]], 1.0)
    assert encoder.load().semicrf_delta_workspace_size(ctypes.byref(s), 0, ctypes.byref(n)) == 0
    L = 64 if dtype == "bf16" else 32
    chunks = -(-T // L)
    area = lambda n: (4 * n + 255) // 256 * 256  # noqa: E731
    up = lambda n: -(-n // 4) * 4  # noqa: E731
    left = n.value - area(B * H * chunks * L * L) - area(B * H * chunks * (4 * L + 4))
    for nseg in range(2, chunks + 1):
        if left == area(B * H * nseg * dims[6] * up(dims[6])) + area(B * H * nseg * dims[6] * up(dims[7])):
            return nseg, -(-chunks // nseg) * L
    assert left == 0
    return 1, T


def check(name, got, want, share, dtype, Dk, Dv):
    got = got.detach().float().cpu().double().numpy()
    assert got.shape == want.shape, name
    ulp = ULP[dtype] if name in ("o", "q", "k", "v") else ULP["f32"]
    bar = (1 + math.sqrt(Dk)) * (max(Dk, Dv) + 128) * 2.0 ** -24 * share
    over = np.abs(got - want) - (bar + ulp * np.abs(want) + 2.0 ** -25)
    assert np.all(over <= 0), (name, float(np.nanmax(over)), np.argwhere(~(over <= 0))[:4].tolist())
    size = np.linalg.norm(want)
    if size > 1e-3 * np.linalg.norm(share):
        assert np.linalg.norm(got - want) <= (2.0 ** -18 + ulp) * size + 2.0 ** -25 * math.sqrt(want.size), (
            name, np.linalg.norm(got - want) / size)


def compare(t, dtype, lengths=None, views=None, ds=True):
    """Forward and backward; lengths outside [0, T]: NaN and gradients of 0."""
    B, T, _, Dk = t["q"].shape
    Dv = t["v"].shape[3]
    assert cut(t, dtype)[0] > 1
    d = {n: None if x is None else x.to(DEV) for n, x in t.items()}
    lt, bad, lens = None, [], [T] * B
    if lengths is not None:
        lt = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        bad = [b for b, n in enumerate(lengths) if not 0 <= n <= T]
        lens = [n if 0 <= n <= T else 0 for n in lengths]
        for b, n in enumerate(lens):
            for name in ("q", "k", "v", "do", "g", "b"):
                d[name][b, n:] = math.nan
    if views is not None:
        d.update(views(d))
    wrt = [n for n in NAMES if d[n] is not None]
    for n in wrt:
        d[n].requires_grad_(True)
    o, last = call(d, lt)
    f = {n: None if x is None else x.double().numpy() for n, x in t.items()}
    if not ds:
        f["ds"] = np.zeros((B, t["g"].shape[2], Dk, Dv))
    want, bar = reference(f["q"], f["k"], f["v"], f["g"], f["b"], lens, f["state"], Dk ** -0.5, f["do"], f["ds"])
    back = torch.autograd.grad((o, last) if ds else o, [d[n] for n in wrt], (d["do"], d["ds"]) if ds else d["do"])
    got = dict(zip(("o", "last", *wrt), (o, last, *back)))
    good = [b for b in range(B) if b not in bad]
    for n, x in got.items():
        check(n, x[good], want[n][good], bar[n][good], dtype, Dk, Dv)
        for b in bad:
            assert x[b].isnan().all() if n in ("o", "last") else not x[b].any(), n
        if n not in ("last", "state"):
            for b in good:
                assert not x[b, lens[b]:].any(), n
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("state", [True, False])
def test_lengths_that_end_anywhere(state, dtype):
    """Inside a segment, at its edge, before it, nowhere and past the end; NaN behind them."""
    t = draw(41, 10, 700, (2, 2, 2), 32, 48, dtype, state)
    nseg, seg = cut(t, dtype)
    assert nseg > 3 and 2 * seg + 1 < 700
    compare(t, dtype, [700, 0, 1, 2 * seg - 1, 2 * seg, 2 * seg + 1, -1, 701, seg, 2 * seg + 40])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Dk,Dv", [(33, 65), (65, 127), (96, 72), (96, 32), (128, 16), (128, 128), (3, 5), (8, 128),
                                   (64, 80)])
def test_widths(Dk, Dv, dtype):
    """Columns of phi past the values' and the other way round, rows that are padded to fours, every number
    of waves."""
    compare(draw(Dk, 1, 650, (2, 2, 2), Dk, Dv, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads", [(4, 2, 1), (1, 3, 3), (2, 1, 2)])
def test_shared_heads(heads, dtype):
    compare(draw(42, 2, 600, heads, 24, 40, dtype), dtype, [600, 411])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_read_by_element(dtype):
    B, T, H, D = 1, 600, 2, 40

    def odd(d):
        x = torch.zeros((B, T, 3 * H, D + 3), dtype=TYPES[dtype], device=DEV)
        for i, n in enumerate("qkv"):
            x[:, :, i * H:(i + 1) * H, 1:D + 1] = d[n]
        return {n: x[:, :, i * H:(i + 1) * H, 1:D + 1] for i, n in enumerate("qkv")}

    def heads_first(d):
        return {n: d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "qkv"}
    for views in (odd, heads_first):
        compare(draw(43, B, T, (H, H, H), D, D, dtype), dtype, views=views)


@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_gradient_of_the_last_state(dtype, state):
    compare(draw(44, 1, 650, (2, 2, 2), 72, 40, dtype, state), dtype, ds=False)


@pytest.mark.parametrize("gates", ["keep", "forget", "none written", "reflected"])
def test_gates_at_their_ends(gates):
    t = draw(45, 2, 700, (2, 2, 2), 40, 32, "f32")
    if gates == "keep":
        t["g"] = torch.zeros_like(t["g"])
    elif gates == "forget":
        t["g"][:, ::97] = -math.inf
        t["g"][0, 250:400] = -math.inf
    elif gates == "none written":
        t["b"][:, ::3] = 0.0
        t["b"][1] = 0.0
    else:
        t["b"] = torch.full_like(t["b"], 1.9)
    compare(t, "f32")


def test_captured():
    """Forward and backward over segments, replayed with other inputs between eager calls."""
    t = draw(46, 2, 700, (2, 2, 1), 96, 64, "bf16")
    assert cut(t, "bf16")[0] > 1
    d = {n: x.to(DEV) for n, x in t.items()}
    lt = torch.tensor([700, 333], dtype=torch.int32, device=DEV)

    def step(d, lt):
        leaves = {n: d[n].detach().requires_grad_(True) for n in NAMES}
        o, last = call({**d, **leaves}, lt)
        return o.detach(), last.detach(), *torch.autograd.grad((o, last), list(leaves.values()), (d["do"], d["ds"]))
    step(d, lt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(d, lt)
    for i, n in enumerate((700, 128, 0)):
        d["v"].copy_(torch.randn_like(d["v"]))
        d["do"].copy_(torch.randn_like(d["do"]))
        lt[1] = n
        want = step({m: x.clone() for m, x in d.items()}, lt.clone())
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), i
