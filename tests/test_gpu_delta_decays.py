"""Gradients of strong decays, which are as small as the decays themselves.

d g_t is the product of the decayed state before position t with the gradient of that state: all that
comes from before t times all that asks from t on, each term with the factor a = e^(g_t).  So is its bar: with m, n, S
and D as in test_gpu_delta.py, before t and after it,
    a (sum_c n_c (m_c + |S_c|) + |D_c| m_c) (1 + b)
of w = (D + 128) 2^-24, over segments 1 + sqrt(Dk) times it: and nothing absolute but float32's least number."""
import math

import numpy as np
import pytest
import torch

from semi_markov_crf_zero_amd import encoder
from tests.test_gpu_delta import DEV, NAMES, call, draw, norm

pytestmark = pytest.mark.gpu


def decays(t, lengths):
    """d g and its bar in float64."""
    q, k, v, g, b, do, state, ds = (None if t[n] is None else t[n].double().numpy()
                                    for n in ("q", "k", "v", "g", "b", "do", "state", "ds"))
    H = g.shape[2]
    q, k, v = (np.repeat(x, H // x.shape[2], axis=2) for x in (q, k, v))
    w = do * q.shape[3] ** -0.5
    out, bar = np.zeros(g.shape), np.zeros(g.shape)
    for i, n in enumerate(lengths):
        S, m, a = np.zeros((n + 1, *ds.shape[1:])), np.zeros((n + 1, H, v.shape[3])), np.exp(g[i])
        S[0] = state[i] if state is not None else 0
        for s in range(n):
            old = a[s, :, None, None] * S[s]
            bt, kt = b[i, s, :, None], k[i, s]
            S[s + 1] = old + (bt * kt)[:, :, None] * (v[i, s] - np.einsum("hi,hij->hj", kt, old))[:, None, :]
            m[s + 1] = a[s, :, None] * (m[s] + (1 + bt) * norm(S[s], 1)) + bt * np.abs(v[i, s])
        D, nn = ds[i].copy(), np.zeros((H, v.shape[3]))
        for s in reversed(range(n)):
            D = D + q[i, s][:, :, None] * w[i, s][:, None, :]
            nn = nn + norm(D, 1) + norm(q[i, s])[:, None] * np.abs(w[i, s])
            bt, kt = b[i, s, :, None], k[i, s]
            P = D - kt[:, :, None] * (bt * np.einsum("hi,hij->hj", kt, D))[:, None, :]
            out[i, s] = a[s] * (P * S[s]).sum((1, 2))
            bar[i, s] = a[s] * (nn * (m[s] + norm(S[s], 1)) + norm(D, 1) * m[s]).sum(-1) * (1 + b[i, s])
            nn = a[s, :, None] * (nn + (1 + bt) * norm(D, 1))
            D = a[s, :, None, None] * P
    return out, bar


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,heads,Dk,Dv", [(1, (2, 2, 2), 32, 48), (40, (2, 1, 2), 64, 64), (200, (2, 2, 2), 64, 64),
                                           (150, (2, 2, 2), 33, 20), (150, (1, 2, 2), 128, 96), (130, (2, 2, 2), 90, 72),
                                           (700, (2, 2, 2), 40, 72)])
@pytest.mark.parametrize("strong", ["some", "most", "the first", "the last"])
def test_gradients_of_strong_decays(strong, T, heads, Dk, Dv, dtype):
    t = draw(51, 2, T, heads, Dk, Dv, dtype)
    if strong == "some":
        t["g"][:, ::11], t["g"][:, 5::11] = -30.0, -60.0
    elif strong == "most":
        t["g"] = torch.where(torch.arange(T)[None, :, None] % 5 == 0, t["g"], t["g"] * 20)
    elif strong == "the first":
        t["g"][:, :1] = -40.0
    else:
        t["g"][:, -1:] = -40.0
    lengths = [T, (T + 1) // 2]
    d = {n: x.to(DEV).requires_grad_(n in NAMES) for n, x in t.items()}
    o, last = call(d, torch.tensor(lengths, dtype=torch.int32, device=DEV))
    got, = torch.autograd.grad((o, last), d["g"], (d["do"], d["ds"]))
    want, share = decays(t, lengths)
    bar = (1 + math.sqrt(Dk) * (T > 500)) * (max(Dk, Dv) + 128) * 2.0 ** -24 * share + 2.0 ** -126
    off = np.abs(got.double().cpu().numpy() - want) - bar
    assert np.all(off <= 0), (float(off.max()), np.argwhere(~(off <= 0))[:4].tolist())


def test_a_reset_has_no_gradient_but_its_own():
    """A decay of e^-50 between two halves: e^-50 of products of states and their gradients, of
    64 x 32 elements below 2^4 and 2^4 each, and nothing of the halves' own terms."""
    t = draw(52, 1, 120, (2, 2, 2), 32, 32, "f32")
    t["g"][:, 60] = -50.0
    d = {n: x.to(DEV).requires_grad_(n == "g") for n, x in t.items()}
    o, last = encoder.gated_delta(*(d[n] for n in "qkvgb"), state=d["state"], return_state=True)
    got, = torch.autograd.grad((o, last), d["g"], (d["do"], d["ds"]))
    assert float(got[:, 60].abs().max()) <= math.exp(-50) * 2.0 ** 19
