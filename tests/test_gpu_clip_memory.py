"""Clipping: which gradients share memory."""
import pytest
import torch

from semi_markov_crf_zero_amd import optim

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def params(*grads):
    out = []
    for g in grads:
        p = torch.zeros(g.shape, dtype=g.dtype, device=DEV, requires_grad=True)
        p.grad = g
        out.append(p)
    return out


def test_empty_gradients_share_nothing():
    """Two without elements, both at address 0, beside one that is not contiguous: the norm of ones is
    the root of their number, and 0.5 over it is exact for 64 of them (the 1e-6 aside, 2^-22)."""
    turned = torch.ones((4, 16), device=DEV).t()
    assert not turned.is_contiguous()
    norm = optim.clip_grad_norm_(params(torch.zeros(0, device=DEV), turned, torch.zeros((3, 0), device=DEV)), 0.5)
    assert float(norm) == 8.0
    assert ((turned - 0.5 / (8.0 + 1e-6)).abs() <= 2.0 ** -22 / 16).all()
