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


def test_overlaps_of_any_layout_are_refused():
    flat = torch.ones(600, device=DEV)
    m = flat.view(20, 30)
    for grads in ((m[:, :3], m[:, 2:5]), (m, m[:, 1:3]), (m[::2], m[:1]), (m.t(), m[3]),
                  (flat.as_strided((3, 4), (2, 3)), m[0]), (m[:, 7], flat[187:200]), (m[:, ::2], m[:, ::3])):
        ps = params(*grads)
        with pytest.raises(ValueError, match="twice"):
            optim.clip_grad_norm_(ps, 1.0)
    for g in (flat[:4].expand(3, 4), flat.as_strided((5, 4), (2, 1)), flat.as_strided((1000, 600), (0, 1))):
        with pytest.raises(ValueError, match="twice"):
            optim.clip_grad_norm_(params(g), 1.0)
    assert (flat == 1).all()


def test_neighbours_that_interlock_are_clipped():
    """Columns of one matrix, every other row, dimensions whose strides cross: each element once.
    600 ones in all, a norm of sqrt(600): 2^-22 of a coefficient."""
    flat = torch.ones(600, device=DEV)
    m = flat[:594].view(18, 33)
    grads = m[:, :3], m[:, 3:20:2], m[:, 4:20:2], m[::2, 20:], m[1::2, 20:].t(), flat[594:].as_strided((2, 3), (3, 1))
    norm = optim.clip_grad_norm_(params(*grads), 1.0)
    assert abs(float(norm) - 600 ** 0.5) <= 2.0 ** -23 * 600 ** 0.5
    want = 1.0 / (600 ** 0.5 + 1e-6)
    assert ((flat.double() - want).abs() <= 2.0 ** -22 * want).all()
    crossed = torch.ones(8, device=DEV)  # strides 3 and 2 reach elements 0 2 3 4 5 7
    norm = optim.clip_grad_norm_(params(crossed.as_strided((2, 3), (3, 2))), 1.0)
    assert abs(float(norm) - 6 ** 0.5) <= 2.0 ** -23 * 6 ** 0.5
    assert ((crossed == 1).nonzero().flatten().cpu() == torch.tensor([1, 6])).all()
