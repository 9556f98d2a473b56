"""Host-side checks of the layer's operators (no GPU): exports, argument
errors returned before any launch, and the refusals of the Python entry points."""
import ctypes
import os
import re

import pytest
import torch

from semi_markov_crf_zero_amd import encoder, optim

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "semicrf_layer.h")
P = ctypes.c_void_p(0x1000)  # never dereferenced: every call fails validation


@pytest.fixture(scope="module")
def lib():
    encoder.load()
    return optim.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(semicrf_[a-z_0-9]+)\s*\(", text))
    assert names == set(encoder.LAYER_EXPORTS) | set(optim.LAYER_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def shape(**kw):
    d = dict(B=2, T=5, H=4, Hq=4, Hk=2, Hv=1, Dk=8, Dv=6, dtype=1, scale=1.0)
    d.update(kw)
    s = encoder._LinattnShape()
    for k, v in d.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 2), (dict(T=0), 2), (dict(H=0), 2), (dict(Hq=3), 2), (dict(Hk=8), 2), (dict(Hv=0), 2),
    (dict(Dk=0), 2), (dict(Dv=0), 2), (dict(Dk=129), 3), (dict(Dv=300), 3), (dict(dtype=3), 6),
    (dict(dtype=-1), 6), (dict(B=1 << 28), 2), (dict(T=(1 << 30) + 1), 2), (dict(T=1 << 29), 2),
])
def test_delta_shapes_refused(lib, kw, code):
    s, n = shape(**kw), ctypes.c_size_t(0)
    r = ctypes.byref(s)
    assert lib.semicrf_delta_workspace_size(r, 0, ctypes.byref(n)) == code
    assert lib.semicrf_delta_fwd(r, 0, P, P, P, P, P, None, None, P, None, P, 1 << 60, None) == code
    assert lib.semicrf_delta_bwd(r, P, P, P, P, P, None, P, P, None, P, P, P, P, P, None, P, 1 << 60,
                                 None) == code


def test_delta_null_and_workspace(lib):
    s, n = shape(), ctypes.c_size_t(0)
    r = ctypes.byref(s)
    assert lib.semicrf_delta_workspace_size(r, 1, None) == 1
    assert lib.semicrf_delta_workspace_size(None, 1, ctypes.byref(n)) == 1
    assert lib.semicrf_delta_workspace_size(r, 3, ctypes.byref(n)) == 6
    for way in (0, 1, 2):
        assert lib.semicrf_delta_workspace_size(r, way, ctypes.byref(n)) == 0 and n.value > 0
    for i in (0, 1, 2, 3, 4, 7):
        a = [P, P, P, P, P, None, None, P, None]
        a[i] = None
        assert lib.semicrf_delta_fwd(r, 1, *a, P, 1 << 40, None) == 1
    for i in (0, 1, 2, 3, 4, 6, 7):
        b = [P, P, P, P, P, None, P, P, None, P, P, P, P, P, P]
        b[i] = None
        assert lib.semicrf_delta_bwd(r, *b, P, 1 << 40, None) == 1
    b = [P, P, P, P, P, None, P, P, None, P, P, P, P, P, P]
    assert lib.semicrf_delta_bwd(r, *b, P, n.value - 1, None) == 4
    assert lib.semicrf_delta_bwd(r, *b, None, n.value, None) == 4
    for keep in (0, 1):
        assert lib.semicrf_delta_workspace_size(r, keep, ctypes.byref(n)) == 0
        assert lib.semicrf_delta_fwd(r, keep, P, P, P, P, P, None, None, P, None, P, n.value - 1, None) == 4
    step = [P, P, P, P, P, None, 4, P, P]
    assert lib.semicrf_delta_step(r, *step, None) == 2  # T is not 1
    s.T = 1
    assert lib.semicrf_delta_step(r, P, P, P, P, P, None, 0, P, P, None) == 2
    for i in (0, 1, 2, 3, 4, 7, 8):
        a = list(step)
        a[i] = None
        assert lib.semicrf_delta_step(r, *a, None) == 1


def turn(**kw):
    d = dict(B=2, T=3, heads=2, heads2=1, D=8, turn=4, dtype=0, layout=0, positions=0, inverse=0, scale=1.0)
    d.update(kw)
    s = encoder._RotaryShape()
    for k, v in d.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 2), (dict(T=0), 2), (dict(heads=0), 2), (dict(heads2=-1), 2), (dict(D=1), 2), (dict(turn=0), 2),
    (dict(turn=3), 2), (dict(turn=10), 2), (dict(D=8194), 3), (dict(dtype=3), 6), (dict(layout=2), 6),
    (dict(positions=3), 6), (dict(B=(1 << 30) + 1), 2), (dict(heads=1 << 26), 2),
])
def test_rotary_shapes_refused(lib, kw, code):
    assert lib.semicrf_rotary(ctypes.byref(turn(**kw)), P, P, P, P, P, P, None) == code


def test_rotary_null(lib):
    for i in (0, 1, 2, 3, 5, 6):
        a = [ctypes.byref(turn()), P, P, P, None, P, P]
        a[i] = None
        assert lib.semicrf_rotary(*a, None) == 1
    assert lib.semicrf_rotary(ctypes.byref(turn(positions=1)), P, P, P, None, P, P, None) == 1


def test_grad_norm_arguments(lib):
    n = ctypes.c_size_t(0)
    sizes = (ctypes.c_int64 * 3)(5000, 0, 3)
    grads = (ctypes.c_void_p * 3)(0x1000, None, 0x100000)
    types = bytes([0, 1, 2])
    size = lambda s, c: lib.semicrf_grad_norm_workspace_size(s, c, ctypes.byref(n))  # noqa: E731
    assert size(sizes, 3) == 0 and n.value == 3 * 8
    assert size(None, 0) == 0 and n.value == 0
    assert size(sizes, -1) == 2 and size(None, 3) == 1
    assert lib.semicrf_grad_norm_workspace_size(sizes, 3, None) == 1
    assert size((ctypes.c_int64 * 1)(-1), 1) == 2 and size((ctypes.c_int64 * 1)(1 << 62), 1) == 2
    call = lambda g, t, c=3, order=2, most=1.0, clip=1, ws=P, have=24: lib.semicrf_grad_norm(  # noqa: E731
        g, sizes, t, c, order, most, clip, P, P, ws, have, None)
    assert call(None, types) == 1 and call(grads, None) == 1
    assert call(grads, bytes([0, 1, 3])) == 6 and call(grads, types, order=3) == 6
    assert call(grads, types, most=-1.0) == 6 and call(grads, types, most=float("nan")) == 6
    assert call(grads, types, ws=None) == 4 and call(grads, types, have=23) == 4
    assert call((ctypes.c_void_p * 3)(0x1000, None, None), types) == 1
    # the last tensor lies in the first
    assert call((ctypes.c_void_p * 3)(0x1000, None, 0x2000), types) == 6


def test_python_refusals():
    x, g = torch.zeros((2, 3, 2, 4)), torch.zeros((2, 3, 2))
    with pytest.raises(ValueError, match="GPU only"):
        encoder.gated_delta(x, x, x, g, g)
    with pytest.raises(ValueError, match="GPU only"):
        encoder.gated_delta_step(x[:, 0], x[:, 0], x[:, 0], g[:, 0], g[:, 0], torch.zeros((2, 2, 4, 4)))
    with pytest.raises(ValueError, match="GPU only"):
        encoder.rotary(x, x, torch.zeros(2, dtype=torch.float64))
    p = torch.zeros(3, requires_grad=True)
    p.grad = torch.zeros(3)
    with pytest.raises(ValueError, match="GPU only"):
        optim.clip_grad_norm_([p], 1.0)
    with pytest.raises(ValueError, match="1, 2 or inf"):
        optim.grad_norm([p], norm_type=3.0)
    for most in (-1.0, float("nan")):
        with pytest.raises(ValueError, match="max_norm"):
            optim.clip_grad_norm_([p], most)
    for bad in (dict(turn=3), dict(turn=0), dict(turn=4, scaling="none"), dict(turn=4, stretch=0.0),
                dict(turn=4, base=-1.0), dict(turn=4, fast=1.0)):
        with pytest.raises(ValueError):
            encoder.rotary_frequencies(**bad)
    assert float(optim.clip_grad_norm_([], 1.0)) == 0.0


def test_frequencies():
    f = encoder.rotary_frequencies(8, base=10000.0)
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert torch.allclose(encoder.rotary_frequencies(8, stretch=4.0, scaling="linear"), f / 4, rtol=1e-14)
    assert torch.allclose(encoder.rotary_frequencies(8, stretch=4.0, scaling="base")[-1], f[-1] / 4, rtol=1e-14)
    bands = encoder.rotary_frequencies(8, stretch=4.0, context=6283, fast=100.0, slow=1.0)
    assert torch.allclose(bands[0], f[0], rtol=1e-14) and torch.allclose(bands[3], f[3] / 4, rtol=1e-3)
