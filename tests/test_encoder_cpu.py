"""Host-side checks of the encoder's and the optimiser's C ABI (no GPU):
exports, argument errors returned before any launch, and the refusals of the
Python entry points."""
import ctypes
import os
import re

import pytest
import torch

from semi_markov_crf_zero_amd import binding as bd
from semi_markov_crf_zero_amd import encoder, optim

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "semicrf_encoder.h")
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call fails validation


@pytest.fixture(scope="module")
def lib():
    encoder.load()
    return optim.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(semicrf_[a-z_0-9]+)\s*\(", text))
    assert names == set(encoder.EXPORTS) | set(optim.EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def lin(**kw):
    d = dict(B=2, T=5, H=4, Hq=4, Hk=2, Hv=1, Dk=8, Dv=6, dtype=1, scale=1.0)
    d.update(kw)
    s = encoder._LinattnShape()
    for k, v in d.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 2), (dict(T=0), 2), (dict(H=0), 2), (dict(Hq=3), 2), (dict(Hk=8), 2),
    (dict(Hv=0), 2), (dict(Dk=0), 2), (dict(Dv=0), 2), (dict(Dk=257), 3), (dict(Dv=300), 3),
    (dict(dtype=3), 6), (dict(dtype=-1), 6), (dict(B=1 << 28, H=4), 2),
])
def test_linattn_shapes_refused(lib, kw, code):
    s, n = lin(**kw), ctypes.c_size_t(0)
    assert lib.semicrf_linattn_workspace_size(ctypes.byref(s), 0, ctypes.byref(n)) == code
    P = FAKE
    assert lib.semicrf_linattn_fwd(ctypes.byref(s), P, P, P, P, None, None, P, None, P, 1 << 40,
                                   None) == code
    assert lib.semicrf_linattn_bwd(ctypes.byref(s), P, P, P, P, None, None, None, P, None, P, P, P,
                                   None, P, 1 << 40, None) == code


def test_linattn_null_and_workspace(lib):
    s, n, P = lin(), ctypes.c_size_t(0), FAKE
    r = ctypes.byref(s)
    assert lib.semicrf_linattn_workspace_size(r, 1, None) == 1
    assert lib.semicrf_linattn_workspace_size(None, 1, ctypes.byref(n)) == 1
    assert lib.semicrf_linattn_workspace_size(r, 1, ctypes.byref(n)) == 0
    assert n.value > 0  # parts of the shared heads' gradients
    for i in (0, 1, 2, 3, 6):
        a = [P, P, P, P, None, None, P, None]
        a[i] = None
        assert lib.semicrf_linattn_fwd(r, *a, P, 1 << 40, None) == 1
        b = [P, P, P, P, None, None, None, P, None, P, P, P, None]
        b[i if i < 4 else 7] = None
        assert lib.semicrf_linattn_bwd(r, *b, P, 1 << 40, None) == 1
    b = [P, P, P, P, None, None, None, P, None, P, P, P, None]
    assert lib.semicrf_linattn_bwd(r, *b, P, n.value - 1, None) == 4
    assert lib.semicrf_linattn_bwd(r, *b, None, n.value, None) == 4
    assert lib.semicrf_linattn_step(r, P, P, P, P, None, 4, P, P, None) == 2  # T is not 1
    s.T = 1
    assert lib.semicrf_linattn_step(r, P, P, P, P, None, 0, P, P, None) == 2
    assert lib.semicrf_linattn_step(r, P, P, P, P, None, 4, None, P, None) == 1


def gn(**kw):
    d = dict(B=2, T=5, C=12, G=3, dtype=0, act=1, eps=1e-5)
    d.update(kw)
    s = encoder._GroupnormShape()
    for k, v in d.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 2), (dict(T=0), 2), (dict(C=0), 2), (dict(G=0), 2), (dict(G=5), 2),
    (dict(dtype=5), 6), (dict(act=4), 6), (dict(act=-1), 6), (dict(eps=-1.0), 6),
    (dict(eps=float("nan")), 6), (dict(T=(1 << 30) + 1), 2),
])
def test_groupnorm_shapes_refused(lib, kw, code):
    s, n, P = gn(**kw), ctypes.c_size_t(0), FAKE
    r = ctypes.byref(s)
    assert lib.semicrf_groupnorm_workspace_size(r, 0, ctypes.byref(n)) == code
    assert lib.semicrf_groupnorm_fwd(r, P, P, P, None, P, P, P, 1 << 40, None) == code
    assert lib.semicrf_groupnorm_bwd(r, P, P, P, None, P, P, P, P, P, P, 1 << 40, None) == code


def test_groupnorm_null_and_workspace(lib):
    s, n, P = gn(T=4096, B=4), ctypes.c_size_t(0), FAKE
    r = ctypes.byref(s)
    for i in (0, 4, 5):
        a = [P, P, P, None, P, P]
        a[i if i == 0 else i] = None
        assert lib.semicrf_groupnorm_fwd(r, *a, P, 1 << 40, None) == 1
    for i in (0, 4, 5, 6):
        b = [P, P, P, None, P, P, P, P, P]
        b[i] = None
        assert lib.semicrf_groupnorm_bwd(r, *b, P, 1 << 40, None) == 1
    for back, args in ((0, [P, P, P, None, P, P]), (1, [P, P, P, None, P, P, P, P, P])):
        f = lib.semicrf_groupnorm_bwd if back else lib.semicrf_groupnorm_fwd
        assert lib.semicrf_groupnorm_workspace_size(r, back, ctypes.byref(n)) == 0
        assert n.value > 0
        assert f(r, *args, P, n.value - 1, None) == 4
        assert f(r, *args, None, n.value, None) == 4


def test_adamw_table(lib):
    n = ctypes.c_size_t(0)
    rows = (optim._Tensor * 3)()
    for i, e in enumerate((4096, 0, 4097)):
        rows[i] = optim._Tensor(0x1000, None, 0x1000, 0x1000, 0x1000, 0x1000, e, 0, 0, 0)
    assert lib.semicrf_adamw_table_size(rows, 3, 8, ctypes.byref(n)) == 0
    assert n.value == 3 * ctypes.sizeof(optim._Tensor) + 3 * 4
    buf = (ctypes.c_uint8 * n.value)()
    assert lib.semicrf_adamw_table(rows, 3, 8, buf, n.value - 1) == 4
    assert lib.semicrf_adamw_table(rows, 3, 8, buf, n.value) == 0
    out = (optim._Tensor * 3).from_buffer(buf)
    assert [t.first for t in out] == [0, 1, 1]
    at = ctypes.sizeof(optim._Tensor) * 3
    assert list((ctypes.c_int32 * 3).from_buffer(buf, at)) == [0, 2, 2]
    assert lib.semicrf_adamw_table_size(rows, 0, 8, ctypes.byref(n)) == 2
    assert lib.semicrf_adamw_table_size(rows, 3, 16, ctypes.byref(n)) == 6
    assert lib.semicrf_adamw_table_size(None, 3, 8, ctypes.byref(n)) == 1
    rows[2].v_scale = None
    assert lib.semicrf_adamw_table_size(rows, 3, 8, ctypes.byref(n)) == 1
    assert lib.semicrf_adamw_table_size(rows, 3, 32, ctypes.byref(n)) == 0
    rows[1].n = -1
    assert lib.semicrf_adamw_table_size(rows, 3, 32, ctypes.byref(n)) == 2
    rows[1].n = 1 << 44
    assert lib.semicrf_adamw_table_size(rows, 3, 32, ctypes.byref(n)) == 2


def test_adamw_step_arguments(lib):
    P, g, t = FAKE, (ctypes.c_void_p * 1)(0x1000), bytes(1)
    ok = dict(host=P, dev=P, g=g, t=t, count=1, bits=32, step=1, lr=1e-3, b1=0.9, b2=0.999,
              eps=1e-8, wd=0.0)
    for kw, code in ((dict(host=None), 1), (dict(dev=None), 1), (dict(g=None), 1),
                     (dict(t=None), 1), (dict(count=0), 2), (dict(bits=4), 6), (dict(step=0), 6),
                     (dict(b1=1.0), 6), (dict(b2=-0.1), 6), (dict(eps=-1.0), 6),
                     (dict(t=bytes([7])), 6)):
        a = dict(ok, **kw)
        assert lib.semicrf_adamw_step(*a.values(), None, None) == code, kw
    assert lib.semicrf_adamw_values(P, P, 0, 0, P, None) == 2
    assert lib.semicrf_adamw_values(None, P, 4, 0, P, None) == 1


def test_python_refuses_cpu_tensors():
    q = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError):
        encoder.linear_attention(q, q, q, torch.zeros(2))
    with pytest.raises(ValueError):
        encoder.linear_attention_step(q[:, 0], q[:, 0], q[:, 0], torch.zeros(2),
                                      torch.zeros(1, 2, 8, 8))
    with pytest.raises(ValueError):
        encoder.group_norm(q, 2)
    with pytest.raises(ValueError):
        optim.AdamWPlan([q])
    with pytest.raises(ValueError):
        optim.AdamWPlan([])
    with pytest.raises(ValueError):
        optim.AdamW([torch.nn.Parameter(q)], bits=4)
    with pytest.raises(ValueError):
        optim.AdamW([torch.nn.Parameter(q)], betas=(0.9, 1.0))
    with pytest.raises(ValueError):
        optim.moment_values(torch.zeros(4, dtype=torch.uint8), torch.zeros(1))
    assert bd.STATUS[4] == "SEMICRF_ERR_WORKSPACE"


def test_python_refuses_sizes_past_the_library_s():
    """ctypes would cut a size past 31 bits without a word."""
    with pytest.raises(ValueError, match="sizes"):
        encoder._workspace_bytes("semicrf_groupnorm_workspace_size", encoder._GroupnormShape,
                                 (2 ** 32 + 1, 1, 8, 2, 0, 0, 1e-5), 0)


@pytest.mark.parametrize("kw,code", [
    # a norm of each position by itself, for the longest sequences and for many
    (dict(B=1 << 20, T=1, C=64, G=4), 0), (dict(B=1 << 20, T=1, C=256, G=32), 0),
    (dict(B=908793, T=1, C=32, G=4, dtype=1), 0), (dict(B=1 << 28, T=1, C=16, G=2), 0),
    (dict(B=1 << 20, T=1, C=8192, G=16, dtype=1), 0), (dict(B=1 << 20, T=64, C=128, G=8), 0),
    # 2^32 threads and more
    (dict(B=1 << 26, T=1, C=8192, G=1), 2), (dict(B=1 << 24, T=1, C=8192, G=4096), 2),
    (dict(B=(1 << 30) + 1, T=1, C=1, G=1), 2), (dict(B=1, C=1 << 30, G=1, T=1), 2),
])
@pytest.mark.parametrize("backward", [0, 1])
def test_groupnorm_sizes(lib, kw, code, backward):
    n = ctypes.c_size_t(0)
    assert lib.semicrf_groupnorm_workspace_size(ctypes.byref(gn(**kw)), backward,
                                                ctypes.byref(n)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=(1 << 24) - 1, H=1, Dk=64, Dv=64), 0), (dict(B=1 << 24, H=1, Dk=64, Dv=64), 2),
    (dict(B=(1 << 20) - 1, H=8, Dk=128, Dv=33), 0), (dict(B=1 << 20, H=8, Dk=33, Dv=128), 2),
    (dict(B=(1 << 21) - 1, H=2, Dk=256, Dv=256), 0), (dict(B=1 << 21, H=2, Dk=256, Dv=8), 2),
    (dict(B=1, T=1 << 30, H=4, Dk=256, Dv=256), 0), (dict(B=1, T=(1 << 30) + 1, H=4), 2),
])
@pytest.mark.parametrize("backward", [0, 1])
def test_linattn_sizes(lib, kw, code, backward):
    s = lin(**dict(kw, Hq=1, Hk=1, Hv=1))
    n = ctypes.c_size_t(0)
    assert lib.semicrf_linattn_workspace_size(ctypes.byref(s), backward, ctypes.byref(n)) == code


def test_linattn_workspace_of_shared_heads(lib):
    """Parts of one gradient at a time: one float32 row a head, of the widest."""
    def size(backward, **kw):
        s, n = lin(B=1, T=1 << 20, H=16, Dk=64, Dv=64, **kw), ctypes.c_size_t(0)
        assert lib.semicrf_linattn_workspace_size(ctypes.byref(s), backward, ctypes.byref(n)) == 0
        return n.value
    part = (1 << 20) * 16 * 64 * 4
    for kw in (dict(Hq=1, Hk=1, Hv=1), dict(Hq=16, Hk=2, Hv=2), dict(Hq=16, Hk=16, Hv=4)):
        assert size(1, **kw) - size(0, **kw) == part
    assert size(1, Hq=16, Hk=16, Hv=16) == size(0, Hq=16, Hk=16, Hv=16)
