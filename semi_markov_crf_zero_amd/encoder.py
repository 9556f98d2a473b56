"""The encoder's operators over libsemicrf.so (the C ABI in
include/semicrf_encoder.h and semicrf_layer.h): linear attention with a decay
for each head, the gated delta rule (a decay for each position, writes that
take out what was there), their single-token forms, rotary positions, and
group norm with an activation, channels last.

    o = linear_attention(q, k, v, log_decay, lengths=lengths)
    o = linear_attention_step(q, k, v, log_decay, state, slots=slots)
    o = gated_delta(q, k, v, log_decay, beta, lengths=lengths)
    o = gated_delta_step(q, k, v, log_decay, beta, state, slots=slots)
    q, k = rotary(q, k, rotary_frequencies(64, device=q.device))
    y = group_norm(x, groups, weight, bias, lengths=lengths, activation="silu")

The operators over sequences carry gradients (torch.autograd.Function over the
library's backward entry points; a gradient of a gradient, forward-mode tangents and,
but for group norm, tracing are refused); a step moves a pool of states in place and
carries none.  Tensors are CUDA (HIP) tensors, float32, bfloat16 or float16; states,
norms' weights and decays are float32, lengths and slots int32.  Outputs and workspaces are
allocated with torch on the input's device and the work is enqueued on
torch's current stream.  Positions at or past a sequence's length are never
read into any result (they may hold NaN) and their rows of every output and
gradient are 0; a length outside [0, T] gives NaN outputs and zero gradients (rotary has
no lengths: it turns every row as it is).  There is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import binding as bd

EXPORTS = (
    "semicrf_linattn_workspace_size", "semicrf_linattn_fwd", "semicrf_linattn_bwd",
    "semicrf_linattn_step", "semicrf_groupnorm_workspace_size", "semicrf_groupnorm_fwd",
    "semicrf_groupnorm_bwd",
)
# declared in semicrf_layer.h
LAYER_EXPORTS = (
    "semicrf_delta_workspace_size", "semicrf_delta_fwd", "semicrf_delta_bwd",
    "semicrf_delta_step", "semicrf_rotary",
)
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "relu": 3}
ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}
MAX_HEAD = 256  # the widest Dk and Dv of linear attention
MAX_DELTA_HEAD = 128  # of the gated delta rule
MAX_TURNED = 8192  # the widest row rotary positions turn
MAX_SIZE = 2 ** 31 - 1  # of a dimension: the library's int


class _LinattnShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "T", "H", "Hq", "Hk", "Hv", "Dk", "Dv", "dtype")]
                + [("scale", ctypes.c_float)]
                + [(n, ctypes.c_int64 * 3) for n in ("q_stride", "k_stride", "v_stride")])


class _GroupnormShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "T", "C", "G", "dtype", "act")]
                + [("eps", ctypes.c_float)])


class _RotaryShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "T", "heads", "heads2", "D", "turn", "dtype",
                                             "layout", "positions", "inverse")]
                + [("scale", ctypes.c_float)]
                + [(n, ctypes.c_int64 * 3) for n in ("stride", "stride2")])


_lib = None
_dispatch_mode, _PROXY = torch._C._get_dispatch_mode, torch._C._TorchDispatchModeKey.PROXY
_is_tracing = torch._C._is_tracing


def load():
    """The library with the signatures of the encoder's entry points."""
    global _lib
    if _lib is None:
        lib = bd.load()
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        for name in ("linattn", "groupnorm", "delta"):
            f = getattr(lib, "semicrf_%s_workspace_size" % name)
            f.argtypes, f.restype = [P, I, ctypes.POINTER(Z)], I
        lib.semicrf_linattn_fwd.argtypes = [P] * 9 + [P, Z, P]
        lib.semicrf_linattn_bwd.argtypes = [P] * 14 + [P, Z, P]
        lib.semicrf_linattn_step.argtypes = [P] * 6 + [I, P, P, P]
        lib.semicrf_groupnorm_fwd.argtypes = [P] * 7 + [P, Z, P]
        lib.semicrf_groupnorm_bwd.argtypes = [P] * 10 + [P, Z, P]
        lib.semicrf_delta_fwd.argtypes = [P, I] + [P] * 9 + [P, Z, P]
        lib.semicrf_delta_bwd.argtypes = [P] * 16 + [P, Z, P]
        lib.semicrf_delta_step.argtypes = [P] * 7 + [I, P, P, P]
        lib.semicrf_rotary.argtypes = [P] * 8
        for name in EXPORTS + LAYER_EXPORTS:
            getattr(lib, name).restype = I
        _lib = lib
    return _lib


def _ptr(t):
    return None if t is None else t.data_ptr()


def launch(fn, dev, *args):
    """fn(*args, stream) on `dev`'s current stream, with `dev` current.  Refused while a
    graph of torch's operators is recorded from real tensors: the call would not be in it."""
    if _dispatch_mode(_PROXY) is not None:
        raise RuntimeError("the library's operators cannot be traced")
    was = torch._C._cuda_getDevice()
    if was == dev.index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(was))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if rc:
        raise bd.SemiCRFError(rc, fn.__name__)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name, kind, fields, backward):
    """Workspace of a shape (a tuple of the structure's fields)."""
    if max(f for f in fields if isinstance(f, int)) > MAX_SIZE:
        raise ValueError("sizes are at most %d" % MAX_SIZE)
    n = ctypes.c_size_t(0)
    rc = getattr(load(), name)(ctypes.byref(kind(*fields)), backward, ctypes.byref(n))
    if rc:
        raise bd.SemiCRFError(rc, name)
    return n.value


def _workspace(name, kind, fields, backward, dev):
    n = _workspace_bytes(name, kind, fields, backward)
    return (torch.empty(n, dtype=torch.uint8, device=dev) if n else None), n


def _check(name, t, dev, dtype, shape):
    if t.device != dev or t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != shape:
        raise ValueError("%s must be a contiguous %s %s tensor on %s"
                         % (name, dtype, list(shape), dev))


def _check_device(t):
    if t.device.type != "cuda":
        raise ValueError("the encoder's operators run on the GPU only; got a %s tensor"
                         % t.device.type)
    if t.dtype not in DTYPES:
        raise ValueError("unsupported type %s (float32, bfloat16 or float16)" % t.dtype)


def _refuse_tangents(*tensors):
    if any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError("the library's operators have no forward-mode derivatives")


def refuse_modes(*tensors):
    """Refuses what would otherwise go wrong without a word: a traced call (the graph
    would hold its empty outputs and no operator) and forward-mode tangents (the result
    would have none)."""
    if _is_tracing():
        raise RuntimeError("the library's operators cannot be traced")
    if forward_ad._current_level >= 0:
        _refuse_tangents(*tensors)


def _rows(t):
    """t itself if its last dimension is contiguous, else a copy."""
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _heads_check(q, k, v, step, most):
    """Checks q, k, v ([B, T, heads, D], or [B, heads, D] for a step), heads
    up to `most` wide; B, T, H, Hq, Hk, Hv, Dk, Dv, dtype."""
    _check_device(q)
    dev, dtype = q.device, q.dtype
    dims = 3 if step else 4
    for name, t in (("k", k), ("v", v), ("q", q)):
        if t.dim() != dims or t.dtype != dtype or t.device != dev:
            raise ValueError("%s must be a [B, %sheads, D] %s tensor on %s"
                             % (name, "" if step else "T, ", dtype, dev))
    if step:
        (B, Hq, Dk), (Bk, Hk, Dk2), (Bv, Hv, Dv), T = q.shape, k.shape, v.shape, 1
    else:
        (B, T, Hq, Dk), (Bk, Tk, Hk, Dk2), (Bv, Tv, Hv, Dv) = q.shape, k.shape, v.shape
        if Tk != T or Tv != T:
            raise ValueError("q, k and v must have the same T")
    if Bk != B or Bv != B:
        raise ValueError("q, k and v must have the same B")
    if Dk2 != Dk:
        raise ValueError("q and k must have the same width")
    if not (1 <= Dk <= most and 1 <= Dv <= most):
        raise ValueError("heads are 1 to %d wide" % most)
    H = max(Hq, Hk, Hv)
    if B > MAX_SIZE or T > MAX_SIZE or H > MAX_SIZE:
        raise ValueError("sizes are at most %d" % MAX_SIZE)
    if min(Hq, Hk, Hv) < 1 or H % Hq or H % Hk or H % Hv:
        raise ValueError("the larger number of heads must be a multiple of the others: %s"
                         % [Hq, Hk, Hv])
    return B, T, H, Hq, Hk, Hv, Dk, Dv, DTYPES[dtype]


def _linattn_check(q, k, v, log_decay, step):
    dims = _heads_check(q, k, v, step, MAX_HEAD)
    if log_decay.requires_grad and torch.is_grad_enabled():
        raise ValueError("log_decay is a constant of the model: it gets no gradient")
    _check("log_decay", log_decay, q.device, torch.float32, (dims[2],))
    return dims


def _delta_check(q, k, v, log_decay, beta, step):
    """As _linattn_check, with the gates [B, T, H] (or [B, H]); the gates
    contiguous."""
    dims = _heads_check(q, k, v, step, MAX_DELTA_HEAD)
    B, T, H = dims[:3]
    gates = []
    for name, t in (("log_decay", log_decay), ("beta", beta)):
        t = t.contiguous()
        _check(name, t, q.device, torch.float32, (B, H) if step else (B, T, H))
        gates.append(t)
    return dims, *gates


def _pool_check(state, slots, dims, dev):
    """Checks a pool of states and the streams' rows; the number of rows."""
    B, _, H, _, _, _, Dk, Dv, _ = dims
    if state.dim() != 4 or not 1 <= state.shape[0] <= MAX_SIZE:
        raise ValueError("state must be [slots, H, Dk, Dv] with 1 to %d slots" % MAX_SIZE)
    N = state.shape[0]
    _check("state", state, dev, torch.float32, (N, H, Dk, Dv))
    if slots is not None:
        _check("slots", slots, dev, torch.int32, (B,))
    if state.requires_grad and torch.is_grad_enabled():
        raise ValueError("a state that requires a gradient cannot be moved in place")
    return N


def _strides(t):
    s = t.stride()
    return (s[0], s[1] if len(s) == 4 else 0, s[-2])


class _Refused(torch.autograd.Function):
    """The first n tensors as they are, depending on the others in a way that
    is not known: a backward pass through them fails."""

    @staticmethod
    def forward(ctx, message, n, *tensors):
        ctx.message = message
        return tensors[:n]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(ctx.message)


def _once(backward):
    """A backward pass whose results carry no gradients: where they would be
    recorded (create_graph), a backward pass through them fails, whether the
    gradients it came from carry any or not."""
    @functools.wraps(backward)
    def call(ctx, *grads):
        if forward_ad._current_level >= 0:
            _refuse_tangents(*grads)
        if not torch.is_grad_enabled():
            return backward(ctx, *grads)
        with torch.no_grad():
            out = backward(ctx, *grads)
        there = [t for t in out if t is not None]
        on = [t for t in (*ctx.saved_tensors, *grads) if t is not None and t.requires_grad]
        there = iter(_Refused.apply("the gradients of the encoder's operators are "
                                    "once_differentiable: they have no gradients of their own",
                                    len(there), *there, *on))
        return tuple(None if t is None else next(there) for t in out)
    return call


class LinearAttention(torch.autograd.Function):
    """o [B, T, H, Dv] and the state after each sequence [B, H, Dk, Dv]; dims
    is what _linattn_check gives."""

    @staticmethod
    def forward(ctx, q, k, v, state, log_decay, lengths, dims, scale):
        ctx.set_materialize_grads(False)
        ctx.dims, ctx.scale = dims, scale
        saved = q, k, v, state, log_decay, lengths
        B, T, H, _, _, _, Dk, Dv, _ = dims
        q, k, v = _rows(q), _rows(k), _rows(v)
        dev = q.device
        fields = (*dims, scale, _strides(q), _strides(k), _strides(v))
        o = torch.empty((B, T, H, Dv), dtype=q.dtype, device=dev)
        last = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev)
        ws, n = _workspace("semicrf_linattn_workspace_size", _LinattnShape, fields, 0, dev)
        launch(load().semicrf_linattn_fwd, dev, ctypes.byref(_LinattnShape(*fields)), _ptr(q),
               _ptr(k), _ptr(v), _ptr(log_decay), _ptr(lengths), _ptr(state), _ptr(o), _ptr(last),
               _ptr(ws), n)
        ctx.save_for_backward(*saved, ws)
        return o, last

    @staticmethod
    @_once
    def backward(ctx, do, dlast):
        q, k, v, state, log_decay, lengths, states = ctx.saved_tensors
        B, T, H, _, _, _, _, Dv, _ = ctx.dims
        need, dev = ctx.needs_input_grad, q.device
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=dev) if n else None
                      for t, n in ((q, need[0]), (k, need[1]), (v, need[2])))
        dstate = torch.empty_like(state) if state is not None and need[3] else None
        q, k, v = _rows(q), _rows(k), _rows(v)
        fields = (*ctx.dims, ctx.scale, _strides(q), _strides(k), _strides(v))
        if do is None:
            do = torch.zeros((B, T, H, Dv), dtype=q.dtype, device=dev)
        do = do.contiguous()
        dlast = None if dlast is None else dlast.contiguous()
        ws, n = _workspace("semicrf_linattn_workspace_size", _LinattnShape, fields, 1, dev)
        launch(load().semicrf_linattn_bwd, dev, ctypes.byref(_LinattnShape(*fields)), _ptr(q),
               _ptr(k), _ptr(v), _ptr(log_decay), _ptr(lengths), _ptr(state), _ptr(states),
               _ptr(do), _ptr(dlast), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dstate), _ptr(ws), n)
        return dq, dk, dv, dstate, None, None, None, None


def linear_attention(q, k, v, log_decay, lengths=None, state=None, scale=None,
                     return_state: bool = False):
    """Linear attention with a decay for each head, over whole sequences:

        S_t = exp(log_decay_h) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t

    q, k [B, T, heads, Dk] and v [B, T, heads, Dv] of one type, any strides
    with contiguous rows; their numbers of heads divide the largest, H, and
    head h reads head h // (H // heads) of a tensor with fewer (shared
    heads).  log_decay [H] float32, at most 0, a constant of the model (it
    gets no gradient).  lengths [B] int32; state [B, H, Dk, Dv] float32, the
    state before the first position (zeros by default); scale, Dk ** -0.5 by
    default.  Returns o [B, T, H, Dv] or, with return_state, (o, the state
    after each sequence's last position).  Gradients flow to q, k, v and
    state."""
    dims = _linattn_check(q, k, v, log_decay, False)
    refuse_modes(q, k, v, log_decay, state)
    B, T, H, _, _, _, Dk, Dv, _ = dims
    if lengths is not None:
        _check("lengths", lengths, q.device, torch.int32, (B,))
    if state is not None:
        _check("state", state, q.device, torch.float32, (B, H, Dk, Dv))
    if B == 0 or T == 0:
        none = q.sum() + k.sum() + v.sum()  # 0, and part of the graph
        o = none.expand(B, T, H, Dv).clone()
        last = none.float().expand(B, H, Dk, Dv).clone() if state is None else state.clone()
        if lengths is not None:  # NaN where they are none, as with positions
            bad = ((lengths < 0) | (lengths > T))[:, None, None, None]
            last = torch.where(bad, math.nan, last)
    else:
        o, last = LinearAttention.apply(q, k, v, state, log_decay, lengths, dims,
                                        Dk ** -0.5 if scale is None else float(scale))
    return (o, last) if return_state else o


def linear_attention_step(q, k, v, log_decay, state, slots=None, scale=None):
    """One position of B streams: q, k [B, heads, Dk], v [B, heads, Dv].
    state [slots, H, Dk, Dv] float32 is a pool; stream b's is state[slots[b]]
    (slots [B] int32, distinct; stream b's own row b by default) and is moved
    in place.  A stream whose slot is outside the pool is idle: its row of
    the result [B, H, Dv] is 0.  No gradients: a backward pass through the
    result fails, and a state that requires a gradient is moved under
    torch.no_grad() only."""
    dims = _linattn_check(q, k, v, log_decay, True)
    refuse_modes(q, k, v, log_decay, state)
    B, _, H, _, _, _, Dk, Dv, _ = dims
    dev = q.device
    N = _pool_check(state, slots, dims, dev)
    recorded = ()
    if torch.is_grad_enabled():
        if q.requires_grad or k.requires_grad or v.requires_grad:
            recorded = [t for t in (q, k, v) if t.requires_grad]
    o = torch.empty((B, H, Dv), dtype=q.dtype, device=dev)
    if B:
        q, k, v = _rows(q), _rows(k), _rows(v)
        shape = _LinattnShape(*dims, Dk ** -0.5 if scale is None else scale, _strides(q),
                              _strides(k), _strides(v))
        launch(load().semicrf_linattn_step, dev, ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
               _ptr(log_decay), _ptr(slots), N, _ptr(state), _ptr(o))
        increment_version(state)  # a backward pass that saved the old states must fail
    if recorded:
        return _Refused.apply("linear_attention_step has no gradients", 1, o, *recorded)[0]
    return o


def _delta(q, k, v, log_decay, beta, state, lengths, dims, scale, keep):
    """o, the states after, and the workspace, which with keep holds what the
    backward pass reads again."""
    B, T, H, _, _, _, Dk, Dv, _ = dims
    q, k, v, dev = _rows(q), _rows(k), _rows(v), q.device
    fields = (*dims, scale, _strides(q), _strides(k), _strides(v))
    o = torch.empty((B, T, H, Dv), dtype=q.dtype, device=dev)
    last = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev)
    ws, n = _workspace("semicrf_delta_workspace_size", _LinattnShape, fields, keep, dev)
    launch(load().semicrf_delta_fwd, dev, ctypes.byref(_LinattnShape(*fields)), keep, _ptr(q),
           _ptr(k), _ptr(v), _ptr(log_decay), _ptr(beta), _ptr(lengths), _ptr(state), _ptr(o),
           _ptr(last), _ptr(ws), n)
    return o, last, ws


class GatedDelta(torch.autograd.Function):
    """o [B, T, H, Dv] and the state after each sequence [B, H, Dk, Dv]; dims
    is what _delta_check gives."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, beta, state, lengths, dims, scale):
        ctx.set_materialize_grads(False)
        ctx.dims, ctx.scale = dims, scale
        o, last, work = _delta(q, k, v, log_decay, beta, state, lengths, dims, scale, 1)
        ctx.save_for_backward(q, k, v, log_decay, beta, lengths, work)
        return o, last

    @staticmethod
    @_once
    def backward(ctx, do, dlast):
        q, k, v, log_decay, beta, lengths, work = ctx.saved_tensors
        B, T, H, _, _, _, Dk, Dv, _ = ctx.dims
        need, dev = ctx.needs_input_grad, q.device
        dq, dk, dv, dg, db = (torch.empty(t.shape, dtype=t.dtype, device=dev) if n else None
                              for t, n in zip((q, k, v, log_decay, beta), need))
        dstate = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev) if need[5] else None
        q, k, v = _rows(q), _rows(k), _rows(v)
        fields = (*ctx.dims, ctx.scale, _strides(q), _strides(k), _strides(v))
        if do is None:
            do = torch.zeros((B, T, H, Dv), dtype=q.dtype, device=dev)
        do = do.contiguous()
        dlast = None if dlast is None else dlast.contiguous()
        ws, n = _workspace("semicrf_delta_workspace_size", _LinattnShape, fields, 2, dev)
        launch(load().semicrf_delta_bwd, dev, ctypes.byref(_LinattnShape(*fields)), _ptr(q),
               _ptr(k), _ptr(v), _ptr(log_decay), _ptr(beta), _ptr(lengths), _ptr(work), _ptr(do),
               _ptr(dlast), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(db), _ptr(dstate),
               _ptr(ws), n)
        return dq, dk, dv, dg, db, dstate, None, None, None


def gated_delta(q, k, v, log_decay, beta, lengths=None, state=None, scale=None,
                return_state: bool = False):
    """The gated delta rule, over whole sequences:

        S_t = exp(log_decay_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T
        o_t = scale S_t^T q_t

    q, k, v, shared heads, lengths, state and what is returned are those of
    linear_attention, with heads up to 128 wide.  log_decay and beta
    [B, T, H] float32: the decays of each position and head (at most 0 in use;
    -inf forgets) and how much of a write is taken, 0 to 1 (up to 2) for keys of
    length 1.  Gradients flow to q, k, v, log_decay, beta and state."""
    dims, log_decay, beta = _delta_check(q, k, v, log_decay, beta, False)
    refuse_modes(q, k, v, log_decay, beta, state)
    B, T, H, _, _, _, Dk, Dv, _ = dims
    if lengths is not None:
        _check("lengths", lengths, q.device, torch.int32, (B,))
    if state is not None:
        _check("state", state, q.device, torch.float32, (B, H, Dk, Dv))
    if B == 0 or T == 0:
        # 0, and part of the graph
        none = q.sum() + k.sum() + v.sum() + (log_decay.sum() + beta.sum()).to(q.dtype)
        o = none.expand(B, T, H, Dv).clone()
        last = none.float().expand(B, H, Dk, Dv).clone() if state is None else state.clone()
        if lengths is not None:  # NaN where they are none, as with positions
            bad = ((lengths < 0) | (lengths > T))[:, None, None, None]
            last = torch.where(bad, math.nan, last)
    else:
        scale = Dk ** -0.5 if scale is None else float(scale)
        args = q, k, v, log_decay, beta, state, lengths, dims, scale
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in args[:6]):
            o, last = GatedDelta.apply(*args)
        else:
            o, last, _ = _delta(*args, 0)
    return (o, last) if return_state else o


def gated_delta_step(q, k, v, log_decay, beta, state, slots=None, scale=None):
    """One position of B streams by the gated delta rule: q, k [B, heads, Dk],
    v [B, heads, Dv], log_decay, beta [B, H].  The pool of states [slots, H,
    Dk, Dv], slots, idle streams and gradients (none) are those of
    linear_attention_step."""
    dims, log_decay, beta = _delta_check(q, k, v, log_decay, beta, True)
    refuse_modes(q, k, v, log_decay, beta, state)
    B, _, H, _, _, _, Dk, Dv, _ = dims
    dev = q.device
    N = _pool_check(state, slots, dims, dev)
    recorded = ()
    if torch.is_grad_enabled():
        recorded = [t for t in (q, k, v, log_decay, beta) if t.requires_grad]
    o = torch.empty((B, H, Dv), dtype=q.dtype, device=dev)
    if B:
        q, k, v = _rows(q), _rows(k), _rows(v)
        shape = _LinattnShape(*dims, Dk ** -0.5 if scale is None else scale, _strides(q),
                              _strides(k), _strides(v))
        launch(load().semicrf_delta_step, dev, ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
               _ptr(log_decay), _ptr(beta), _ptr(slots), N, _ptr(state), _ptr(o))
        increment_version(state)  # a backward pass that saved the old states must fail
    if recorded:
        return _Refused.apply("gated_delta_step has no gradients", 1, o, *recorded)[0]
    return o


def rotary_frequencies(turn: int, base: float = 10000.0, stretch: float = 1.0,
                       scaling: str = "bands", context: int = 4096, fast: float = 32.0,
                       slow: float = 1.0, device=None):
    """Frequencies [turn / 2] float64 for rotary: base ** (-2 i / turn) radians a
    position, stretched for contexts `stretch` times as long as the trained
    one by

        "linear"  dividing all of them by stretch;
        "base"    raising the base so that the slowest is divided by stretch (a single
                  frequency, 1, stays);
        "bands"   dividing those that turn fewer than `slow` times in `context`
                  positions, leaving those that turn more than `fast` times, and
                  in between a mean of both, linear in the number of turns."""
    if turn < 2 or turn % 2:
        raise ValueError("an even number of elements is turned")
    if scaling not in ("linear", "base", "bands"):
        raise ValueError('scaling must be "linear", "base" or "bands"')
    if not (base > 0 and stretch > 0 and context > 0 and fast > slow):
        raise ValueError("base, stretch and context must be positive, fast above slow")
    i = torch.arange(turn // 2, dtype=torch.float64)
    if scaling == "base" and turn > 2:
        base = base * stretch ** (turn / (turn - 2))
    f = base ** (-2.0 * i / turn)
    if scaling == "linear":
        f = f / stretch
    elif scaling == "bands":
        share = ((context * f / (2 * math.pi)).clamp(slow, fast) - slow) / (fast - slow)
        f = f * share + f / stretch * (1 - share)
    return f.to(device)


class Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, frequencies, positions, layout, scale, inverse):
        ctx.save_for_backward(frequencies, positions)
        ctx.args = layout, scale, inverse
        return _turn(q, k, frequencies, positions, layout, scale, inverse)

    @staticmethod
    @_once
    def backward(ctx, dq, dk=None):
        layout, scale, inverse = ctx.args
        return *_turn(dq, dk, *ctx.saved_tensors, layout, scale, not inverse), *[None] * 5


def _turn(q, k, frequencies, positions, layout, scale, inverse):
    B, T, heads, D = q.shape
    q, dev = _rows(q), q.device
    y = torch.empty(q.shape, dtype=q.dtype, device=dev)
    heads2, y2, strides2 = 0, None, (0, 0, 0)
    if k is not None:
        k = _rows(k)
        heads2, y2, strides2 = k.shape[2], torch.empty(k.shape, dtype=k.dtype, device=dev), _strides(k)
    shape = _RotaryShape(B, T, heads, heads2, D, 2 * frequencies.numel(), DTYPES[q.dtype], layout,
                         0 if positions is None else positions.dim(), inverse, scale, _strides(q),
                         strides2)
    launch(load().semicrf_rotary, dev, ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(frequencies),
           _ptr(positions), _ptr(y), _ptr(y2))
    return y, y2


def rotary(q, k, frequencies, positions=None, layout: str = "half", scale: float = 1.0):
    """Rotary positions: each row of q [B, T, heads, D] and k [B, T, heads, D]
    (or None) at position p is turned in its planes i by the angle
    p frequencies[i] and multiplied by scale there; the planes are elements
    (i, i + n) of a row ("half") or (2 i, 2 i + 1) ("interleaved") for n
    frequencies [n] float64 (rotary_frequencies); elements from 2 n on are
    copied.  positions: row t is at t (None), at positions[b] + t ([B] int32),
    or at positions[b, t] ([B, T] int32).  Rows [B, heads, D] of single
    positions are taken with positions [B].  Rows past a sequence's length
    are turned like the others.  Returns (q', k'), or q' where k is None.
    Gradients flow to q and k."""
    _check_device(q)
    refuse_modes(q, k, frequencies)
    dev, single = q.device, q.dim() == 3
    for name, t in (("q", q), ("k", k)):
        if t is not None and (t.dim() != q.dim() or q.dim() not in (3, 4) or t.dtype != q.dtype
                              or t.device != dev or t.shape[-1] != q.shape[-1]
                              or t.shape[:-2] != q.shape[:-2]):
            raise ValueError("%s must be a [B, T, heads, D] or [B, heads, D] %s tensor on %s, as "
                             "the other" % (name, q.dtype, dev))
    if frequencies.requires_grad and torch.is_grad_enabled():
        raise ValueError("frequencies are constants of the model: they get no gradient")
    D, n = q.shape[-1], frequencies.numel()
    _check("frequencies", frequencies, dev, torch.float64, (n,))
    if not 1 <= 2 * n <= D <= MAX_TURNED:
        raise ValueError("between 1 frequency and one for every two elements of a row, rows of up "
                         "to %d elements" % MAX_TURNED)
    if layout not in ROTARY_LAYOUTS:
        raise ValueError('layout must be "half" or "interleaved"')
    if single:
        if positions is None:
            raise ValueError("single positions need positions [B]")
        q, k = q[:, None], None if k is None else k[:, None]
    B, T = q.shape[:2]
    if max(B, T, q.shape[2], 0 if k is None else k.shape[2]) > MAX_SIZE:
        raise ValueError("sizes are at most %d" % MAX_SIZE)
    if positions is not None:
        _check("positions", positions, dev, torch.int32,
               (B,) if single or positions.dim() == 1 else (B, T))
    if q.numel() == 0:  # no rows, or no heads of q: nothing or only k is turned
        y = q.clone()
        if k is None or k.numel() == 0:
            y2 = None if k is None else k.clone()
        else:
            y2 = Rotary.apply(k, None, frequencies, positions, ROTARY_LAYOUTS[layout],
                              float(scale), False)[0]
    else:
        there = k is not None and k.numel() > 0
        recorded = torch.is_grad_enabled() and (q.requires_grad or there and k.requires_grad)
        y, y2 = (Rotary.apply if recorded else _turn)(
            q, k if there else None, frequencies, positions, ROTARY_LAYOUTS[layout], float(scale),
            False)
        if k is not None and not there:
            y2 = k.clone()
    if single:
        y, y2 = y[:, 0], None if y2 is None else y2[:, 0]
    return y if k is None else (y, y2)


class GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, lengths, groups, eps, act):
        B, T, C = x.shape
        dev = x.device
        ctx.fields = fields = (B, T, C, groups, DTYPES[x.dtype], act, eps)
        y = torch.empty_like(x)
        stats = torch.empty((B, groups, 2), dtype=torch.float32, device=dev)
        ws, n = _workspace("semicrf_groupnorm_workspace_size", _GroupnormShape, fields, 0, dev)
        launch(load().semicrf_groupnorm_fwd, dev, ctypes.byref(_GroupnormShape(*fields)), _ptr(x),
               _ptr(weight), _ptr(bias), _ptr(lengths), _ptr(y), _ptr(stats), _ptr(ws), n)
        ctx.save_for_backward(x, weight, bias, lengths, stats)
        return y

    @staticmethod
    @_once
    def backward(ctx, dy):
        x, weight, bias, lengths, stats = ctx.saved_tensors
        need, dev = ctx.needs_input_grad, x.device
        dy = dy.contiguous()
        dx = torch.empty_like(x)
        dw = torch.empty_like(weight) if need[1] else None
        db = torch.empty_like(bias) if need[2] else None
        ws, n = _workspace("semicrf_groupnorm_workspace_size", _GroupnormShape, ctx.fields, 1, dev)
        launch(load().semicrf_groupnorm_bwd, dev, ctypes.byref(_GroupnormShape(*ctx.fields)),
               _ptr(x), _ptr(weight), _ptr(bias), _ptr(lengths), _ptr(dy), _ptr(stats), _ptr(dx),
               _ptr(dw), _ptr(db), _ptr(ws), n)
        return dx, dw, db, None, None, None, None


def group_norm(x, groups: int, weight=None, bias=None, lengths=None, eps: float = 1e-5,
               activation: str = "none"):
    """Group norm of x [B, ..., C] over the positions of a sequence and the
    C / groups neighbouring channels of a group, then weight and bias ([C]
    float32, each optional) and the activation ("none", "silu", "gelu" with
    the error function, "relu").  lengths [B] int32 for x [B, T, C]:
    statistics over the first lengths[b] positions.  Gradients flow to x,
    weight and bias.  A norm of each position by itself is that of
    x.view(B * T, 1, C)."""
    _check_device(x)
    if x.dim() < 2 or x.shape[-1] < 1:
        raise ValueError("x must be [B, ..., C]")
    C = x.shape[-1]
    if groups < 1 or C % groups:
        raise ValueError("%d channels do not divide into %d groups" % (C, groups))
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be one of %s" % ", ".join(ACTIVATIONS))
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _check(name, t, x.device, torch.float32, (C,))
    if lengths is not None:
        if x.dim() != 3:
            raise ValueError("lengths go with x [B, T, C]")
        _check("lengths", lengths, x.device, torch.int32, (x.shape[0],))
    if x.numel() == 0:
        y = x.clone()
        for t in (weight, bias):  # gradients of 0
            y = y if t is None else y * t.to(x.dtype)
        return y
    flat = x.contiguous()
    if x.dim() != 3:
        flat = flat.view(x.shape[0], -1, C)
    y = GroupNorm.apply(flat, weight, bias, lengths, int(groups), float(eps),
                        ACTIVATIONS[activation])
    return y if x.dim() == 3 else y.view(x.shape)
