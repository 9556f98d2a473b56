"""AdamW over many tensors at once, over libsemicrf.so (semicrf_adamw_step in
include/semicrf_encoder.h, which gives the formula and the 8-bit forms).

    opt = AdamW(model.parameters(), lr=3e-4, bits=8)      # a torch optimizer
    loss.backward(); opt.step()

Clipping by the global norm of the gradients, in place before the step, or with
the coefficient alone, which the step applies as it reads them:

    clip_grad_norm_(model.parameters(), 1.0); opt.step()
    norm, c = grad_norm(model.parameters(), max_norm=1.0); opt.step(grad_scale=c)

AdamWPlan is the step itself for one list of tensors: a table of their
addresses on the device, made once, and `run(grads, step, ...)`.  One launch
covers 416 tensors; the gradients' addresses, new in every step, go with the
launch.  Parameters and gradients are float32, bfloat16 or float16, states
float32 or 8 bits, and a float32 master copy of a 16-bit parameter is
optional.
"""
from __future__ import annotations

import ctypes
import math
import operator
from array import array

import numpy as np
import torch
from torch.autograd.graph import increment_version

from . import binding as bd
from .encoder import DTYPES, launch, refuse_modes

EXPORTS = ("semicrf_adamw_table_size", "semicrf_adamw_table", "semicrf_adamw_step",
           "semicrf_adamw_values")
# declared in semicrf_layer.h
LAYER_EXPORTS = ("semicrf_grad_norm_workspace_size", "semicrf_grad_norm")
NORMS = {float("inf"): 0, 1.0: 1, 2.0: 2}
BLOCK = 256  # elements that share one scale of an 8-bit state
MOMENT_TYPES = {torch.float8_e4m3fn: 0, torch.uint8: 1}  # codes of m; of the root of v


_dtype, _nbytes = operator.attrgetter("dtype"), operator.attrgetter("nbytes")
_numel, _data_ptr = torch.Tensor.numel, torch.Tensor.data_ptr
_TWICE = "a gradient is there twice, whole or in part: it would be scaled twice"
_get_device, _is_contiguous = torch.Tensor.get_device, torch.Tensor.is_contiguous


# an optimizer's state tensors by their bits
_HELD = {32: operator.itemgetter("exp_avg", "exp_avg_sq"),
         8: operator.itemgetter("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")}


class _Tensor(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("p", "master", "m", "v", "m_scale", "v_scale")]
                + [("n", ctypes.c_int64), ("first", ctypes.c_int64), ("dtype", ctypes.c_int32),
                   ("reserved", ctypes.c_int32)])


_lib = None


def load():
    """The library with the signatures of the optimiser's entry points."""
    global _lib
    if _lib is None:
        lib = bd.load()
        P, I, L, D, Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double,
                         ctypes.c_size_t)
        lib.semicrf_adamw_table_size.argtypes = [P, I, I, ctypes.POINTER(Z)]
        lib.semicrf_adamw_table.argtypes = [P, I, I, P, Z]
        lib.semicrf_adamw_step.argtypes = [P, P, P, ctypes.c_char_p, I, I, L, D, D, D, D, D, P, P]
        lib.semicrf_adamw_values.argtypes = [P, P, L, I, P, P]
        lib.semicrf_grad_norm_workspace_size.argtypes = [P, I, ctypes.POINTER(Z)]
        lib.semicrf_grad_norm.argtypes = [P, P, ctypes.c_char_p, I, I, D, I, P, P, P, Z, P]
        for name in EXPORTS + LAYER_EXPORTS:
            getattr(lib, name).restype = I
        _lib = lib
    return _lib


def moment_values(codes, scale):
    """The float32 values an 8-bit state stands for: codes float8_e4m3fn (m)
    or uint8 (v, held by its root) of any shape, scale [ceil(n / 256)]
    float32."""
    if codes.device.type != "cuda" or codes.dtype not in MOMENT_TYPES or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous float8_e4m3fn or uint8 tensor on the GPU")
    if (scale.device != codes.device or scale.dtype != torch.float32 or not scale.is_contiguous()
            or scale.shape != (-(-codes.numel() // BLOCK),)):
        raise ValueError("scale must hold one float32 for each %d codes, on their device" % BLOCK)
    out = torch.empty(codes.shape, dtype=torch.float32, device=codes.device)
    if codes.numel():
        launch(load().semicrf_adamw_values, codes.device, codes.data_ptr(), scale.data_ptr(),
               codes.numel(), MOMENT_TYPES[codes.dtype], out.data_ptr())
    return out


def _zeros8(p, dtype):
    return (torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(dtype),
            torch.zeros(-(-p.numel() // BLOCK), dtype=torch.float32, device=p.device))


def _overlap(tensors):
    """Whether two of these contiguous tensors share memory."""
    at = sorted((start, start + size) for start, size in
                zip(map(_data_ptr, tensors), map(_nbytes, tensors)) if size)
    return any(end > start for (_, end), (start, _) in zip(at, at[1:]))


class AdamWPlan:
    """The step for one list of parameters (one device, contiguous, stepped
    in place).  exp_avg and exp_avg_sq are lists of float32 tensors or, for
    bits=8, of (codes, scale) pairs (float8_e4m3fn and uint8 codes); zeros
    are made where they are not given.  masters: a list of float32 copies of
    16-bit parameters (or None entries).  The plan keeps these tensors and their
    addresses: make a new one when a parameter's storage changes."""

    def __init__(self, params, bits: int = 32, exp_avg=None, exp_avg_sq=None, masters=None):
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        if bits not in (32, 8):
            raise ValueError("states are held in 32 bits or in 8")
        self.bits = bits
        self.dev = dev = self.params[0].device
        n = len(self.params)
        for what, given in (("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq),
                            ("masters", masters)):
            if given is not None and len(given) != n:
                raise ValueError("%s must have one entry for each parameter" % what)
        for p in self.params:
            if (p.device.type != "cuda" or p.device != dev or p.dtype not in DTYPES
                    or not p.is_contiguous()):
                raise ValueError("parameters must be contiguous float32, bfloat16 or float16 "
                                 "tensors on one GPU")
        self.masters = list(masters) if masters is not None else [None] * n
        for p, t in zip(self.params, self.masters):
            if t is not None:
                self._check("a master copy", t, p, torch.float32)
        if bits == 8:
            self.exp_avg = list(exp_avg) if exp_avg is not None else [
                _zeros8(p, torch.float8_e4m3fn) for p in self.params]
            self.exp_avg_sq = list(exp_avg_sq) if exp_avg_sq is not None else [
                _zeros8(p, torch.uint8) for p in self.params]
            for states, dtype in ((self.exp_avg, torch.float8_e4m3fn),
                                  (self.exp_avg_sq, torch.uint8)):
                for p, (c, s) in zip(self.params, states):
                    self._check("codes", c, p, dtype)
                    if (s.device != dev or s.dtype != torch.float32 or not s.is_contiguous()
                            or s.shape != (-(-p.numel() // BLOCK),)):
                        raise ValueError("scales must hold one float32 for each %d elements"
                                         % BLOCK)
        else:
            self.exp_avg, self.exp_avg_sq = (
                list(s) if s is not None else [
                    torch.zeros(p.shape, dtype=torch.float32, device=dev) for p in self.params]
                for s in (exp_avg, exp_avg_sq))
            for states in (self.exp_avg, self.exp_avg_sq):
                for p, t in zip(self.params, states):
                    self._check("a state", t, p, torch.float32)
        held = [t for s in (self.exp_avg, self.exp_avg_sq) for t in s]
        if bits == 8:
            held = [t for pair in held for t in pair]
        # a float32 parameter may be its own master copy
        held += [t for p, t in zip(self.params, self.masters)
                 if t is not None and t.data_ptr() != p.data_ptr()]
        if _overlap(self.params + held):
            raise ValueError("a parameter is there twice, whole or in part: two steps would race "
                             "for it" if _overlap(self.params) else
                             "a state or a master copy is there twice, or is part of another")
        self.numels = [p.numel() for p in self.params]
        self._table()

    @staticmethod
    def _check(what, t, p, dtype):
        if (t.device != p.device or t.dtype != dtype or not t.is_contiguous()
                or t.numel() != p.numel()):
            raise ValueError("%s must be contiguous, %s, on the parameter's device and of its "
                             "size" % (what, dtype))

    def _table(self):
        n = len(self.params)
        rows = (_Tensor * n)()
        for i, p in enumerate(self.params):
            small = self.bits == 8
            m, v = self.exp_avg[i], self.exp_avg_sq[i]
            rows[i] = _Tensor(
                p.data_ptr(), None if self.masters[i] is None else self.masters[i].data_ptr(),
                (m[0] if small else m).data_ptr(), (v[0] if small else v).data_ptr(),
                m[1].data_ptr() if small else None, v[1].data_ptr() if small else None,
                p.numel(), 0, DTYPES[p.dtype], 0)
        lib, size = load(), ctypes.c_size_t(0)
        rc = lib.semicrf_adamw_table_size(rows, n, self.bits, ctypes.byref(size))
        if rc:
            raise bd.SemiCRFError(rc, "semicrf_adamw_table_size")
        self.host = torch.empty(size.value, dtype=torch.uint8)
        rc = lib.semicrf_adamw_table(rows, n, self.bits, self.host.data_ptr(), size.value)
        if rc:
            raise bd.SemiCRFError(rc, "semicrf_adamw_table")
        self.table = self.host.to(self.dev)
        self._streams = {torch.cuda.current_stream(self.dev).cuda_stream}
        self._host, self._device = self.host.data_ptr(), self.table.data_ptr()
        self._dtypes = [], b""

    def _use(self, stream):
        """Another stream reads the table and moves the states: should the plan
        go, their memory waits for it."""
        current = torch.cuda.current_stream(self.dev)
        held = [t for s in (self.exp_avg, self.exp_avg_sq) for t in s]
        if self.bits == 8:
            held = [t for pair in held for t in pair]
        for t in (self.table, *held, *(t for t in self.masters if t is not None)):
            t.record_stream(current)
        self._streams.add(stream)

    def run(self, grads, step: int, lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999,
            eps: float = 1e-8, weight_decay: float = 1e-2, grad_scale=None):
        """One step.  grads: one tensor for each parameter (contiguous, its
        size, float32, bfloat16 or float16), or None to leave that parameter
        and its states as they are.  step counts from 1.  grad_scale: a
        float32 tensor of one element that multiplies every gradient (a clip
        coefficient, an inverse loss scale), read on the device."""
        if len(grads) != len(self.params):
            raise ValueError("need one gradient for each of the %d parameters" % len(self.params))
        there, numels, moved = grads, self.numels, self.params
        try:
            dtypes = list(map(_dtype, grads))
        except AttributeError:  # None among them
            there = [g for g in grads if g is not None]
            numels = [n for n, g in zip(numels, grads) if g is not None]
            moved = [p for p, g in zip(moved, grads) if g is not None]
            dtypes = list(map(_dtype, there))
        if dtypes != self._dtypes[0]:  # the types' codes, worked out once for a list of types
            if not set(dtypes) <= DTYPES.keys():
                raise ValueError("gradients must be float32, bfloat16 or float16")
            self._dtypes = dtypes, bytes(map(DTYPES.get, dtypes))
        if not (list(map(_numel, there)) == numels
                and set(map(_get_device, there)) <= {self.dev.index}
                and all(map(_is_contiguous, there))):
            raise ValueError("gradients must be contiguous tensors of their parameters' sizes on %s"
                             % self.dev)
        at, types = array("Q", map(_data_ptr, there)), self._dtypes[1]
        if there is not grads:
            full, kinds, it = array("Q"), bytearray(), iter(zip(at, types))
            for g in grads:
                a, k = (0, 0) if g is None else next(it)
                full.append(a)
                kinds.append(k)
            at, types = full, bytes(kinds)
        if grad_scale is not None and (grad_scale.device != self.dev or grad_scale.numel() != 1
                                       or grad_scale.dtype != torch.float32):
            raise ValueError("grad_scale must be one float32 on %s" % self.dev)
        stream = torch._C._cuda_getCurrentRawStream(self.dev.index)
        if stream not in self._streams:
            self._use(stream)
        launch(load().semicrf_adamw_step, self.dev, self._host, self._device, at.buffer_info()[0],
               types, len(grads), self.bits, int(step), lr, beta1, beta2, eps, weight_decay,
               None if grad_scale is None else grad_scale.data_ptr())
        increment_version(moved)  # a backward pass that saved the old values must fail


class AdamW(torch.optim.Optimizer):
    """torch optimizer over AdamWPlan, one plan a parameter group.  bits: 32
    or 8, how the states are held; masters: keep float32 copies of 16-bit
    parameters, which follow a parameter that is changed from outside between
    steps (loaded, clamped; not through .data, which leaves no trace).
    Parameters without a gradient are left as they are."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 1e-2, bits: int = 32, masters: bool = False):
        if not (lr >= 0 and eps >= 0 and weight_decay >= 0 and all(0 <= b < 1 for b in betas)):
            raise ValueError("lr, eps and weight_decay must not be negative, betas in [0, 1)")
        if bits not in (32, 8):
            raise ValueError("states are held in 32 bits or in 8")
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps,
                                      weight_decay=weight_decay, bits=bits, masters=masters))
        self._plans, self._versions = {}, {}

    def __setstate__(self, state):  # a copy, or from a file: plans are made anew
        super().__setstate__(state)
        self._plans, self._versions = {}, {}

    def _plan(self, i, group):
        """The group's plan, made anew when a tensor in it has changed its
        storage, size, type or layout."""
        ps, bits = group["params"], group["bits"]
        held = _HELD[bits]
        tensors = []
        for p in ps:
            s = self.state[p]
            if "step" not in s:
                s["step"] = 0
                if bits == 8:
                    s["exp_avg"], s["exp_avg_scale"] = _zeros8(p, torch.float8_e4m3fn)
                    s["exp_avg_sq"], s["exp_avg_sq_scale"] = _zeros8(p, torch.uint8)
                else:
                    s["exp_avg"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                    s["exp_avg_sq"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                if group["masters"] and p.dtype != torch.float32:
                    s["master"] = p.detach().float().contiguous()
            tensors.append(p)
            tensors.extend(held(s))
            if "master" in s:
                tensors.append(s["master"])
        key = (bits, list(map(_data_ptr, tensors)), list(map(_numel, tensors)),
               list(map(_dtype, tensors)))
        old = self._plans.get(i)
        # a plan takes what is contiguous only: making one refuses the rest
        if old is not None and old[0] == key and all(map(_is_contiguous, tensors)):
            return old[1]

        def states(name):
            if bits == 8:
                return [(self.state[p][name], self.state[p][name + "_scale"]) for p in ps]
            return [self.state[p][name] for p in ps]

        plan = AdamWPlan([p.detach() for p in ps], bits, states("exp_avg"),
                         states("exp_avg_sq"), [self.state[p].get("master") for p in ps])
        self._plans[i] = (key, plan)
        self._versions.pop(i, None)
        return plan

    def _follow(self, i, group):
        """Where a parameter is no longer its master's rounding, it was changed
        from outside since the last step: the master takes its value."""
        kept = [p for p in group["params"] if "master" in self.state[p]]
        now = [p._version for p in kept]
        for p, version, last in zip(kept, now, self._versions.get(i) or [None] * len(kept)):
            if version != last:
                m = self.state[p]["master"]
                torch.where(m.to(p.dtype) == p, m, p.float(), out=m)
        return kept

    @torch.no_grad()
    def step(self, closure=None, grad_scale=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for i, group in enumerate(self.param_groups):
            if not group["params"]:
                continue
            plan = self._plan(i, group)
            kept = self._follow(i, group) if group["masters"] else ()
            # parameters may have taken different numbers of steps: one run a count
            by_step = {}
            for j, p in enumerate(group["params"]):
                if p.grad is not None:
                    by_step.setdefault(int(self.state[p]["step"]) + 1, []).append(j)
            for count, who in by_step.items():
                grads = [None] * len(group["params"])
                for j in who:
                    grads[j] = group["params"][j].grad.contiguous()
                b1, b2 = group["betas"]
                plan.run(grads, count, group["lr"], b1, b2, group["eps"], group["weight_decay"],
                         grad_scale)
                for j in who:  # after the run: one that is refused does not count
                    self.state[group["params"][j]]["step"] += 1
            if kept:
                self._versions[i] = [p._version for p in kept]
        return loss

    def load_state_dict(self, state_dict):
        """torch casts floating states to the parameter's type: what is held
        in 8 bits or in float32 is put back as it was saved."""
        super().load_state_dict(state_dict)
        saved = state_dict["state"]
        ids = [i for g in state_dict["param_groups"] for i in g["params"]]
        for i, p in zip(ids, (p for g in self.param_groups for p in g["params"])):
            for name, t in saved.get(i, {}).items():
                if isinstance(t, torch.Tensor):
                    self.state[p][name] = t.detach().clone().to(p.device)
        self._plans = {}


class _Layout:
    """The memory of a tensor as numpy is told of it, which asks about addresses and reads
    nothing."""

    def __init__(self, t):
        size = t.element_size()
        self.__array_interface__ = {
            "version": 3, "data": (t.data_ptr(), True), "typestr": "<u%d" % size,
            "shape": tuple(t.shape), "strides": tuple(size * n for n in t.stride())}


def _folded(t):
    """Whether two elements of a tensor are one in memory."""
    dims = sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1)
    reach = 1
    for s, n in dims:
        if s < reach:  # dimensions that interlock: by counting
            at = torch.zeros(1, dtype=torch.int64)
            for s, n in dims:
                at = (at[:, None] + s * torch.arange(n)).flatten()
            return at.unique().numel() < t.numel()
        reach += s * (n - 1)
    return False


def _shared(grads):
    """Whether some memory is twice in these gradients where one of them is not contiguous (the
    library looks at the others)."""
    spans = []
    for g in grads:
        if not g.numel():  # empty ones are all at address 0
            continue
        start, size = g.data_ptr(), g.nbytes
        inside = torch._debug_has_internal_overlap(g)  # 0: no, and no gaps; 1: yes
        if inside:
            last = sum((n - 1) * s for n, s in zip(g.shape, g.stride()))
            if inside == 1 or last < g.numel() - 1 or _folded(g):
                return True
            size = g.element_size() * (last + 1)
        spans.append((start, start + size, g, g.is_contiguous()))
    spans.sort(key=operator.itemgetter(0))
    before = []  # those that reach past the next one's start
    for start, end, g, whole in spans:
        before = [x for x in before if x[0] > start]
        for _, h, w in before:
            if w and whole:
                continue
            try:
                if np.shares_memory(*(np.asarray(_Layout(t)) for t in (g, h)), max_work=1 << 20):
                    return True
            except np.exceptions.TooHardError:
                return True
        before.append((end, g, whole))
    return False


def _grad_norm(parameters, max_norm, norm_type, clip):
    """(norm, coefficient) of the parameters' gradients, scaled if clip."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [g for p in parameters if (g := p.grad) is not None]
    order = NORMS.get(float(norm_type))
    if order is None:
        raise ValueError("the norm is 1, 2 or inf")
    max_norm = float(max_norm)
    if not max_norm >= 0:
        raise ValueError("max_norm must not be negative")
    if not grads:
        return torch.zeros(()), torch.ones(())  # on the host: no gradient names a device
    refuse_modes(*grads)
    dev = grads[0].device
    if dev.type != "cuda":
        raise ValueError("gradients are normed on the GPU only; got a %s tensor" % dev.type)
    dtypes = list(map(_dtype, grads))
    if not set(dtypes) <= DTYPES.keys() or set(map(_get_device, grads)) != {dev.index}:
        raise ValueError("gradients must be dense float32, bfloat16 or float16 tensors on one GPU")
    # a copy of what is not contiguous is scaled in its place and copied back (torch
    # refuses the question for sparse gradients)
    flat = grads if all(map(_is_contiguous, grads)) else [g.contiguous() for g in grads]
    n = len(flat)
    at, sizes = array("Q", map(_data_ptr, flat)), array("q", map(_numel, flat))
    lib, size = load(), ctypes.c_size_t(0)
    rc = lib.semicrf_grad_norm_workspace_size(sizes.buffer_info()[0], n, ctypes.byref(size))
    if rc:
        raise bd.SemiCRFError(rc, "semicrf_grad_norm_workspace_size")
    work = torch.empty(size.value, dtype=torch.uint8, device=dev)
    norm = torch.empty((), dtype=torch.float32, device=dev)
    coefficient = None if clip else torch.empty_like(norm)
    if clip and flat is not grads and _shared(grads):
        raise ValueError(_TWICE)
    try:
        launch(lib.semicrf_grad_norm, dev, at.buffer_info()[0], sizes.buffer_info()[0],
               bytes(map(DTYPES.get, dtypes)), n, order, max_norm, clip, norm.data_ptr(),
               None if clip else coefficient.data_ptr(), work.data_ptr(), size.value)
    except bd.SemiCRFError as e:
        if clip and e.code == 6:  # the one argument that was not looked at above
            raise ValueError(_TWICE) from None
        raise
    if clip:
        if flat is not grads:
            for g, f in zip(grads, flat):
                if g is not f:
                    g.copy_(f)
        increment_version(grads)  # a backward pass that saved the old values must fail
    return norm, coefficient


@torch.no_grad()
def grad_norm(parameters, max_norm=None, norm_type: float = 2.0):
    """The norm (1, 2 or inf) of all gradients of `parameters` together, a
    float32 tensor of no dimensions on their device; summed in float64.  With
    max_norm, (norm, coefficient), the coefficient min(1, max_norm / (norm +
    1e-6)) that clipping multiplies by: AdamW.step(grad_scale=coefficient)
    applies it without another pass over the gradients."""
    norm, coefficient = _grad_norm(parameters, math.inf if max_norm is None else max_norm,
                                   norm_type, False)
    return norm if max_norm is None else (norm, coefficient)


@torch.no_grad()
def clip_grad_norm_(parameters, max_norm: float, norm_type: float = 2.0):
    """Multiplies all gradients of `parameters` by min(1, max_norm / (norm +
    1e-6)), in place; the norm before, as grad_norm gives it.  Gradients that
    share memory are refused."""
    return _grad_norm(parameters, max_norm, norm_type, True)[0]
