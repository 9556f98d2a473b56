"""The operators of a tagger's layer with data-dependent memory, and of its training step, as they are
measured: the gated delta rule (whole sequences, training, single positions), rotary positions
(inference, training, streams), and the global norm of many gradients with clipping.

`own` False: elementary torch operations in float32 (angles, cumulated decays and the norm's sum in
float64), rounded once to the output's type.
`own` True: the calls a user makes of semi_markov_crf_zero_amd.encoder and .optim.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # The encoder of the sentence tagger (32 sentences of up to 512 tokens, the NLP workload).
        dict(name="delta-nlp-fwd", op="delta", train=False, B=32, T=512, H=4, Hq=4, Hk=4, Hv=4, Dk=64, Dv=64,
             dtype="bf16", ragged=True, state=False),
        # One chromosome-length sequence read in inference, continued from a prefix's state (2^20
        # positions, the extreme workload).
        dict(name="delta-extreme-fwd", op="delta", train=False, B=1, T=1048576, H=4, Hq=4, Hk=4, Hv=4, Dk=64, Dv=64,
             dtype="bf16", ragged=False, state=True),
        # A training step of a speech encoder with 256 channels (16 utterances, the speech workload).
        dict(name="delta-speech-train", op="delta", train=True, B=16, T=4096, H=4, Hq=4, Hk=4, Hv=4, Dk=64, Dv=64,
             dtype="bf16", ragged=True, state=False),
        # Windows of a genome trained in float32 with keys shared by two heads and odd sizes.
        dict(name="delta-genome-train", op="delta", train=True, B=4, T=20001, H=4, Hq=4, Hk=2, Hv=4, Dk=40, Dv=72,
             dtype="f32", ragged=False, state=True),
        # Genome windows of odd lengths read in inference by wide heads.
        dict(name="delta-wide-fwd", op="delta", train=False, B=4, T=20001, H=4, Hq=4, Hk=4, Hv=4, Dk=128, Dv=128,
             dtype="f16", ragged=True, state=True),
        # Streams tagged as they arrive: the next position of a few streams (latency) ...
        dict(name="delta-step-small", op="step", B=4, N=16, H=4, Dk=64, Dv=64, dtype="bf16"),
        # ... and of many streams of a wide encoder.
        dict(name="delta-step-large", op="step", B=256, N=320, H=16, Dk=128, Dv=128, dtype="bf16"),
        # The positions of the 2^20-position sequence: half of each head turned, in frequencies
        # stretched for a context longer than the trained one.
        dict(name="rotary-extreme-fwd", op="rotary", train=False, B=1, T=1048576, Hq=4, Hk=4, D=64, turn=32,
             layout="half", stretch=64.0, starts="none", dtype="bf16"),
        # Windows of a genome in float32, each from its own place on, shared keys, odd sizes, training.
        dict(name="rotary-genome-train", op="rotary", train=True, B=4, T=20001, Hq=4, Hk=2, D=40, turn=36,
             layout="interleaved", stretch=1.0, starts="sequence", dtype="f32"),
        # The next positions of many streams of a wide encoder, each somewhere else in its sequence.
        dict(name="rotary-streams", op="rotary", train=False, B=256, T=1, Hq=16, Hk=16, D=128, turn=128,
             layout="half", stretch=1.0, starts="position", dtype="bf16"),
        # The gradients of a small tagger: many small tensors, clipped (latency).
        dict(name="clip-tagger", op="clip", tensors=120, total=1500000, dtype="f32", order=2.0),
        # The gradients of a wide encoder in bfloat16, clipped in place.
        dict(name="clip-wide", op="clip", tensors=64, total=80000000, dtype="bf16", order=2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["delta", "delta", "delta", "step", "rotary", "rotary", "clip"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if kind == "delta":
        H = rng.choice([1, 2, 3, 4, 6, 8])
        share = rng.choice(["none", "none", "kv", "qk"])
        few = max(h for h in (1, 2, 3) if H % h == 0)
        Dk, Dv = rng.choice([16, 32, 40, 64, 64, 96, 128]), rng.choice([16, 32, 64, 64, 72, 128])
        heads = _log(rng, 600, 100000 if max(Dk, Dv) > 64 else 400000)
        T = min(max(1, heads // H), _log(rng, 1, 200000))
        # the decay of a sequence's only position reaches nothing but the state before it
        return dict(op="delta", train=rng.random() < 0.5, B=max(1, min(64, heads // (H * T))), T=T, H=H,
                    Hq=few if share == "qk" else H, Hk=few if share != "none" else H, Hv=few if share == "kv" else H,
                    Dk=Dk, Dv=Dv, dtype=dtype, ragged=rng.random() < 0.5, state=T == 1 or rng.random() < 0.5)
    if kind == "step":
        B = _log(rng, 1, 256)
        return dict(op="step", B=B, N=B + rng.randrange(0, 65), H=rng.choice([1, 2, 4, 5, 8, 16]),
                    Dk=rng.choice([32, 40, 64, 64, 128]), Dv=rng.choice([32, 64, 64, 72, 128]), dtype=dtype)
    if kind == "rotary":
        Hk = rng.choice([1, 2, 3, 4, 8])
        D = rng.choice([16, 32, 40, 64, 64, 72, 128])
        rows = _log(rng, 1, min(500000, 60000000 // (3 * Hk * D)))
        T = min(rows, _log(rng, 1, 500000))
        return dict(op="rotary", train=rng.random() < 0.5, B=max(1, rows // T), T=T, Hq=Hk * rng.choice([1, 1, 2]),
                    Hk=Hk, D=D, turn=rng.choice([D, D, D // 2, D // 4 * 2]), layout=rng.choice(["half", "interleaved"]),
                    stretch=rng.choice([1.0, 8.0, 64.0]), starts=rng.choice(["none", "sequence", "position"]),
                    dtype=dtype)
    return dict(op="clip", tensors=_log(rng, 1, 400), total=_log(rng, 3000, 60000000), dtype=dtype,
                order=rng.choice([2.0, 2.0, math.inf]))


# ---------------------------------------------------------------------------------------------
# inputs

def _sizes(case):
    """Matrices and vectors of an encoder, the vectors a quarter of the tensors; odd sizes among them."""
    n, total = case["tensors"], case["total"]
    vec = [64 + 37 * i % 448 for i in range(n // 4)]
    rest = max(1, n - len(vec))
    share = [1.0 + (i * 7 % 11) for i in range(rest)]
    left = max(rest, total - sum(vec))
    return vec + [max(1, int(left * s / sum(share))) for s in share]


def _gates(shape, kind):
    """Log decays of a memory of 8 to 2048 positions, and how much of a write is taken."""
    g = -torch.exp2(-3.0 - 8.0 * torch.rand(shape, **kind))
    return g, torch.sigmoid(torch.randn(shape, **kind))


def _unit(shape, dtype, kind):
    x = torch.randn(shape, **kind)
    return (x / torch.sqrt((x * x).sum(-1, keepdim=True))).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind, op, dt = dict(device="cuda", generator=gen), case["op"], DTYPES[case["dtype"]]
    if op == "delta":
        B, T, H, Dk, Dv = (case[k] for k in ("B", "T", "H", "Dk", "Dv"))
        s = {"case": case, "lengths": None, "q": _unit((B, T, case["Hq"], Dk), dt, kind),
             "k": _unit((B, T, case["Hk"], Dk), dt, kind), "v": torch.randn((B, T, case["Hv"], Dv), **kind).to(dt)}
        if case["ragged"]:
            s["lengths"] = torch.randint((T + 1) // 2, T + 1, (B,), dtype=torch.int32, **kind)
        s["log_decay"], s["beta"] = _gates((B, T, H), kind)
        s["state"] = torch.randn((B, H, Dk, Dv), **kind) if case["state"] else None
        if case["train"]:
            s["do"] = torch.randn((B, T, H, Dv), **kind).to(dt)
            s["ds"] = torch.randn((B, H, Dk, Dv), **kind) if case["state"] else None
            for name in ("q", "k", "v", "log_decay", "beta", "state"):
                if s[name] is not None:
                    s[name].requires_grad_(True)
        return s
    if op == "step":
        B, N, H, Dk, Dv = (case[k] for k in ("B", "N", "H", "Dk", "Dv"))
        slots = torch.randperm(N, **kind)[:B].to(torch.int32)
        if B > 8:
            slots[B // 3] = -1  # a stream that has ended
        g, beta = _gates((B, H), kind)
        # row N takes what the plain form writes for such streams
        return {"case": case, "slots": slots, "log_decay": g, "beta": beta, "pool": torch.randn((N + 1, H, Dk, Dv), **kind),
                "q": _unit((B, H, Dk), dt, kind), "k": _unit((B, H, Dk), dt, kind),
                "v": torch.randn((B, H, Dv), **kind).to(dt)}
    if op == "rotary":
        B, T, D, turn = (case[k] for k in ("B", "T", "D", "turn"))
        f = 10000.0 ** (-torch.arange(0, turn, 2, dtype=torch.float64, device="cuda") / turn)
        if case["stretch"] > 1.0:  # wavelengths over a 32nd of 4096 positions are stretched, by all of it over 4096
            share = ((4096 * f / (2 * math.pi)).clamp(1, 32) - 1) / 31
            f = f * share + f / case["stretch"] * (1 - share)
        s = {"case": case, "frequencies": f, "positions": None,
             "q": torch.randn((B, T, case["Hq"], D), **kind).to(dt), "k": torch.randn((B, T, case["Hk"], D), **kind).to(dt)}
        if case["starts"] != "none":
            s["positions"] = torch.randint(0, 1 << 20, (B,) if case["starts"] == "sequence" else (B, T),
                                           dtype=torch.int32, **kind)
        if case["train"]:
            for name, to in (("q", "dq"), ("k", "dk")):
                s[to] = torch.randn(s[name].shape, **kind).to(dt)
                s[name].requires_grad_(True)
        return s
    sizes = _sizes(case)
    at = [0]
    for n in sizes:  # each on 512 bytes
        at.append(at[-1] + -(-n // 256) * 256)
    flat = torch.zeros(at[-1], dtype=dt, device="cuda")
    params = []
    for i, n in enumerate(sizes):
        flat[at[i]:at[i] + n] = torch.randn(n, **kind) * 1e-2
        p = torch.empty(n, dtype=dt, device="cuda", requires_grad=True)
        p.grad = flat[at[i]:at[i] + n]
        params.append(p)
    most = 1e-2 if case["order"] == math.inf else 5e-3 * math.sqrt(sum(sizes))
    return {"case": case, "params": params, "flat": flat, "max_norm": most}


# ---------------------------------------------------------------------------------------------
# one pass

def run(state):
    return _RUN[state["case"]["op"]](state)


def _run_delta(s):
    case = s["case"]
    if not own:
        return _plain_delta(s)
    from semi_markov_crf_zero_amd import encoder
    o, last = encoder.gated_delta(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], lengths=s["lengths"],
                                  state=s["state"], return_state=True)
    if not case["train"]:
        return o, last
    wrt = [s[n] for n in ("q", "k", "v", "log_decay", "beta", "state") if s[n] is not None]
    if s["ds"] is None:
        return (o.detach(), last.detach(), *torch.autograd.grad(o, wrt, s["do"]))
    return (o.detach(), last.detach(), *torch.autograd.grad((o, last), wrt, (s["do"], s["ds"])))


def _scan(A, b):
    """X_n = A_n X_{n-1} + b_n for all n (dimension 2) as (products of A, sums): X_n = A'_n X_{-1} + b'_n."""
    d = 1
    while d < A.shape[2]:
        b = torch.cat((b[:, :, :d], b[:, :, d:] + A[:, :, d:] @ b[:, :, :-d]), 2)
        A = torch.cat((A[:, :, :d], A[:, :, d:] @ A[:, :, :-d]), 2)
        d *= 2
    return A, b


def _inverse(M):
    """(I + M)^-1 of strictly lower triangular M [..., L, L], L a power of two: blocks of 1, 2, 4, ..."""
    L = M.shape[-1]
    i = torch.arange(L, device=M.device)
    X = torch.eye(L, device=M.device).expand(M.shape)
    n = 1
    while n < L:
        beside = (i[:, None] // (2 * n) == i // (2 * n)) & (i[:, None] // n != i // n)
        X = X - X @ torch.where(beside, M, 0.0) @ X
        n *= 2
    return X


def _plain_delta(s, L=64):
    case = s["case"]
    B, T, H, dt = case["B"], case["T"], case["H"], DTYPES[case["dtype"]]
    scale, N = case["Dk"] ** -0.5, -(-T // L)
    t = torch.arange(N * L, device="cuda")
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"]
    live = (t < n[:, None])[:, None].view(B, 1, N, L)

    def cut(x):
        """[B, T, heads, ...] to float32 [B, H, N, L, ...], shared heads repeated, nothing past the lengths."""
        x = x.detach().float()
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, N * L - T)).transpose(1, 2)
        x = x.repeat_interleave(H // x.shape[1], dim=1).reshape(B, H, N, L, *x.shape[3:])
        return torch.where(live if x.dim() == 4 else live[..., None], x, 0.0)

    def back(x, heads):
        """[B, H, N, L, ...] to [B, T, heads, ...]: sums over the heads that share one."""
        x = x.reshape(B, heads, H // heads, N * L, *x.shape[4:]).sum(2)[:, :, :T]
        return x.transpose(1, 2).contiguous()

    q, k, v, g, beta = (cut(s[x]) for x in ("q", "k", "v", "log_decay", "beta"))
    G = torch.cumsum(g.double(), -1)
    i = torch.arange(L, device="cuda")
    decay = torch.where(i[:, None] >= i, torch.exp((G[..., None] - G[..., None, :]).clamp(max=0.0).float()), 0.0)
    from_start, to_end = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    before = torch.where(i[:, None] > i, decay * (k @ k.transpose(-1, -2)), 0.0)
    inverse = _inverse(beta[..., None] * before)
    X = inverse * beta[..., None, :]
    W, kh = X @ (from_start * k), to_end * k
    A = from_start[..., -1:, :] * torch.eye(case["Dk"], device="cuda") - kh.transpose(-1, -2) @ W
    U = X @ v
    through, added = _scan(A, kh.transpose(-1, -2) @ U)
    first = torch.zeros((B, H, case["Dk"], case["Dv"]), device="cuda") if s["state"] is None else s["state"].detach()
    after = added + through @ first[:, :, None]
    del through, added
    S = torch.cat((first[:, :, None], after[:, :, :-1]), 2)
    U = U - W @ S
    P = decay * (q @ k.transpose(-1, -2))
    o = back(((from_start * q) @ S + P @ U) * scale, H).to(dt)
    last = after[:, :, -1]
    if not case["train"]:
        return o, last
    do = cut(s["do"]) * scale
    dU = P.transpose(-1, -2) @ do
    ds = torch.zeros_like(first) if s["ds"] is None else s["ds"]
    through, added = _scan(A.transpose(-1, -2).flip(2), ((from_start * q).transpose(-1, -2) @ do
                                                         - W.transpose(-1, -2) @ dU).flip(2))
    D = (added + through @ ds[:, :, None]).flip(2)  # gradients of the states before the chunks
    dS = torch.cat((D[:, :, 1:], ds[:, :, None]), 2)
    dU = dU + kh @ dS
    dY = inverse.transpose(-1, -2) @ dU
    dv = beta[..., None] * dY
    dP = decay * (do @ U.transpose(-1, -2))
    dM = torch.where(i[:, None] > i, decay * -(dv @ U.transpose(-1, -2)), 0.0)
    dq = (from_start * do) @ S.transpose(-1, -2) + dP @ k
    as_query = dM @ k - (from_start * dv) @ S.transpose(-1, -2)
    as_key = dP.transpose(-1, -2) @ q + dM.transpose(-1, -2) @ k + to_end * (U @ dS.transpose(-1, -2))
    dbeta = (dY * (v - (from_start * k) @ S - before @ U)).sum(-1)
    dG = (q * dq + k * (as_query - as_key)).sum(-1).double()
    dg = dG.sum(-1, keepdim=True) - torch.cumsum(dG, -1) + dG + (after * dS).sum((-1, -2), dtype=torch.float64)[..., None]
    dg = torch.where(live, dg, 0.0)
    grads = (back(dq, case["Hq"]).to(dt), back(as_query + as_key, case["Hk"]).to(dt), back(dv, case["Hv"]).to(dt),
             back(dg, H).float(), back(dbeta, H))
    return (o, last, *grads) if s["state"] is None else (o, last, *grads, D[:, :, 0])


def _run_step(s):
    N = s["case"]["N"]
    if own:
        from semi_markov_crf_zero_amd import encoder
        o = encoder.gated_delta_step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["pool"][:N], slots=s["slots"])
        return o, s["pool"][:N]
    idle = s["slots"] < 0
    rows = torch.where(idle, N, s["slots"]).long()
    k, v, q = (s[n].float() for n in ("k", "v", "q"))
    old = torch.exp(s["log_decay"])[..., None, None] * s["pool"][rows]
    new = old + (s["beta"][..., None] * k)[..., None] * (v[..., None, :] - k[..., None, :] @ old)
    s["pool"][rows] = new
    o = (q[..., None, :] @ new)[..., 0, :] * q.shape[-1] ** -0.5
    return torch.where(idle[:, None, None], 0.0, o).to(s["q"].dtype), s["pool"][:N]


def _positions(s):
    case, p = s["case"], s["positions"]
    t = torch.arange(case["T"], device="cuda")
    return t.expand(case["B"], -1) if p is None else p[:, None] + t if p.dim() == 1 else p


def _turned(x, case, cos, sin):
    turn = case["turn"]
    a, b = (x[..., :turn // 2], x[..., turn // 2:turn]) if case["layout"] == "half" else (x[..., 0:turn:2], x[..., 1:turn:2])
    pair = (a * cos - b * sin, a * sin + b * cos)
    y = torch.cat(pair, -1) if case["layout"] == "half" else torch.stack(pair, -1).flatten(-2)
    return torch.cat((y, x[..., turn:]), -1)


def _run_rotary(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    if own:
        from semi_markov_crf_zero_amd import encoder
        q, k = encoder.rotary(s["q"], s["k"], s["frequencies"], positions=s["positions"], layout=case["layout"])
        if not case["train"]:
            return q, k
        return (q.detach(), k.detach(), *torch.autograd.grad((q, k), (s["q"], s["k"]), (s["dq"], s["dk"])))
    angle = (_positions(s)[..., None] * s["frequencies"])[:, :, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = [_turned(s[x].detach().float(), case, cos, sin).to(dt) for x in ("q", "k")]
    if case["train"]:
        out += [_turned(s[x].float(), case, cos, -sin).to(dt) for x in ("dq", "dk")]
    return tuple(out)


def _run_clip(s):
    case = s["case"]
    s["max_norm"] *= 0.9995  # every pass clips
    if own:
        from semi_markov_crf_zero_amd import optim
        return optim.clip_grad_norm_(s["params"], s["max_norm"], norm_type=case["order"]), s["flat"]
    if case["order"] == math.inf:
        norm = torch.stack([p.grad.abs().amax() for p in s["params"]]).amax().float()
    else:
        norm = torch.sqrt(torch.stack([p.grad.double().square().sum() for p in s["params"]]).sum()).float()
    coefficient = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    s["flat"].copy_(s["flat"].float() * coefficient)
    return norm, s["flat"]


_RUN = {"delta": _run_delta, "step": _run_step, "rotary": _run_rotary, "clip": _run_clip}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "delta":
        H, Dk, Dv, at = case["H"], case["Dk"], case["Dv"], case["B"] * case["T"]
        live = at * (0.75 if case["ragged"] else 1.0)
        qkv = ((case["Hq"] + case["Hk"]) * Dk + case["Hv"] * Dv) * e + 8 * H
        states = case["B"] * H * Dk * Dv * 4
        # forward: inputs read, o written; a state is decayed, read twice and added to
        n, flops = live * qkv + at * H * Dv * e + states * (2 if case["state"] else 1), 7 * Dk * Dv
        if case["train"]:
            # inputs and do read, their gradients written; both states rebuilt, six products with them
            n += live * (qkv + H * Dv * e) + at * qkv + states * (3 if case["state"] else 0)
            flops += 17 * Dk * Dv
        return {"bytes": n, "flops": live * H * flops}
    if op == "step":
        B, H, Dk, Dv = case["B"], case["H"], case["Dk"], case["Dv"]
        return {"bytes": B * H * (8 * Dk * Dv + e * (2 * Dk + 2 * Dv) + 8), "flops": 7 * B * H * Dk * Dv}
    if op == "rotary":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * (2 if case["train"] else 1)
        return {"bytes": 2 * n * case["D"] * e, "flops": 3 * n * case["turn"]}
    total = sum(_sizes(case))
    return {"bytes": 2 * total * e, "flops": 3 * total}


# ---------------------------------------------------------------------------------------------
# the same outputs from the definitions, in float64

def exact(case, seed):
    op = case["op"]
    if op == "delta":
        return _exact_delta(case, seed)
    s = prepare(dict(case), seed)
    if op == "step":
        N, pool = case["N"], s["pool"][:case["N"]].double()
        o = torch.zeros((case["B"], case["H"], case["Dv"]), dtype=torch.float64, device="cuda")
        for i, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                q, k, v, b, g = (s[n][i].double() for n in ("q", "k", "v", "beta", "log_decay"))
                kept = pool[slot] * torch.exp(g)[:, None, None]
                told = torch.einsum("hi,hij->hj", k, kept)
                pool[slot] = kept + torch.einsum("h,hi,hj->hij", b, k, v - told)
                o[i] = torch.einsum("hi,hij->hj", q, pool[slot]) / math.sqrt(case["Dk"])
        return o, pool
    if op == "rotary":
        if case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["D"] > 6e8:
            return None
        at = _positions(s).double()
        half = case["turn"] // 2
        pair = torch.arange(half, device="cuda")
        pair = (pair, pair + half) if case["layout"] == "half" else (2 * pair, 2 * pair + 1)
        turns = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), at[..., None] * s["frequencies"])[:, :, None]
        out = []
        for x, z in [("q", turns), ("k", turns)] + ([("dq", turns.conj()), ("dk", turns.conj())] if case["train"] else []):
            y = s[x].detach().double()
            w = torch.complex(y[..., pair[0]], y[..., pair[1]]) * z
            y[..., pair[0]], y[..., pair[1]] = w.real, w.imag
            out.append(y)
        return tuple(out)
    g = s["flat"].double()
    norm = torch.linalg.vector_norm(g, case["order"])
    coefficient = torch.clamp(s["max_norm"] * 0.9995 / (norm + 1e-6), max=1.0)
    return norm, g * coefficient


def _exact_delta(case, seed):
    B, T, H, Dk, Dv = (case[k] for k in ("B", "T", "H", "Dk", "Dv"))
    if T > 25000 or B * T * H * Dk * Dv > (2e9 if case["train"] else 6e9):
        return None
    s = prepare(dict(case), seed)
    R = B * H
    live = torch.ones((B, T), dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        live = torch.arange(T, device="cuda") < s["lengths"][:, None]

    def rows(x):
        """[B, T, heads, ...] to float64 [T, B * H, ...], 0 past the lengths."""
        x = x.detach().double().repeat_interleave(H // x.shape[2], 2)
        x = torch.where(live.view(B, T, *[1] * (x.dim() - 2)), x, 0.0)
        return x.transpose(0, 1).flatten(1, 2).contiguous()

    q, k, v, g, b = (rows(s[n]) for n in ("q", "k", "v", "log_decay", "beta"))
    a, bk = torch.exp(g), b[..., None] * k
    f64 = dict(dtype=torch.float64, device="cuda")
    S = torch.zeros((T + 1, R, Dk, Dv), **f64)  # S[t]: before position t
    if s["state"] is not None:
        S[0] = s["state"].detach().double().view(R, Dk, Dv)
    for t in range(T):
        old = S[t] * a[t, :, None, None]
        torch.baddbmm(old, bk[t, :, :, None], v[t, :, None] - torch.bmm(k[t, :, None], old), out=S[t + 1])
    scale, part = 1 / math.sqrt(Dk), max(1, 2 ** 28 // (R * Dk * Dv))

    def over(f):
        """f(slice of positions), put together."""
        got = [f(slice(i, min(T, i + part))) for i in range(0, T, part)]
        return [torch.cat(x) for x in zip(*got)]

    def back(x, heads):
        x = x.view(T, B, heads, H // heads, *x.shape[2:]).sum(3).transpose(0, 1)
        return x

    def after(i):
        return S[i.start + 1:i.stop + 1]

    o, = over(lambda i: ((q[i, :, None] @ after(i))[:, :, 0] * scale,))
    out = (back(o, H), S[T].view(B, H, Dk, Dv).clone())
    if not case["train"]:
        return out
    do = rows(s["do"]) * scale
    D = torch.zeros((T + 1, R, Dk, Dv), **f64)  # D[t + 1]: the gradient of the state after position t
    d = torch.zeros((R, Dk, Dv), **f64) if s["ds"] is None else s["ds"].double().view(R, Dk, Dv)
    for t in range(T - 1, -1, -1):
        torch.baddbmm(d, q[t, :, :, None], do[t, :, None], out=D[t + 1])
        d = torch.baddbmm(D[t + 1], k[t, :, :, None], torch.bmm(bk[t, :, None], D[t + 1]), alpha=-1) * a[t, :, None, None]

    def grads(i):
        old, new, dS = S[i] * a[i, :, None, None], after(i), D[i.start + 1:i.stop + 1]
        miss = v[i] - (k[i, :, None] @ old)[:, :, 0]
        said = (dS @ miss[..., None])[..., 0]
        dv = (bk[i, :, None] @ dS)[:, :, 0]
        dq = (new @ do[i, :, :, None])[..., 0]
        pulled = (old @ dv[..., None])[..., 0]
        dk = b[i][..., None] * said - pulled
        return dq, dk, dv, (dS * old).sum((-1, -2)) - (k[i] * pulled).sum(-1), (k[i] * said).sum(-1)

    dq, dk, dv, dg, db = over(grads)
    dg = torch.where(live.T[:, :, None].expand(T, B, H).reshape(T, R), dg, 0.0)
    out += back(dq, case["Hq"]), back(dk, case["Hk"]), back(dv, case["Hv"]), back(dg, H), back(db, H)
    return out if s["state"] is None else (*out, d.view(B, H, Dk, Dv))
