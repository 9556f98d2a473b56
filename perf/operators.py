"""The encoder and training operators as they are measured: linear attention with a decay for each
head (whole sequences, training, single tokens), group norm with an activation over
channels-last sequences (inference, training), and the AdamW step over many tensors (states in 32
bits or in 8).

`own` False: elementary torch operations in float32, rounded once to the output's type.
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
        dict(name="linattn-nlp-fwd", op="linattn", train=False, B=32, T=512, H=4, Hq=4, Hk=4, Hv=4, Dk=64, Dv=64,
             dtype="bf16", ragged=True, state=False),
        # One chromosome-length sequence read in inference, continued from a prefix's state (2^20
        # positions, the extreme workload).
        dict(name="linattn-extreme-fwd", op="linattn", train=False, B=1, T=1048576, H=4, Hq=4, Hk=4, Hv=4, Dk=64,
             Dv=64, dtype="bf16", ragged=False, state=True),
        # A training step of a speech encoder with 256 channels (16 utterances, the speech workload).
        dict(name="linattn-speech-train", op="linattn", train=True, B=16, T=4096, H=4, Hq=4, Hk=4, Hv=4, Dk=64, Dv=64,
             dtype="bf16", ragged=True, state=False),
        # A genome encoder trained in float32 with keys shared by two heads and odd sizes.
        dict(name="linattn-genome-train", op="linattn", train=True, B=2, T=50001, H=4, Hq=4, Hk=2, Hv=4, Dk=40, Dv=72,
             dtype="f32", ragged=False, state=True),
        # Streams tagged as they arrive: the next token of a few streams (latency) ...
        dict(name="linattn-step-small", op="step", B=4, N=16, H=4, Dk=64, Dv=64, dtype="bf16"),
        # ... and of many streams of a wide encoder.
        dict(name="linattn-step-large", op="step", B=256, N=320, H=16, Dk=128, Dv=128, dtype="bf16"),
        # The front end of the sentence tagger.
        dict(name="groupnorm-nlp-fwd", op="groupnorm", train=False, B=32, T=512, C=256, G=32, act="silu",
             dtype="bf16", ragged=True),
        # The front end of the speech encoder in a training step.
        dict(name="groupnorm-speech-train", op="groupnorm", train=True, B=16, T=4096, C=256, G=32, act="silu",
             dtype="bf16", ragged=True),
        # The 2^20-position sequence with 64 channels in float32, in inference.
        dict(name="groupnorm-extreme-fwd", op="groupnorm", train=False, B=1, T=1048576, C=64, G=8, act="gelu",
             dtype="f32", ragged=False),
        # Each position of a batch normalised by itself (a norm over heads of odd width), training.
        dict(name="groupnorm-positions-train", op="groupnorm", train=True, B=16384, T=1, C=250, G=10, act="none",
             dtype="f32", ragged=False),
        # The parameters of a small tagger: many small tensors, states in 32 bits (latency).
        dict(name="adamw-tagger-32", op="adamw", tensors=120, total=1500000, dtype="f32", grad="f32", bits=32),
        # A wide encoder trained with bfloat16 gradients and states in 8 bits.
        dict(name="adamw-wide-8", op="adamw", tensors=64, total=80000000, dtype="f32", grad="bf16", bits=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linattn", "linattn", "step", "groupnorm", "groupnorm", "adamw"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if kind == "linattn":
        H = rng.choice([1, 2, 3, 4, 6, 8])
        share = rng.choice(["none", "none", "kv", "qk"])
        few = max(h for h in (1, 2, 3) if H % h == 0)
        Dk, Dv = rng.choice([16, 32, 40, 64, 64, 96, 128]), rng.choice([16, 32, 64, 64, 72, 128])
        tokens = _log(rng, 600, 400000)
        T = min(tokens, _log(rng, 1, 300000))
        B = max(1, min(64, tokens // T))
        return dict(op="linattn", train=rng.random() < 0.5, B=B, T=T, H=H, Hq=few if share == "qk" else H,
                    Hk=few if share != "none" else H, Hv=few if share == "kv" else H, Dk=Dk, Dv=Dv, dtype=dtype,
                    ragged=rng.random() < 0.5, state=rng.random() < 0.5)
    if kind == "step":
        B = _log(rng, 1, 256)
        return dict(op="step", B=B, N=B + rng.randrange(0, 65), H=rng.choice([1, 2, 4, 5, 8, 16]),
                    Dk=rng.choice([32, 40, 64, 64, 128]), Dv=rng.choice([32, 64, 64, 72, 128]), dtype=dtype)
    if kind == "groupnorm":
        G = rng.choice([1, 2, 4, 8, 10, 16, 32])
        C = G * rng.choice([1, 3, 4, 8, 8, 16, 25])
        positions = _log(rng, 100, min(1000000, 60000000 // C))
        T = min(positions, _log(rng, 1, 1000000))
        return dict(op="groupnorm", train=rng.random() < 0.5, B=max(1, positions // T), T=T, C=C, G=G,
                    act=rng.choice(["none", "silu", "silu", "gelu", "relu"]), dtype=dtype,
                    ragged=T > 1 and rng.random() < 0.5)
    return dict(op="adamw", tensors=_log(rng, 1, 400), total=_log(rng, 3000, 40000000),
                dtype=rng.choice(["f32", "f32", "bf16"]), grad=rng.choice(["f32", "bf16"]),
                bits=rng.choice([32, 8]))


# ---------------------------------------------------------------------------------------------
# inputs

def _lengths(case, gen):
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return None
    return torch.randint((T + 1) // 2, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)


def _log_decay(H):
    # from a memory of 8 positions to one of 2048
    e = torch.linspace(3.0, 11.0, H, dtype=torch.float64) if H > 1 else torch.tensor([7.0], dtype=torch.float64)
    return torch.log1p(-torch.exp2(-e)).float().cuda()


def _sizes(case):
    """Matrices and vectors of an encoder, the vectors a quarter of the tensors; odd sizes among them."""
    n, total = case["tensors"], case["total"]
    vec = [64 + 37 * i % 448 for i in range(n // 4)]
    rest = max(1, n - len(vec))
    share = [1.0 + (i * 7 % 11) for i in range(rest)]
    left = max(rest, total - sum(vec))
    return vec + [max(1, int(left * s / sum(share))) for s in share]


BLOCK = 256  # elements that share one scale of an 8-bit state


def _places(sizes):
    """Starts of the tensors in one buffer, each on 512 bytes and on whole blocks."""
    at, places = 0, []
    for n in sizes:
        places.append(at)
        at += -(-n // BLOCK) * BLOCK
    return places, at


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind, op = dict(device="cuda", generator=gen), case["op"]
    if op == "linattn":
        dt = DTYPES[case["dtype"]]
        B, T, H, Dk, Dv = (case[k] for k in ("B", "T", "H", "Dk", "Dv"))
        s = {"case": case, "lengths": _lengths(case, gen), "log_decay": _log_decay(H)}
        for name, heads, d in (("q", case["Hq"], Dk), ("k", case["Hk"], Dk), ("v", case["Hv"], Dv)):
            s[name] = torch.randn((B, T, heads, d), dtype=dt, **kind)
        s["state"] = torch.randn((B, H, Dk, Dv), **kind) if case["state"] else None
        if case["train"]:
            s["do"] = torch.randn((B, T, H, Dv), dtype=dt, **kind)
            s["ds"] = torch.randn((B, H, Dk, Dv), **kind) if case["state"] else None
            for name in ("q", "k", "v", "state"):
                if s[name] is not None:
                    s[name].requires_grad_(True)
        return s
    if op == "step":
        dt = DTYPES[case["dtype"]]
        B, N, H, Dk, Dv = (case[k] for k in ("B", "N", "H", "Dk", "Dv"))
        slots = torch.randperm(N, device="cuda", generator=gen)[:B].to(torch.int32)
        if B > 8:
            slots[B // 3] = -1  # a stream that has ended
        # row N takes what the plain form writes for such streams
        pool = torch.randn((N + 1, H, Dk, Dv), **kind)
        return {"case": case, "slots": slots, "log_decay": _log_decay(H), "pool": pool,
                "q": torch.randn((B, H, Dk), dtype=dt, **kind), "k": torch.randn((B, H, Dk), dtype=dt, **kind),
                "v": torch.randn((B, H, Dv), dtype=dt, **kind)}
    if op == "groupnorm":
        dt, C = DTYPES[case["dtype"]], case["C"]
        shape = (case["B"], case["T"], C)
        s = {"case": case, "lengths": _lengths(case, gen),
             "x": (torch.randn(shape, **kind) * 1.5 + torch.randn(C, **kind)).to(dt),
             "weight": 1.0 + 0.2 * torch.randn(C, **kind), "bias": 0.2 * torch.randn(C, **kind)}
        if case["train"]:
            s["dy"] = torch.randn(shape, dtype=dt, **kind)
            for name in ("x", "weight", "bias"):
                s[name].requires_grad_(True)
        return s
    sizes = _sizes(case)
    places, total = _places(sizes)
    used = torch.zeros(total, device="cuda")
    for at, n in zip(places, sizes):
        used[at:at + n] = 1.0

    def flat(std):
        return torch.randn(total, **kind) * used * std

    p, g = flat(0.05).to(DTYPES[case["dtype"]]), flat(1e-3).to(DTYPES[case["grad"]])
    m, v = flat(3e-4), (flat(1e-3) ** 2 + 1e-8 * used)
    s = {"case": case, "p": p, "step": 100, "cut": (places, sizes),
         "grads": [g[at:at + n] for at, n in zip(places, sizes)],
         "hyper": dict(lr=3e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)}
    if case["bits"] == 8:
        s["m"], s["ms"] = _to_signed8(m)
        s["r"], s["rs"] = _to_root8(v)
    else:
        s["m"], s["v"] = m, v
    if own:
        s["plan"] = _plan(s)
    return s


# ---------------------------------------------------------------------------------------------
# one pass

def run(state):
    return _RUN[state["case"]["op"]](state)


def _run_linattn(s):
    case = s["case"]
    if own:
        from semi_markov_crf_zero_amd import encoder
        if not case["train"]:
            return encoder.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], lengths=s["lengths"],
                                            state=s["state"], return_state=True)
        o, last = encoder.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], lengths=s["lengths"],
                                           state=s["state"], return_state=True)
        wrt = [s[n] for n in ("q", "k", "v", "state") if s[n] is not None]
        if s["ds"] is None:
            return (o.detach(), last.detach(), *torch.autograd.grad(o, wrt, s["do"]))
        return (o.detach(), last.detach(), *torch.autograd.grad((o, last), wrt, (s["do"], s["ds"])))
    return _plain_linattn(s)


def _heads(x, mask, H):
    """[B, T, heads, D] to float32 [B, H, T, D] with shared heads repeated and nothing past the lengths."""
    x = x.detach().float()
    if mask is not None:
        x = torch.where(mask, x, 0.0)
    return x.permute(0, 2, 1, 3).repeat_interleave(H // x.shape[2], dim=1)


def _decayed(a, b, c, g, L=256):
    """sum over j <= i of exp(g (i - j)) (a_i . b_j) c_j, in blocks of L positions."""
    B, H, T, _ = a.shape
    L = min(L, T)
    N = -(-T // L)
    a, b, c = (torch.nn.functional.pad(x, (0, 0, 0, N * L - T)).reshape(B, H, N, L, -1) for x in (a, b, c))
    i = torch.arange(L, device=a.device)
    far = (i[:, None] - i).clamp(min=0)
    inside = torch.where(i[:, None] >= i, torch.exp(g[:, None, None] * far), 0.0)[:, None]
    out = ((a @ b.transpose(-1, -2)) * inside) @ c
    if N > 1:
        added = (b * torch.exp(g[:, None, None] * (L - 1 - i)[:, None])[:, None]).transpose(-1, -2) @ c
        n = torch.arange(N, device=a.device)
        gap = (n[:, None] - n - 1).clamp(min=0) * L
        between = torch.where(n[:, None] > n, torch.exp(g[:, None, None] * gap), 0.0)
        before = (between @ added.reshape(B, H, N, -1)).reshape(added.shape)
        out = out + (a * torch.exp(g[:, None, None] * (i + 1)[:, None])[:, None]) @ before
    return out.reshape(B, H, N * L, -1)[:, :, :T]


def _shared(x, heads):
    """The gradient of a shared head: the sum over the heads that use it. [B, H, T, D] to [B, T, heads, D]."""
    B, H, T, D = x.shape
    return x.reshape(B, heads, H // heads, T, D).sum(2).permute(0, 2, 1, 3)


def _plain_linattn(s):
    case, g = s["case"], s["log_decay"]
    B, T, H, Dk, dt = case["B"], case["T"], case["H"], case["Dk"], DTYPES[case["dtype"]]
    scale = Dk ** -0.5
    t = torch.arange(T, device=g.device)
    n = s["lengths"] if s["lengths"] is not None else torch.full((B,), T, device=g.device)
    mask = (t < n[:, None])[:, :, None, None] if s["lengths"] is not None else None
    live = (t < n[:, None])[:, None, :, None]
    q, k, v = (_heads(s[x], mask, H) for x in ("q", "k", "v"))
    gh = g[None, :, None]
    left = (n[:, None, None] - 1 - t).clamp(min=0)
    to_end = torch.exp(gh * left)[..., None] * live      # from position t to the last one
    to_start = torch.exp(gh * (t + 1))[..., None] * live  # from before the first one to position t
    o = _decayed(q, k, v, g)
    last = (k * to_end).transpose(-1, -2) @ v
    if s["state"] is not None:
        first = s["state"].detach()
        o = o + (q * to_start) @ first
        last = last + torch.exp(gh * n[:, None, None])[..., None] * first
    o = (o * scale).permute(0, 2, 1, 3)
    o = (torch.where(mask, o, 0.0) if mask is not None else o).to(dt).contiguous()
    if not case["train"]:
        return o, last
    do = s["do"].float().permute(0, 2, 1, 3) * live * scale
    dq = _decayed(do, v, k, g)
    dk = _decayed(v.flip(2), do.flip(2), q.flip(2), g).flip(2)
    dv = _decayed(k.flip(2), q.flip(2), do.flip(2), g).flip(2)
    grads = []
    if s["state"] is not None:
        ds = s["ds"]
        dq = dq + (do * to_start) @ first.transpose(-1, -2)
        dk = dk + (v * to_end) @ ds.transpose(-1, -2)
        dv = dv + (k * to_end) @ ds
        grads = [(q * to_start).transpose(-1, -2) @ do + torch.exp(gh * n[:, None, None])[..., None] * ds]
    out = [_shared(x * live, case[h]).to(dt).contiguous() for x, h in ((dq, "Hq"), (dk, "Hk"), (dv, "Hv"))]
    return (o, last, *out, *grads)


def _run_step(s):
    N = s["case"]["N"]
    if own:
        from semi_markov_crf_zero_amd import encoder
        o = encoder.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["pool"][:N], slots=s["slots"])
        return o, s["pool"][:N]
    idle = s["slots"] < 0
    rows = torch.where(idle, N, s["slots"]).long()
    k, v, q = (s[n].float() for n in ("k", "v", "q"))
    new = torch.exp(s["log_decay"])[:, None, None] * s["pool"][rows] + k[..., None] * v[..., None, :]
    s["pool"][rows] = new
    o = (q[..., None, :] @ new)[..., 0, :] * q.shape[-1] ** -0.5
    return torch.where(idle[:, None, None], 0.0, o).to(s["q"].dtype), s["pool"][:N]


def _act(z, act):
    """The activation and its derivative."""
    if act == "silu":
        e = 1.0 / (1.0 + torch.exp(-z))
        return z * e, e * (1.0 + z * (1.0 - e))
    if act == "gelu":
        c = 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5))
        return z * c, c + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    if act == "relu":
        return z.clamp(min=0.0), (z > 0).to(z.dtype)
    return z, torch.ones_like(z)


def _run_groupnorm(s):
    case = s["case"]
    if own:
        from semi_markov_crf_zero_amd import encoder
        y = encoder.group_norm(s["x"], case["G"], s["weight"], s["bias"], lengths=s["lengths"],
                               activation=case["act"])
        if not case["train"]:
            return y
        return (y.detach(), *torch.autograd.grad(y, (s["x"], s["weight"], s["bias"]), s["dy"]))
    B, T, C, G, dt = case["B"], case["T"], case["C"], case["G"], DTYPES[case["dtype"]]
    x, w, b = s["x"].detach().float().view(B, T, G, C // G), s["weight"].detach(), s["bias"].detach()
    n = torch.full((B,), T, device=x.device) if s["lengths"] is None else s["lengths"]
    count = (n * (C // G)).clamp(min=1)[:, None, None, None]
    live = (torch.arange(T, device=x.device) < n[:, None])[:, :, None, None]
    x = torch.where(live, x, 0.0) if s["lengths"] is not None else x
    off = torch.where(live, x - x.sum((1, 3), keepdim=True) / count, 0.0)
    rstd = 1.0 / torch.sqrt((off * off).sum((1, 3), keepdim=True) / count + 1e-5)
    h = off * rstd
    w, b = w.view(G, -1), b.view(G, -1)
    y, slope = _act(h * w + b, case["act"])
    y = torch.where(live, y, 0.0).to(dt).view(B, T, C)
    if not case["train"]:
        return y
    dz = torch.where(live, s["dy"].float().view(h.shape) * slope, 0.0)
    dw, db = (dz * h).sum((0, 1)).view(-1), dz.sum((0, 1)).view(-1)
    dh = dz * w
    dx = rstd * (dh - dh.sum((1, 3), keepdim=True) / count - h * ((dh * h).sum((1, 3), keepdim=True) / count))
    return y, torch.where(live, dx, 0.0).to(dt).view(B, T, C), dw, db


# The 8-bit states. m: signed, 4 bits of exponent and 3 of mantissa (float8_e4m3fn), times its
# block's scale, which takes the block's largest magnitude to 448. v: its root, unsigned, 4 bits of
# exponent and 4 of mantissa, times its block's scale, which takes the largest root to 496. A block
# with nothing over 2^-100 holds zeros. All arithmetic in float32, each operation rounded by itself.

TINY = 2.0 ** -100


def _to_signed8(m):
    top = m.view(-1, BLOCK).abs().amax(1, keepdim=True)
    inv = torch.where(top > TINY, top.reciprocal() * 448.0, 0.0)
    return (m.view(-1, BLOCK) * inv).to(torch.float8_e4m3fn).view(-1), (top * (1.0 / 448.0)).view(-1)


def _from_signed8(code, scale):
    return (code.view(-1, BLOCK).float() * scale[:, None]).view(-1)


def _to_root8(v):
    root = torch.sqrt(v).view(-1, BLOCK)
    top = root.amax(1, keepdim=True)
    x = root * torch.where(top > TINY, top.reciprocal() * 496.0, 0.0)
    # 2^-6 is the smallest value with a whole mantissa; below it steps of 2^-10
    bits = x.view(torch.int32)
    normal = ((bits + 0x3FFFF + ((bits >> 19) & 1)) >> 19) - (120 << 4)
    small = torch.round(x * 1024.0).to(torch.int32)
    code = torch.where(x >= 0.015625, normal, small)
    return code.to(torch.uint8).view(-1), (top * (1.0 / 496.0)).view(-1)


def _from_root8(code, scale):
    c = code.view(-1, BLOCK).to(torch.int32)
    x = torch.where(c >= 16, ((c + (120 << 4)) << 19).view(torch.float32), c.float() * (1.0 / 1024.0))
    root = x * scale[:, None]
    return (root * root).view(-1)


def _plan(s):
    from semi_markov_crf_zero_amd import optim
    places, sizes = s["cut"]

    def cut(x, by=1):
        return [x[at // by:-(-(at + n) // by)] for at, n in zip(places, sizes)]

    if s["case"]["bits"] == 8:
        return optim.AdamWPlan(cut(s["p"]), bits=8, exp_avg=list(zip(cut(s["m"]), cut(s["ms"], BLOCK))),
                               exp_avg_sq=list(zip(cut(s["r"]), cut(s["rs"], BLOCK))))
    return optim.AdamWPlan(cut(s["p"]), exp_avg=cut(s["m"]), exp_avg_sq=cut(s["v"]))


def _run_adamw(s):
    s["step"] += 1
    hy, p, small = s["hyper"], s["p"], s["case"]["bits"] == 8
    if own:
        s["plan"].run(s["grads"], s["step"], **hy)
        if not small:
            return p, s["m"], s["v"]
        from semi_markov_crf_zero_amd import optim
        return p, optim.moment_values(s["m"], s["ms"]), optim.moment_values(s["r"], s["rs"])
    places, sizes = s["cut"]
    m = _from_signed8(s["m"], s["ms"]) if small else s["m"]
    v = _from_root8(s["r"], s["rs"]) if small else s["v"]
    b1, b2 = hy["beta1"], hy["beta2"]
    P, M, V = ([x[at:at + n] for at, n in zip(places, sizes)] for x in (p, m, v))
    G = [x.float() for x in s["grads"]]
    torch._foreach_mul_(M, b1)
    torch._foreach_add_(M, torch._foreach_mul(G, 1.0 - b1))
    torch._foreach_mul_(V, b2)
    torch._foreach_add_(V, torch._foreach_mul(torch._foreach_mul(G, 1.0 - b2), G))
    down = torch._foreach_sqrt(V)
    torch._foreach_mul_(down, 1.0 / math.sqrt(1.0 - b2 ** s["step"]))
    torch._foreach_add_(down, hy["eps"])
    move = torch._foreach_div(M, down)
    torch._foreach_mul_(move, hy["lr"] / (1.0 - b1 ** s["step"]))
    new = torch._foreach_mul([x.float() for x in P], 1.0 - hy["lr"] * hy["weight_decay"])
    torch._foreach_sub_(new, move)
    torch._foreach_copy_(P, new)
    if not small:
        return p, m, v
    s["m"], s["ms"] = _to_signed8(m)
    s["r"], s["rs"] = _to_root8(v)
    return p, _from_signed8(s["m"], s["ms"]), _from_root8(s["r"], s["rs"])


_RUN = {"linattn": _run_linattn, "step": _run_step, "groupnorm": _run_groupnorm, "adamw": _run_adamw}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "linattn":
        e, H, Dk, Dv = SIZE[case["dtype"]], case["H"], case["Dk"], case["Dv"]
        at = case["B"] * case["T"]
        live = at * (0.75 if case["ragged"] else 1.0)
        qkv = (case["Hq"] + case["Hk"]) * Dk + case["Hv"] * Dv
        states = case["B"] * H * Dk * Dv * 4
        # forward: q, k, v read, o written; a state is one product to update and one to read
        n, flops = live * qkv * e + at * H * Dv * e + states * (2 if case["state"] else 1), 4 * Dk * Dv
        if case["train"]:
            # q, k, v and do read, dq, dk, dv written; both states rebuilt, three products with them
            n += live * (qkv + H * Dv) * e + at * qkv * e + states * (3 if case["state"] else 0)
            flops += 10 * Dk * Dv
        return {"bytes": n, "flops": live * H * flops}
    if op == "step":
        B, H, Dk, Dv, e = case["B"], case["H"], case["Dk"], case["Dv"], SIZE[case["dtype"]]
        return {"bytes": B * H * (8 * Dk * Dv + e * (2 * Dk + 2 * Dv)), "flops": 5 * B * H * Dk * Dv}
    if op == "groupnorm":
        at = case["B"] * case["T"] * case["C"]
        live = at * (0.75 if case["ragged"] else 1.0)
        e = SIZE[case["dtype"]]
        n, flops = live * e + at * e, 9 * live
        if case["train"]:
            n, flops = n + 2 * live * e + at * e, flops + 20 * live
        return {"bytes": n + 8 * case["C"], "flops": flops}
    total, g, p = sum(_sizes(case)), SIZE[case["grad"]], SIZE[case["dtype"]]
    # 8 bits: both states read and written as codes, and their values returned
    states = 4 * (1 + 4.0 / BLOCK) + 8 if case["bits"] == 8 else 16
    return {"bytes": total * (2 * p + g + states), "flops": 14 * total}


# ---------------------------------------------------------------------------------------------
# the same outputs from the definitions, in float64

def exact(case, seed):
    op = case["op"]
    if op == "linattn":
        return _exact_linattn(case, seed)
    s = prepare(dict(case), seed)
    if op == "step":
        N, pool = case["N"], s["pool"][:case["N"]].double()
        o = torch.zeros((case["B"], case["H"], case["Dv"]), dtype=torch.float64, device="cuda")
        for i, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                q, k, v = (s[n][i].double() for n in "qkv")
                pool[slot] = (pool[slot] * torch.exp(s["log_decay"].double())[:, None, None]
                              + torch.einsum("hi,hj->hij", k, v))
                o[i] = torch.einsum("hi,hij->hj", q, pool[slot]) / math.sqrt(case["Dk"])
        return o, pool
    if op == "groupnorm":
        return _exact_groupnorm(case, s)
    hy, t = s["hyper"], s["step"] + 1
    g = torch.zeros(s["p"].shape, dtype=torch.float64, device="cuda")
    for at, x in zip(s["cut"][0], s["grads"]):
        g[at:at + x.numel()] = x.double()
    if case["bits"] == 8:
        m = s["m"].double() * s["ms"].double().repeat_interleave(BLOCK)
        c = s["r"].double()
        root = torch.where(c < 16, c / 1024, (1 + (c % 16) / 16) * torch.exp2(torch.floor(c / 16) - 7))
        v = (root * s["rs"].double().repeat_interleave(BLOCK)) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = hy["beta1"] * m + (1 - hy["beta1"]) * g
    v = hy["beta2"] * v + (1 - hy["beta2"]) * g * g
    p = s["p"].double() * (1 - hy["lr"] * hy["weight_decay"])
    p = p - hy["lr"] * (m / (1 - hy["beta1"] ** t)) / (torch.sqrt(v / (1 - hy["beta2"] ** t)) + hy["eps"])
    # which of two neighbouring codes holds a new state is settled by a rounding
    return (p, None, None) if case["bits"] == 8 else (p, m, v)


def _exact_linattn(case, seed):
    B, T, H, Dk, Dv = (case[k] for k in ("B", "T", "H", "Dk", "Dv"))
    if B * H * float(T) * T > 6e10:
        return None
    s = prepare(dict(case), seed)
    n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    f64 = dict(dtype=torch.float64, device="cuda")
    o, last = torch.zeros((B, T, H, Dv), **f64), torch.zeros((B, H, Dk, Dv), **f64)
    dq, dk, dv = (torch.zeros((B, T, case[h], d), **f64) for h, d in (("Hq", Dk), ("Hk", Dk), ("Hv", Dv)))
    dfirst = torch.zeros((B, H, Dk, Dv), **f64)
    scale, rows = 1 / math.sqrt(Dk), 2048
    for b in range(B):
        L = n[b]
        t = torch.arange(L, **f64)
        for h in range(H):
            g = float(s["log_decay"][h])
            hq, hk, hv = (h * case[x] // H for x in ("Hq", "Hk", "Hv"))
            q, k, v = (s[x].detach()[b, :L, i].double() for x, i in (("q", hq), ("k", hk), ("v", hv)))
            w0, w1 = torch.exp(g * (t + 1))[:, None], torch.exp(g * (L - 1 - t))[:, None]
            last[b, h] = (w1 * k).T @ v
            do = s["do"][b, :L, h].double() if case["train"] else None
            for i in range(0, L, rows):
                j = min(L, i + rows)
                decay = torch.exp(g * (t[i:j, None] - t[:j]).clamp(min=0)) * (t[i:j, None] >= t[:j]) * scale
                A = (q[i:j] @ k[:j].T) * decay
                o[b, i:j, h] = A @ v[:j]
                if case["train"]:
                    dA = (do[i:j] @ v[:j].T) * decay
                    dq[b, i:j, hq] += dA @ k[:j]
                    dk[b, :j, hk] += dA.T @ q[i:j]
                    dv[b, :j, hv] += A.T @ do[i:j]
            if s["state"] is not None:
                first = s["state"].detach()[b, h].double()
                o[b, :L, h] += scale * (w0 * q) @ first
                last[b, h] += math.exp(g * L) * first
                if case["train"]:
                    ds = s["ds"][b, h].double()
                    dq[b, :L, hq] += scale * (w0 * do) @ first.T
                    dk[b, :L, hk] += (w1 * v) @ ds.T
                    dv[b, :L, hv] += (w1 * k) @ ds
                    dfirst[b, h] = scale * (w0 * q).T @ do + math.exp(g * L) * ds
    if not case["train"]:
        return o, last
    return (o, last, dq, dk, dv, dfirst) if s["state"] is not None else (o, last, dq, dk, dv)


def _exact_groupnorm(case, s):
    B, T, C, G = case["B"], case["T"], case["C"], case["G"]
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"]
    w, b = s["weight"].detach().double(), s["bias"].detach().double()
    y = torch.zeros((B, T, C), dtype=torch.float64, device="cuda")
    dx, dw, db = torch.zeros_like(y), torch.zeros_like(w), torch.zeros_like(b)
    alike = {}
    for i, length in enumerate(n.tolist()):
        alike.setdefault(length, []).append(i)
    for L, who in alike.items():
        if not L:
            continue
        for part in torch.tensor(who, device="cuda").split(max(1, (1 << 27) // (L * C))):
            x = s["x"].detach()[part, :L].double().view(len(part), L, G, C // G)
            var, mean = torch.var_mean(x, dim=(1, 3), unbiased=False, keepdim=True)
            sd = torch.sqrt(var + 1e-5)
            h = ((x - mean) / sd).view(len(part), L, C)
            z = (h * w + b).requires_grad_(case["train"])
            f = {"none": lambda u: u * 1.0, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
                 "relu": torch.relu}[case["act"]](z)
            y[part, :L] = f.detach()
            if case["train"]:
                dz, = torch.autograd.grad(f, z, s["dy"][part, :L].double())
                dw += (dz * h).sum((0, 1))
                db += dz.sum((0, 1))
                dh = (dz * w).view(x.shape)
                hv = h.view(x.shape)
                d = dh - dh.mean((1, 3), keepdim=True) - hv * (dh * hv).mean((1, 3), keepdim=True)
                dx[part, :L] = (d / sd).view(len(part), L, C)
    return (y, dx, dw, db) if case["train"] else y
