"""A sequence tagger over the semi-CRF head: features [B][T][F] to emissions,
loss and segments, trained with AdamW, whole sequences or position by
position.

    front     linear, group norm, SiLU
    layers    h += linear(norm(attention(q, k, v))), attention the linear
              attention with a decay for each head (its memory: 8 to 2048
              positions over the heads), norm a group norm of each position
              by itself, a group a head
    emissions linear

With memory="delta" attention is the gated delta rule: keys and queries of
length 1, decays and shares of a write from a linear layer (a memory of 8 to
2048 positions over the heads at the start).  With rotary=True keys and queries
are turned by their positions.

The front's norm runs over a whole sequence, or, with causal=True, over each
position by itself: then every position depends on those before it only, and
`step` gives for a stream what `emissions` gives for the sequence.

    model = SemiCRFTagger(features=40, channels=128, labels=16, max_duration=32).cuda()
    opt = optim.AdamW(model.parameters(), lr=1e-3, bits=8)
    loss = model.loss(x, lengths, gold).mean(); loss.backward()
    norm, clip = optim.grad_norm(model.parameters(), max_norm=1.0); opt.step(grad_scale=clip)
    segments = model.decode(x, lengths)

    python -m semi_markov_crf_zero_amd.tagger --steps 60     # synthetic segments
    python -m semi_markov_crf_zero_amd.tagger --memory delta --rotary --clip 1.0
"""
from __future__ import annotations

import torch
from torch import nn

from . import binding as bd
from .encoder import (gated_delta, gated_delta_step, group_norm, linear_attention,
                      linear_attention_step, rotary, rotary_frequencies)
from .training import semicrf_nll


class _Layer(nn.Module):
    def __init__(self, channels, dtype, gates=None):
        """gates: the log decays that a delta layer's heads start from."""
        super().__init__()
        self.qkv = nn.Linear(channels, 3 * channels, bias=False, dtype=dtype)
        self.weight = nn.Parameter(torch.ones(channels))
        self.bias = nn.Parameter(torch.zeros(channels))
        self.out = nn.Linear(channels, channels, dtype=dtype)
        self.gates = None
        if gates is not None:
            # log decay = -softplus(first half), share of a write = sigmoid(second half)
            self.gates = nn.Linear(channels, 2 * len(gates), dtype=dtype)
            with torch.no_grad():
                self.gates.weight.mul_(0.1)
                self.gates.bias[:len(gates)] = torch.log(torch.expm1(-gates.double())).to(dtype)
                self.gates.bias[len(gates):] = 0.0


class SemiCRFTagger(nn.Module):
    """dtype: of the linear layers and what flows between them (float32,
    bfloat16 or float16); norms' parameters, states, emissions and the head
    are float32.  memory: "linear" (linear attention with fixed decays) or
    "delta" (the gated delta rule)."""

    def __init__(self, features: int, channels: int, labels: int, max_duration: int,
                 heads: int = 4, layers: int = 2, groups: int = 8, causal: bool = False,
                 dtype=torch.float32, memory: str = "linear", rotary: bool = False):
        super().__init__()
        if memory not in ("linear", "delta"):
            raise ValueError('memory must be "linear" or "delta"')
        if channels % heads or channels % groups:
            raise ValueError("heads and groups must divide the channels")
        self.heads, self.groups, self.causal, self.dtype = heads, groups, causal, dtype
        self.front = nn.Linear(features, channels, dtype=dtype)
        self.weight = nn.Parameter(torch.ones(channels))
        self.bias = nn.Parameter(torch.zeros(channels))
        memories = torch.logspace(3, 11, heads, base=2.0) if heads > 1 else torch.tensor([128.0])
        decays = torch.log1p(-1.0 / memories)
        self.layers = nn.ModuleList(_Layer(channels, dtype, decays if memory == "delta" else None)
                                    for _ in range(layers))
        self.emit = nn.Linear(channels, labels, dtype=dtype)
        self.trans = nn.Parameter(torch.zeros(labels, labels))
        self.dur = nn.Parameter(torch.zeros(max_duration, labels))
        self.register_buffer("log_decay", decays)
        if rotary and channels // heads < 2:
            raise ValueError("heads of one channel cannot be turned")
        self.register_buffer("frequencies", rotary_frequencies(channels // heads // 2 * 2)
                             if rotary else None, persistent=False)

    def _apply(self, fn, recurse=True):
        """Frequencies follow the device and keep their type, which rotary asks for: angles
        of float32 ones are off by 2^-4 at position 2^20.  A model made without memory
        (on "meta") gets them with it: no state dict holds them."""
        held = self.frequencies
        super()._apply(fn, recurse)
        if held is not None:
            dev = self.frequencies.device
            if held.is_meta and dev.type != "meta":
                self.frequencies = rotary_frequencies(2 * held.numel(), device=dev)
            elif self.frequencies.dtype != held.dtype:
                self.frequencies = held.to(dev)
        return self

    def _norm(self, x, groups, weight, bias, act, lengths=None, alone=True):
        """The norm of each position by itself, or over the sequence."""
        if not alone:
            return group_norm(x, groups, weight, bias, lengths=lengths, activation=act)
        flat = x.reshape(-1, 1, x.shape[-1])
        return group_norm(flat, groups, weight, bias, activation=act).view(x.shape)

    def _mixed(self, layer, h, positions):
        """A layer's queries, keys and values of h [..., channels], and the
        delta rule's log decays and betas."""
        dim = h.dim() - 1
        q, k, v = layer.qkv(h).unflatten(-1, (3, self.heads, -1)).unbind(dim)
        gates = ()
        if layer.gates is not None:
            q, k = (nn.functional.normalize(t.float(), dim=-1).to(t.dtype) for t in (q, k))
            a, b = layer.gates(h).float().unflatten(-1, (2, self.heads)).unbind(dim)
            gates = -nn.functional.softplus(a), torch.sigmoid(b)
        if self.frequencies is not None:
            q, k = rotary(q, k, self.frequencies, positions=positions)
        return q, k, v, gates

    def emissions(self, x, lengths=None, states=None, starts=None):
        """Emissions [B, T, labels] float32 of x [B, T, F], and the layers'
        states after each sequence.  lengths [B] int32; states, a list as
        returned, continues sequences (causal models), with rotary from
        position starts [B] int32 on."""
        if self.frequencies is not None and states is not None and starts is None:
            raise ValueError("a rotary tagger continues sequences from given starts")
        if lengths is not None:
            # the linear layers run over the padding too: what it holds (NaN as well) times
            # a gradient of 0 must be 0
            past = torch.arange(x.shape[1], device=x.device) >= lengths[:, None]
            x = x.masked_fill(past[..., None], 0.0)
        h = self._norm(self.front(x.to(self.dtype)), self.groups, self.weight, self.bias, "silu",
                       lengths, self.causal)
        after = []
        for i, layer in enumerate(self.layers):
            q, k, v, gates = self._mixed(layer, h, starts)
            attention, gates = (gated_delta, gates) if gates else (linear_attention, (self.log_decay,))
            o, state = attention(q, k, v, *gates, lengths=lengths,
                                 state=None if states is None else states[i], return_state=True)
            after.append(state)
            h = h + layer.out(self._norm(o.flatten(2), self.heads, layer.weight, layer.bias, "none"))
        return self.emit(h).float(), after

    def loss(self, x, lengths, gold):
        """Negative log-likelihood [B] of the segmentations `gold` (the layout
        of binding.semicrf_viterbi)."""
        return semicrf_nll(self.emissions(x, lengths)[0], lengths, self.trans, self.dur, gold)

    @torch.no_grad()
    def decode(self, x, lengths):
        """The best segmentation of each sequence (binding.semicrf_viterbi)."""
        return bd.semicrf_viterbi(self.emissions(x, lengths)[0], lengths, self.trans.detach(),
                                  self.dur.detach())

    def stream_states(self, slots: int):
        """Empty states for `slots` streams, one pool a layer."""
        d = self.weight.numel() // self.heads
        return [torch.zeros((slots, self.heads, d, d), device=self.weight.device)
                for _ in self.layers]

    @torch.no_grad()
    def step(self, x, states, slots=None, positions=None):
        """Emissions [B, labels] of the next position x [B, F] of B streams
        (causal models); moves the streams' rows of the pools in `states`.
        slots [B] int32: each stream's row (its own number by default);
        positions [B] int32 where rotary: how many each has taken before."""
        if not self.causal:
            raise ValueError("only a causal tagger can take single positions")
        if self.frequencies is not None and positions is None:
            raise ValueError("a rotary tagger needs the streams' positions")
        h = self._norm(self.front(x.to(self.dtype)), self.groups, self.weight, self.bias, "silu")
        for layer, state in zip(self.layers, states):
            q, k, v, gates = self._mixed(layer, h, positions)
            if gates:
                o = gated_delta_step(q, k, v, *gates, state, slots=slots)
            else:
                o = linear_attention_step(q, k, v, self.log_decay, state, slots=slots)
            h = h + layer.out(self._norm(o.flatten(1), self.heads, layer.weight, layer.bias, "none"))
        return self.emit(h).float()


def synthetic(batch, length, features, labels, max_duration, seed, device="cuda"):
    """Sequences of labelled segments seen through noise: x [B, T, F], lengths
    and the segments.  A label shows as a fixed random direction."""
    gen = torch.Generator().manual_seed(seed)
    shape = torch.Generator().manual_seed(0)
    looks = torch.randn((labels, features), generator=shape)
    lengths = torch.randint(length // 2, length + 1, (batch,), generator=gen, dtype=torch.int32)
    gold = {k: torch.full((batch, length), -1, dtype=torch.int32)
            for k in ("seg_start", "seg_len", "seg_label")}
    gold["num_segs"] = torch.zeros(batch, dtype=torch.int32)
    x = torch.randn((batch, length, features), generator=gen)
    for b in range(batch):
        at = n = 0
        while at < lengths[b]:
            d = min(int(torch.randint(1, max_duration + 1, (), generator=gen)), int(lengths[b]) - at)
            c = int(torch.randint(labels, (), generator=gen))
            for k, v in (("seg_start", at), ("seg_len", d), ("seg_label", c)):
                gold[k][b, n] = v
            x[b, at:at + d] += looks[c]
            at, n = at + d, n + 1
        gold["num_segs"][b] = n
    return x.to(device), lengths.to(device), {k: v.to(device) for k, v in gold.items()}


def main(argv=None):
    import argparse

    from . import optim
    p = argparse.ArgumentParser(description="Trains a small tagger on synthetic segments.")
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--bits", type=int, default=32, choices=(32, 8))
    p.add_argument("--memory", default="linear", choices=("linear", "delta"))
    p.add_argument("--rotary", action="store_true")
    p.add_argument("--clip", type=float, default=None, help="largest norm of the gradients")
    p.add_argument("--dtype", default="float32", choices=("float32", "bfloat16"))
    a = p.parse_args(argv)
    torch.manual_seed(0)
    dtype = getattr(torch, a.dtype)
    model = SemiCRFTagger(24, 64, 8, 16, dtype=dtype, memory=a.memory, rotary=a.rotary).cuda()
    opt = optim.AdamW(model.parameters(), lr=3e-3, bits=a.bits, masters=dtype != torch.float32)
    losses = []
    for i in range(a.steps):
        x, lengths, gold = synthetic(8, 96, 24, 8, 16, seed=1 + i)
        loss = (model.loss(x, lengths, gold) / lengths).mean()
        opt.zero_grad()
        loss.backward()
        clip = None
        if a.clip is not None:
            _, clip = optim.grad_norm(model.parameters(), max_norm=a.clip)
        opt.step(grad_scale=clip)
        losses.append(float(loss.detach()))
        if i % 10 == 0 or i == a.steps - 1:
            print("step %d: %.4f nats a position" % (i, losses[-1]), flush=True)
    return losses


if __name__ == "__main__":
    main()
