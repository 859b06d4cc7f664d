"""A layer of first-order linear attention with everything around it, as a model would run it.

    h = block_norm(x) ;  q, k, v, z = h W_in^T ;  o = linear attention(q, k, v) ;  y = o W_out^T
    r, h' = block_join(x, y, gate z, next layer's norm)

for prompts of different lengths (``prompt``), for single tokens that go on from them with 4-bit weights
(``step``), and for training (``prompt`` and ``backward``).  The joins also form the next layer's
norm, so a stack calls block_norm once.

    python examples/mixer_block.py        # needs a GB300
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunked_scan_mixer_gb300 as hla


def quantise_w4(w, group):
    """(qweight, scales, zeros) of w4_matvec for w [N, K]: each group's range in 16 steps."""
    N, K = w.shape
    g = w.float().reshape(N, K // group, group)
    lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
    scales = ((hi - lo) / 15).clamp(min=1e-8).to(w.dtype)
    zeros = (-lo / scales.float()).round().clamp(0, 15)
    q = (g / scales.float()[..., None] + zeros[..., None]).round().clamp(0, 15).to(torch.uint8).reshape(N, K)
    return q[:, 0::2] | (q[:, 1::2] << 4), scales, zeros.to(torch.uint8)


def dequantise_w4(qweight, scales, zeros):
    """The weights that quantise_w4's parts stand for, in the scales' type."""
    N, groups = scales.shape
    q = torch.stack((qweight & 15, qweight >> 4), -1).reshape(N, groups, -1).float()
    return ((q - zeros.float()[..., None]) * scales.float()[..., None]).reshape(N, -1).to(scales.dtype)


class MixerBlock:
    """One layer: D channels, H query heads on Hk key heads of d, values of dv."""

    def __init__(self, D, H, Hk, d, dv, group=64, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        self.H, self.Hk, self.d, self.dv = H, Hk, d, dv
        self.sizes = (H * d, Hk * d, Hk * dv, D)
        self.scale = d ** -0.5
        self.gamma = 1 - torch.logspace(-1, -3, Hk, device=device)
        self.norm = (1 + 0.1 * rand(D)).to(dtype)
        self.post = (1 + 0.1 * rand(D)).to(dtype)
        self.residual = (0.5 + 0.1 * rand(D)).to(dtype)
        # the 4-bit weights serve single tokens; prompts and training use the same values as a dense matrix
        self.w4_in = quantise_w4((rand(sum(self.sizes), D) * D ** -0.5).to(dtype), group)
        self.w4_out = quantise_w4((rand(D, H * dv) * (H * dv) ** -0.5).to(dtype), group)
        self.w_in, self.w_out = dequantise_w4(*self.w4_in), dequantise_w4(*self.w4_out)

    def prompt(self, x, h, next_norm, lengths=None, state=None):
        """x [B, n, D] and its norm h.  Returns the next layer's (x, h), the state after each prompt's
        last token, and what ``backward`` reads."""
        B, n, _ = x.shape
        q, k, v, z = torch.matmul(h, self.w_in.t()).split(self.sizes, -1)
        # [B, heads, n, d] as views of the projection: the kernels read them in place
        q, k, v = (t.unflatten(-1, (heads, -1)).transpose(1, 2) for t, heads in ((q, self.H), (k, self.Hk), (v, self.Hk)))
        o, after = hla.linattn_forward(q, k, v, gamma=self.gamma, scale=self.scale, lengths=lengths, init_state=state,
                                       return_final_state=True)
        o = o.transpose(1, 2).reshape(B, n, self.H * self.dv)
        y = torch.matmul(o, self.w_out.t())
        r, h_next = hla.block_join(x, y, self.post, gate=z, gate_act="silu", scale=self.residual, next_weight=next_norm)
        return r, h_next, after, (x, h, q, k, v, z, o, y, next_norm, lengths, state)

    def step(self, x, h, next_norm, state):
        """One token for each of up to 16 sequences, x and h [N, D]; ``state`` is updated in place."""
        N = x.shape[0]
        q, k, v, z = hla.w4_matvec(h, self.w4_in[0], self.w4_in[1], zeros=self.w4_in[2]).split(self.sizes, -1)
        o = hla.linattn_decode_step(state, q.reshape(N, self.H, self.d), k.reshape(N, self.Hk, self.d),
                                    v.reshape(N, self.Hk, self.dv), gamma=self.gamma, scale=self.scale)
        y = hla.w4_matvec(o.reshape(N, -1), self.w4_out[0], self.w4_out[1], zeros=self.w4_out[2])
        return hla.block_join(x, y, self.post, gate=z, gate_act="silu", scale=self.residual, next_weight=next_norm)

    def backward(self, saved, dr, dh_next):
        """Gradients for those of ``prompt``'s r and h_next: a dict with dx and dh of its inputs and
        those of the weights ("next_norm" belongs to the layer after)."""
        x, h, q, k, v, z, o, y, next_norm, lengths, state = saved
        j = hla.block_join_backward(x, y, self.post, gate=z, gate_act="silu", scale=self.residual, next_weight=next_norm,
                                    dr=dr, dh=dh_next)
        do = torch.matmul(j.dy, self.w_out).unflatten(-1, (self.H, self.dv)).transpose(1, 2)
        dq, dk, dv = hla.linattn_backward(q, k, v, do, gamma=self.gamma, scale=self.scale, lengths=lengths,
                                          init_state=state)[:3]
        dp = torch.cat([t.transpose(1, 2).flatten(2) for t in (dq, dk, dv)] + [j.dgate], -1)
        return {"dx": j.dx, "dh": torch.matmul(dp, self.w_in), "w_in": torch.matmul(dp.flatten(0, 1).t(), h.flatten(0, 1)),
                "w_out": torch.matmul(j.dy.flatten(0, 1).t(), o.flatten(0, 1)), "post": j.dpost_weight,
                "residual": j.dscale, "next_norm": j.dnext_weight}


class MixerStack:
    """Layers one after another, and a norm at the end."""

    def __init__(self, layers, D, *sizes, **kw):
        self.blocks = [MixerBlock(D, *sizes, seed=i, **kw) for i in range(layers)]
        self.norms = [b.norm for b in self.blocks] + [torch.ones_like(self.blocks[0].norm)]

    def prompt(self, x, lengths=None):
        """(h after the last norm, states, what ``backward`` reads)"""
        first, h, states, saved = x, hla.block_norm(x, self.norms[0]), [], []
        for b, w in zip(self.blocks, self.norms[1:]):
            x, h, s, keep = b.prompt(x, h, w, lengths)
            states.append(s)
            saved.append(keep)
        return h, states, (first, saved)

    def step(self, x, states):
        h = hla.block_norm(x, self.norms[0])
        for b, w, s in zip(self.blocks, self.norms[1:], states):
            x, h = b.step(x, h, w, s)
        return h

    def backward(self, saved, dh):
        """(dx, the layers' gradients) for the gradient dh of ``prompt``'s h."""
        first, kept = saved
        dr, grads = torch.zeros_like(dh), []
        for b, keep in zip(reversed(self.blocks), reversed(kept)):
            g = b.backward(keep, dr, dh)
            dr, dh = g["dx"], g["dh"]
            grads.insert(0, g)
        dx, dnorm = hla.block_norm_backward(first, self.norms[0], dh)
        return dr + dx, grads, dnorm


def main():
    D, n, B = 1024, 1500, 4
    model = MixerStack(4, D, 16, 8, 64, 64)
    lengths = torch.tensor([n, 700, 1, 1203], dtype=torch.int32, device="cuda")
    x = torch.randn(B, n, D, device="cuda", dtype=torch.bfloat16)

    h, states, saved = model.prompt(x, lengths)
    print("prompts of", lengths.tolist(), "tokens ->", tuple(h.shape))
    dx, grads, _ = model.backward(saved, torch.randn_like(h))
    print("training: |dx| %.3g, |dw_in| %s" % (dx.float().norm(), ["%.3g" % g["w_in"].float().norm() for g in grads]))

    # the same step for every token: captured once, replayed
    t = torch.randn(B, D, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model.step(t, [s.clone() for s in states])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = model.step(t, states)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    steps = 100
    for _ in range(steps):
        t.copy_(out)  # a real model would sample a token and look its vector up
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    hla.check_status()
    print("single tokens: %.1f us for %d sequences and %d layers" % (start.elapsed_time(end) * 1e3 / steps, B, len(states)))


if __name__ == "__main__":
    main()
