"""A stack of selective state space layers, as a model would run it.

    h = layer_norm(x) ;  u, z = h W_in^T ;  u = short_conv(u) ;  dt', b, c = u W_x^T ;  dt = dt' W_dt^T
    y = selective scan(u, dt, b, c) gated by z ;  x + y W_out^T

for prompts of different lengths (``prompt``), for single tokens that go on from them (``step``), and for training
(``prompt`` and ``backward``).

    python examples/selective_block.py        # needs a GB300
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunked_scan_mixer_gb300 as hla


class SelectiveBlock:
    """One layer: D channels outside, E inside with N states each, W taps, steps through R values a token."""

    NAMES = ("norm", "norm_bias", "w_in", "conv", "conv_bias", "w_x", "w_dt", "w_out", "a", "skip", "dt_bias")

    def __init__(self, D, E, N=16, W=4, R=None, groups=1, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        self.E, self.N, self.W, self.G, self.R = E, N, W, groups, R or max(1, D // 16)
        self.parts = (self.R, groups * N, groups * N)
        self.norm, self.norm_bias = (1 + 0.1 * rand(D)).to(dtype), (0.1 * rand(D)).to(dtype)
        self.w_in = (rand(2 * E, D) * D ** -0.5).to(dtype)
        self.conv, self.conv_bias = (rand(E, W) * W ** -0.5).to(dtype), (0.1 * rand(E)).to(dtype)
        self.w_x = (rand(sum(self.parts), E) * E ** -0.5).to(dtype)
        self.w_dt = (rand(E, self.R) * self.R ** -0.5 * 0.5).to(dtype)
        self.w_out = (rand(D, E) * E ** -0.5).to(dtype)
        # the scan's own parameters are float32: decays -1 .. -N, steps from 0.001 to 0.1, a skip of 1
        dt = torch.exp(torch.rand(E, generator=gen, device=device) * 4.6 - 6.9)
        self.a = -torch.arange(1, N + 1, device=device, dtype=torch.float32).repeat(E, 1)
        self.dt_bias = dt + torch.log(-torch.expm1(-dt))
        self.skip = torch.ones(E, device=device)

    def _split(self, u):
        """Steps, b and c of the convolution's output, as views of their projection"""
        dt, b, c = torch.matmul(u, self.w_x.t()).split(self.parts, -1)
        return dt, torch.matmul(dt, self.w_dt.t()), *(t.unflatten(-1, (self.G, self.N)) for t in (b, c))

    def _scan_args(self, gate):
        return dict(skip=self.skip, gate=gate, dt_bias=self.dt_bias)

    def state(self, B, like):
        """State before a first token, which ``step`` updates in place"""
        return (torch.zeros(B, self.W - 1, self.E, dtype=like.dtype, device=like.device),
                torch.zeros(B, self.E, self.N, device=like.device))

    def prompt(self, x, lengths=None, state=(None, None)):
        """x [B, n, D].  Returns the layer's output, the state after each prompt's last token, and what ``backward`` reads."""
        h = hla.layer_norm(x, self.norm, bias=self.norm_bias)
        p, z = torch.matmul(h, self.w_in.t()).split(self.E, -1)
        u, conv_after = hla.short_conv_forward(p, self.conv, bias=self.conv_bias, lengths=lengths, init_state=state[0],
                                               return_final_state=True)
        low, dt, b, c = self._split(u)
        y, after = hla.ssm_forward(u, dt, self.a, b, c, lengths=lengths, init_state=state[1], return_final_state=True,
                                   **self._scan_args(z))
        return x + torch.matmul(y, self.w_out.t()), (conv_after, after), (x, h, p, z, u, low, dt, b, c, y, lengths, state)

    def step(self, x, state):
        """One token for each sequence, x [B, D]; ``state`` is updated in place."""
        h = hla.layer_norm(x, self.norm, bias=self.norm_bias)
        p, z = torch.matmul(h, self.w_in.t()).split(self.E, -1)
        u = hla.short_conv_decode_step(state[0], p, self.conv, bias=self.conv_bias)
        _, dt, b, c = self._split(u)
        y = hla.ssm_decode_step(state[1], u, dt, self.a, b, c, **self._scan_args(z))
        return x + torch.matmul(y, self.w_out.t())

    def backward(self, saved, dout):
        """(dx, gradients by name) for the gradient dout of ``prompt``'s output"""
        x, h, p, z, u, low, dt, b, c, y, lengths, state = saved
        rows = lambda t: t.flatten(0, 1)  # noqa: E731
        g = {"w_out": rows(dout).t() @ rows(y)}
        s = hla.ssm_backward(u, dt, self.a, b, c, torch.matmul(dout, self.w_out), lengths=lengths, init_state=state[1],
                             **self._scan_args(z))
        g.update(a=s.da, skip=s.dskip, dt_bias=s.ddt_bias, w_dt=rows(s.ddt).t() @ rows(low))
        parts = torch.cat((torch.matmul(s.ddt, self.w_dt), s.db.flatten(2), s.dc.flatten(2)), -1)
        g["w_x"] = rows(parts).t() @ rows(u)
        k = hla.short_conv_backward(p, self.conv, s.dx + torch.matmul(parts, self.w_x), bias=self.conv_bias, lengths=lengths,
                                    init_state=state[0])
        g.update(conv=k.dweight, conv_bias=k.dbias)
        dp = torch.cat((k.dx, s.dgate), -1)
        g["w_in"] = rows(dp).t() @ rows(h)
        dx, g["norm"], g["norm_bias"] = hla.layer_norm_backward(x, self.norm, torch.matmul(dp, self.w_in))
        return dx + dout, g


class SelectiveStack:
    """Layers one after another."""

    def __init__(self, layers, *sizes, **kw):
        self.blocks = [SelectiveBlock(*sizes, seed=i, **kw) for i in range(layers)]

    def prompt(self, x, lengths=None):
        """(output, states, what ``backward`` reads)"""
        states, saved = [], []
        for b in self.blocks:
            x, s, keep = b.prompt(x, lengths)
            states.append(s)
            saved.append(keep)
        return x, states, saved

    def step(self, x, states):
        for b, s in zip(self.blocks, states):
            x = b.step(x, s)
        return x

    def backward(self, saved, dout):
        grads = []
        for b, keep in zip(reversed(self.blocks), reversed(saved)):
            dout, g = b.backward(keep, dout)
            grads.insert(0, g)
        return dout, grads


def main():
    D, n, B = 1024, 1500, 4
    model = SelectiveStack(4, D, 2 * D)
    lengths = torch.tensor([n, 700, 1, 1203], dtype=torch.int32, device="cuda")
    x = torch.randn(B, n, D, device="cuda", dtype=torch.bfloat16)
    h, states, saved = model.prompt(x, lengths)
    print("prompts of", lengths.tolist(), "tokens ->", tuple(h.shape))
    dx, grads = model.backward(saved, torch.randn_like(h))
    print("training: |dx| %.3g, |dw_in| %s" % (dx.float().norm(), ["%.3g" % g["w_in"].float().norm() for g in grads]))

    # the same step for every token: captured once, replayed
    t = torch.randn(B, D, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model.step(t, [tuple(s.clone() for s in st) for st in states])
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
    print("single tokens: %.1f us for %d sequences and %d layers" % (start.elapsed_time(end) * 1e3 / steps, B, len(states)))


if __name__ == "__main__":
    main()
