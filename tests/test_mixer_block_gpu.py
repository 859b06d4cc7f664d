"""The example's layers on the GPU: prompts and single tokens against each other, gradients against
float64 automatic differentiation of the plain composition.

Tolerances, float32, relative in norm.  Products over K <= 128 terms, norms and states are each off by
some 2^-24 sqrt(K) of their terms, and a layer chains five of them; a stack of two keeps the whole
within 2^-24 * 2 * 5 * sqrt(128) * 10 = 7e-5 (the 10 for norms of small sums).
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
TOL = 7e-5


@pytest.fixture(scope="module")
def example():
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixer_block.py")
    spec = importlib.util.spec_from_file_location("mixer_block", at)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return float((a - b).norm() / b.norm().clamp(min=1e-30))


def make(example, dtype=torch.float32):
    return example.MixerStack(2, 128, 4, 2, 32, 16, group=32, dtype=dtype)


def test_prompt_then_steps(example):
    m = make(example)
    x = torch.randn(3, 41, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    lengths = torch.tensor([37, 1, 20], dtype=torch.int32, device="cuda")
    whole, _, _ = m.prompt(x)
    h, states, _ = m.prompt(x[:, :37].contiguous(), lengths)
    rows = torch.arange(3, device="cuda")
    assert rel(h[rows, lengths.long() - 1], whole[rows, lengths.long() - 1]) <= TOL
    for i in range(4):
        at = lengths.long() + i
        assert rel(m.step(x[rows, at].contiguous(), states), whole[rows, at]) <= TOL


def test_gradients(example):
    m = make(example)
    gen = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(2, 19, 128, device="cuda", generator=gen)
    h, _, saved = m.prompt(x)
    dh = torch.randn(h.shape, device="cuda", generator=gen)
    dx, grads, dnorm = m.backward(saved, dh)

    def leaf(t):
        return t.detach().double().cpu().requires_grad_()

    norm = lambda t, w: t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    x64, norms = leaf(x), [leaf(w) for w in m.norms]
    ws = [{n: leaf(getattr(b, n)) for n in ("w_in", "w_out", "post", "residual")} for b in m.blocks]
    r, hh = x64, norm(x64, norms[0])
    for b, w, nw in zip(m.blocks, ws, norms[1:]):
        q, k, v, z = (hh @ w["w_in"].t()).split(b.sizes, -1)
        q, k, v = (t.unflatten(-1, (n, -1)) for t, n in ((q, b.H), (k, b.Hk), (v, b.Hk)))
        k, v = (t.repeat_interleave(b.H // b.Hk, 2) for t in (k, v))
        g = b.gamma.double().cpu().repeat_interleave(b.H // b.Hk)
        t = torch.arange(x.shape[1])
        lag = t[:, None] - t[None, :]
        decay = torch.where(lag >= 0, g[:, None, None] ** lag.clamp(min=0), 0.0)
        s = torch.einsum("bihd,bjhd->bhij", q, k) * decay * b.scale
        o = torch.einsum("bhij,bjhd->bihd", s, v).flatten(2)
        r = r + w["residual"] * torch.nn.functional.silu(z) * norm(o @ w["w_out"].t(), w["post"])
        hh = norm(r, nw)
    assert rel(h, hh.detach()) <= TOL
    (hh * dh.double().cpu()).sum().backward()
    assert rel(dx, x64.grad) <= TOL
    assert rel(dnorm, norms[0].grad) <= TOL
    for g, w, nw in zip(grads, ws, norms[1:]):
        for n in w:
            assert rel(g[n], w[n].grad) <= TOL, n
        assert rel(g["next_norm"], nw.grad) <= TOL


def test_bf16_stack_runs_in_a_graph(example):
    m = make(example, torch.bfloat16)
    x = torch.randn(2, 130, 128, device="cuda", dtype=torch.bfloat16)
    h, states, _ = m.prompt(x)
    t = x[:, 0].contiguous()
    want_states = [s.clone() for s in states]
    want = m.step(t, want_states)
    graph = torch.cuda.CUDAGraph()
    keep = [s.clone() for s in states]
    with torch.cuda.graph(graph):
        out = m.step(t, states)
    for s, k in zip(states, keep):
        s.copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(torch.equal(a, b) for a, b in zip(states, want_states))
