"""The example's layers on the GPU: prompts and single tokens against each other, gradients against float64 automatic
differentiation of the plain composition.

Tolerances, float32, relative in norm.  Products over K <= 96 terms, norms and scans of at most 41 tokens are each off by some
2^-24 sqrt(K) of their terms, and a layer chains seven of them; a stack of two keeps the whole within
2^-24 * 2 * 7 * sqrt(96) * 10 = 8e-5 (the 10 for norms of small sums)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
TOL = 8e-5


@pytest.fixture(scope="module")
def example():
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "selective_block.py")
    spec = importlib.util.spec_from_file_location("selective_block", at)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(autouse=True)
def full_precision():
    before = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = before


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return float((a - b).norm() / b.norm().clamp(min=1e-30))


def make(example, dtype=torch.float32, groups=2):
    return example.SelectiveStack(2, 48, 96, 16, 4, 5, groups=groups, dtype=dtype)


def test_prompt_then_steps(example):
    m = make(example)
    x = torch.randn(3, 41, 48, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    lengths = torch.tensor([37, 1, 20], dtype=torch.int32, device="cuda")
    whole, _, _ = m.prompt(x)
    h, states, _ = m.prompt(x[:, :37].contiguous(), lengths)
    at = torch.arange(3, device="cuda")
    assert rel(h[at, lengths.long() - 1], whole[at, lengths.long() - 1]) <= TOL
    for i in range(4):
        t = lengths.long() + i
        assert rel(m.step(x[at, t].contiguous(), states), whole[at, t]) <= TOL
    # from nothing, token by token
    states = [b.state(3, x) for b in m.blocks]
    for t in range(6):
        assert rel(m.step(x[:, t].contiguous(), states), whole[:, t]) <= TOL


def test_gradients(example):
    m = make(example)
    gen = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(2, 19, 48, device="cuda", generator=gen)
    h, _, saved = m.prompt(x)
    dh = torch.randn(h.shape, device="cuda", generator=gen)
    dx, grads = m.backward(saved, dh)

    def leaf(t):
        return t.detach().double().cpu().requires_grad_()

    F = torch.nn.functional
    x64 = leaf(x)
    ws = [{n: leaf(getattr(b, n)) for n in b.NAMES} for b in m.blocks]
    r = x64
    for b, w in zip(m.blocks, ws):
        hh = F.layer_norm(r, (48,), w["norm"], w["norm_bias"], 1e-5)
        p, z = (hh @ w["w_in"].t()).split(b.E, -1)
        u = F.silu(F.conv1d(F.pad(p.transpose(1, 2), (b.W - 1, 0)), w["conv"][:, None], w["conv_bias"], groups=b.E)).transpose(1, 2)
        low, bb, cc = (u @ w["w_x"].t()).split(b.parts, -1)
        delta = F.softplus(low @ w["w_dt"].t() + w["dt_bias"])
        bb, cc = (t.unflatten(-1, (b.G, b.N)).repeat_interleave(b.E // b.G, 2) for t in (bb, cc))
        s, ys = torch.zeros(2, b.E, b.N, dtype=torch.float64), []
        for t in range(x.shape[1]):
            s = torch.exp(delta[:, t, :, None] * w["a"]) * s + (delta[:, t] * u[:, t])[..., None] * bb[:, t]
            ys.append((s * cc[:, t]).sum(-1) + w["skip"] * u[:, t])
        r = r + (torch.stack(ys, 1) * F.silu(z)) @ w["w_out"].t()
    assert rel(h, r.detach()) <= TOL
    (r * dh.double().cpu()).sum().backward()
    assert rel(dx, x64.grad) <= TOL
    for g, w in zip(grads, ws):
        assert set(g) == set(w)
        for n in w:
            assert rel(g[n], w[n].grad) <= TOL, n


def test_bf16_stack_runs_in_a_graph(example):
    m = make(example, torch.bfloat16, groups=1)
    x = torch.randn(2, 130, 48, device="cuda", dtype=torch.bfloat16)
    h, states, saved = m.prompt(x)
    dx, grads = m.backward(saved, torch.randn_like(h))
    assert torch.isfinite(h.float()).all() and torch.isfinite(dx.float()).all()
    t = x[:, 0].contiguous()
    keep = [tuple(s.clone() for s in st) for st in states]
    want_states = [tuple(s.clone() for s in st) for st in states]
    want = m.step(t, want_states)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.step(t, states)
    for st, k in zip(states, keep):
        for s, v in zip(st, k):
            s.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for st, ws in zip(states, want_states):
        for s, w in zip(st, ws):
            assert torch.equal(s, w)
