"""First-order linear attention on the GPU against the float64 oracle.

Tolerances.  A rounding to bf16 is off by at most 2^-8 / 2 ulp-wise, 2^-8 relative to the value as a
half step of eps; a uniform rounding error has an rms of its half step over sqrt(3).  A bf16 output passes
through three such roundings of about its own size (the decayed score matrix, the carried state, the
output; the other operands keep 16 bits or more), so the relative Frobenius error is at most
sqrt(3) 2^-8 / sqrt(3) = 2^-8.  Each element is off by at most 2^-8 (|o| + 2 m), with m the same sums over
absolute values, which bound both products.  Float32 values are sums of up to n d products in
some order, each rounded to 2^-24: 2^-24 (16 + 2 sqrt(n d)) in norm, the 16 for the decays (exp2 and
log2 of float32 are good to a few units).
"""
import math

import numpy as np
import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from oracle import mixer_oracle as O

from .helpers import np64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def draw(B, H, Hk, n, d, dv, dtype, seed=0, tokens_first=False, ragged=False, state=False, gamma=(0.9, 0.9995)):
    g = torch.Generator().manual_seed(seed)

    def t(heads, dim, by=1.0):
        if tokens_first:
            return (torch.randn((B, n, heads, dim), generator=g) * by).to(dtype).transpose(1, 2)
        return (torch.randn((B, heads, n, dim), generator=g) * by).to(dtype)

    x = {"q": t(H, d), "k": t(Hk, d, 1 / math.sqrt(d)), "v": t(Hk, dv), "dout": t(H, dv)}
    x["gamma"] = None if gamma is None else torch.linspace(gamma[0], gamma[1], Hk)
    x["lengths"] = torch.randint(0, n + 1, (B,), generator=g, dtype=torch.int32) if ragged else None
    if ragged and B > 2:
        x["lengths"][1], x["lengths"][2] = 0, n
    x["init"] = torch.randn((B, Hk, d, dv), generator=g) if state else None
    x["dfinal"] = torch.randn((B, Hk, d, dv), generator=g) if state else None
    return x


def cuda(x):
    # .to keeps the strides of dense tensors
    return {k: None if t is None else t.cuda() for k, t in x.items()}


def n64(t):
    return None if t is None else np64(t)


def f32_tol(n, d):
    return 2.0 ** -24 * (16 + 2 * math.sqrt(n * d))


def check(got, want, bound, dtype, n, d, what):
    """Frobenius error, and for bf16 every element against the sums of absolute values ``bound``."""
    got = np64(got)
    assert got.shape == want.shape, what
    norm = np.linalg.norm(want)
    err = np.linalg.norm(got - want)
    assert np.isfinite(got).all(), what
    tol = (2.0 ** -8 if dtype == BF else 0.0) + f32_tol(n, d)
    assert err <= tol * max(norm, 1e-30) or norm == err == 0, (what, err / max(norm, 1e-30), tol)
    if dtype == BF and bound is not None:
        lim = 2.0 ** -8 * (np.abs(want) + 2 * bound) + 2.0 ** -20 * bound + 1e-30
        assert (np.abs(got - want) <= lim).all(), (what, float((np.abs(got - want) / lim).max()))


def absolute(x):
    return {k: None if v is None else (v if k in ("gamma", "lengths") else np.abs(v)) for k, v in x.items()}


def run_all(x, scale, dtype, train=True):
    B, H, n, d = x["q"].shape
    dv = x["v"].shape[-1]
    c = cuda(x)
    o64 = {k: (n64(t) if k != "lengths" else None if t is None else t.numpy()) for k, t in x.items()}
    a64 = absolute(o64)
    args = lambda z: (z["q"], z["k"], z["v"])  # noqa: E731
    o, fin = hla.linattn_forward(c["q"], c["k"], c["v"], gamma=c["gamma"], scale=scale, lengths=c["lengths"],
                                 init_state=c["init"], return_final_state=True)
    hla.check_status()
    wo, wP = O.linattn_forward(*args(o64), o64["gamma"], scale, o64["lengths"], o64["init"])
    bo, _ = O.linattn_forward(*args(a64), a64["gamma"], abs(scale), a64["lengths"], a64["init"])
    check(o, wo, bo, dtype, n, max(d, dv), "out")
    check(fin, wP, None, F32, n, 1, "final state")
    # without the state
    o2 = hla.linattn_forward(c["q"], c["k"], c["v"], gamma=c["gamma"], scale=scale, lengths=c["lengths"],
                             init_state=c["init"])
    check(o2, wo, bo, dtype, n, max(d, dv), "out alone")
    if not train:
        return
    got = hla.linattn_backward(c["q"], c["k"], c["v"], c["dout"], gamma=c["gamma"], scale=scale, lengths=c["lengths"],
                               init_state=c["init"], dfinal_state=c["dfinal"])
    hla.check_status()
    want = O.linattn_backward(*args(o64), o64["dout"], o64["gamma"], scale, o64["lengths"], o64["init"], o64["dfinal"])
    bound = O.linattn_backward(*args(a64), a64["dout"], a64["gamma"], abs(scale), a64["lengths"], a64["init"],
                               a64["dfinal"])
    for name, g, w, b in zip(("dq", "dk", "dv"), got, want, bound):
        check(g, w, b, dtype, n * (H // x["k"].shape[1]), max(d, dv), name)
    if x["init"] is not None:
        check(got[3], want[3], None, F32, n * (H // x["k"].shape[1]), 1, "dinit")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 127, 128, 129, 255, 300, 700])
def test_lengths_of_the_sequence(dtype, n):
    run_all(draw(1, 2, 2, n, 64, 64, dtype, seed=n), 0.125, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d, dv", [(16, 16), (32, 32), (64, 64), (128, 128), (16, 128), (128, 16), (32, 64), (64, 128)])
@pytest.mark.parametrize("tokens_first", [False, True])
def test_dimensions_with_states_and_shared_heads(dtype, d, dv, tokens_first):
    run_all(draw(3, 6, 2, 290, d, dv, dtype, seed=d + dv, tokens_first=tokens_first, ragged=True, state=True), 0.3, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gamma", [None, (1.0, 1.0), (0.02, 0.5), (0.5, 0.999)])
def test_decays(dtype, gamma):
    run_all(draw(2, 3, 3, 400, 64, 64, dtype, seed=7, state=True, gamma=gamma), 1.0, dtype)


@pytest.mark.parametrize("dtype, d", [(BF, 64), (BF, 128), (F32, 64)])
def test_long_sequence_in_many_segments(dtype, d):
    run_all(draw(1, 2, 1, 5000, d, d, dtype, seed=3, state=True, gamma=(0.999, 0.999)), 0.125, dtype)


@pytest.mark.parametrize("dtype, d", [(BF, 64), (BF, 128), (F32, 32)])
def test_many_heads_in_one_segment_each(dtype, d):
    run_all(draw(4, 160, 160, 140, d, d, dtype, seed=5), 0.125, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padding_may_hold_anything(dtype):
    x = draw(3, 4, 2, 300, 64, 64, dtype, seed=11, state=True)
    x["lengths"] = torch.tensor([130, 0, 257], dtype=torch.int32)
    c = cuda(x)

    def calls(c):
        o, f = hla.linattn_forward(c["q"], c["k"], c["v"], gamma=c["gamma"], lengths=c["lengths"], init_state=c["init"],
                                   return_final_state=True)
        return (o, f, *hla.linattn_backward(c["q"], c["k"], c["v"], c["dout"], gamma=c["gamma"], lengths=c["lengths"],
                                            init_state=c["init"], dfinal_state=c["dfinal"]))

    clean = [t.clone() for t in calls(c)]
    for name, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("dout", float("-inf"))):
        for b, L in enumerate(x["lengths"].tolist()):
            c[name][b, :, L:] = bad
    for a, b in zip(clean, calls(c)):
        assert torch.equal(a, b)
    for b, L in enumerate(x["lengths"].tolist()):
        assert not clean[0][b, :, L:].any()
    assert torch.equal(clean[1][1], c["init"][1])


def test_lengths_outside_the_sequence_are_clamped():
    x = cuda(draw(2, 2, 2, 200, 64, 64, BF, seed=12))
    kw = dict(gamma=x["gamma"], return_final_state=True)
    a = hla.linattn_forward(x["q"], x["k"], x["v"], lengths=torch.tensor([-5, 900], device="cuda"), **kw)
    b = hla.linattn_forward(x["q"], x["k"], x["v"], lengths=torch.tensor([0, 200], device="cuda"), **kw)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_lengths_past_32_bits_are_clamped_too():
    x = cuda(draw(2, 2, 2, 200, 64, 64, BF, seed=12))
    kw = dict(gamma=x["gamma"], return_final_state=True)
    want = hla.linattn_forward(x["q"], x["k"], x["v"], lengths=torch.tensor([200, 0], device="cuda"), **kw)
    far = [2 ** 32 + 5, -2 ** 32 + 7]
    for lengths in (far, torch.tensor(far), torch.tensor(far, device="cuda")):
        got = hla.linattn_forward(x["q"], x["k"], x["v"], lengths=lengths, **kw)
        assert all(torch.equal(s, t) for s, t in zip(got, want))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_views_are_read_in_place_and_others_copied(dtype):
    g = torch.Generator().manual_seed(21)
    fused = torch.randn((2, 150, 3, 4, 64), generator=g).to(dtype).cuda()  # [B, n, qkv, H, d]
    q, k, v = (fused[:, :, i].transpose(1, 2) for i in range(3))
    want = hla.linattn_forward(q.contiguous(), k.contiguous(), v.contiguous(), gamma=0.97)
    got = hla.linattn_forward(q, k, v, gamma=0.97)
    assert torch.equal(got, want) and got.stride(1) < got.stride(2)
    out = torch.empty((2, 150, 4, 64), dtype=dtype, device="cuda").transpose(1, 2)
    assert hla.linattn_forward(q, k, v, gamma=0.97, out=out) is out and torch.equal(out, want)
    wide = torch.randn((2, 4, 150, 70), generator=g).to(dtype).cuda()
    odd = wide[..., 3:67]  # rows at odd addresses
    assert torch.equal(hla.linattn_forward(odd, k, v, gamma=0.97),
                       hla.linattn_forward(odd.contiguous(), k, v, gamma=0.97))
    one = k[:, :1].expand(2, 4, 150, 64)  # broadcast over heads
    assert torch.equal(hla.linattn_forward(q, one, v, gamma=0.97),
                       hla.linattn_forward(q, one.contiguous(), v, gamma=0.97))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_states_at_odd_addresses_are_copied(dtype):
    x = cuda(draw(2, 4, 2, 200, 32, 64, dtype, seed=22, state=True))
    odd = {k: torch.zeros(x[k].numel() + 1, device="cuda")[1:].view(x[k].shape).copy_(x[k]) for k in ("init", "dfinal")}

    def calls(init, dfinal):
        return (*hla.linattn_forward(x["q"], x["k"], x["v"], gamma=x["gamma"], init_state=init, return_final_state=True),
                *hla.linattn_backward(x["q"], x["k"], x["v"], x["dout"], gamma=x["gamma"], init_state=init,
                                      dfinal_state=dfinal))

    for a, b in zip(calls(x["init"], x["dfinal"]), calls(odd["init"], odd["dfinal"])):
        assert torch.equal(a, b)
    swapped = {k: x[k].transpose(0, 1).contiguous().transpose(0, 1) for k in odd}
    for a, b in zip(calls(x["init"], x["dfinal"]), calls(swapped["init"], swapped["dfinal"])):
        assert torch.equal(a, b)


def test_same_bits_on_every_call_and_on_a_side_stream():
    x = cuda(draw(2, 8, 2, 1500, 64, 64, BF, seed=30, state=True))

    def calls():
        return [*hla.linattn_forward(x["q"], x["k"], x["v"], gamma=x["gamma"], init_state=x["init"],
                                     return_final_state=True),
                *hla.linattn_backward(x["q"], x["k"], x["v"], x["dout"], gamma=x["gamma"], init_state=x["init"])]

    first = calls()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = calls()
    third = calls()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_graph_capture_replays_on_new_inputs():
    x = cuda(draw(1, 4, 4, 700, 64, 64, BF, seed=31))
    run = lambda: (hla.linattn_forward(x["q"], x["k"], x["v"], gamma=x["gamma"]),  # noqa: E731
                   *hla.linattn_backward(x["q"], x["k"], x["v"], x["dout"], gamma=x["gamma"]))
    eager = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    x["v"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], -eager[0])          # linear in v
    assert torch.equal(held[1], -eager[1])          # dq too
    assert torch.equal(held[3], eager[3])           # dv does not depend on v
    again = run()
    for a, b in zip(held, again):
        assert torch.equal(a, b)


def test_empty_calls():
    z = lambda *s: torch.zeros(s, dtype=BF, device="cuda")  # noqa: E731
    init = torch.randn((2, 3, 16, 32), device="cuda")
    o, f = hla.linattn_forward(z(2, 3, 0, 16), z(2, 3, 0, 16), z(2, 3, 0, 32), gamma=0.9, init_state=init,
                               return_final_state=True)
    assert o.shape == (2, 3, 0, 32) and torch.equal(f, init)
    o, f = hla.linattn_forward(z(2, 3, 0, 16), z(2, 3, 0, 16), z(2, 3, 0, 32), return_final_state=True)
    assert not f.any()
    dfin = torch.randn((2, 3, 16, 32), device="cuda")
    *_, di = hla.linattn_backward(z(2, 3, 0, 16), z(2, 3, 0, 16), z(2, 3, 0, 32), z(2, 3, 0, 32), init_state=init,
                                  dfinal_state=dfin)
    assert torch.equal(di, dfin)
    assert hla.linattn_forward(z(0, 3, 5, 16), z(0, 3, 5, 16), z(0, 3, 5, 32)).shape == (0, 3, 5, 32)


def test_gradients_are_differences_of_the_forward():
    x = draw(1, 2, 1, 70, 16, 32, F32, seed=40, state=True)
    c = cuda(x)
    grads = hla.linattn_backward(c["q"], c["k"], c["v"], c["dout"], gamma=c["gamma"], scale=0.5, init_state=c["init"],
                                 dfinal_state=c["dfinal"])

    def loss(z):
        o, f = hla.linattn_forward(z["q"], z["k"], z["v"], gamma=z["gamma"], scale=0.5, init_state=z["init"],
                                   return_final_state=True)
        return (o.double() * z["dout"].double()).sum() + (f.double() * z["dfinal"].double()).sum()

    gen = torch.Generator().manual_seed(41)
    for name, g in zip(("q", "k", "v", "init"), grads):
        u = torch.randn(x[name].shape, generator=gen).cuda()
        h = 2.0 ** -6  # the loss is linear in each input, so a large step costs nothing
        up, down = dict(c), dict(c)
        up[name], down[name] = c[name] + h * u, c[name] - h * u
        diff = float((loss(up) - loss(down)) / (2 * h))
        want = float((g.double() * u.double()).sum())
        assert abs(diff - want) <= 1e-3 * float(g.double().norm() * u.double().norm()), name


# ---- single tokens ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N, H, Hk, d, dv", [(1, 1, 1, 16, 16), (3, 6, 2, 64, 64), (2, 4, 4, 128, 128), (5, 8, 1, 32, 128),
                                             (2, 3, 3, 128, 16), (1, 16, 4, 64, 32), (2, 10, 5, 16, 64)])
def test_step(dtype, N, H, Hk, d, dv):
    x = draw(N, H, Hk, 1, d, dv, dtype, seed=N + H, state=True)
    q, k, v = (x[i][:, :, 0] for i in ("q", "k", "v"))
    P = x["init"].cuda()
    for turn in range(2):
        want, wP = O.linattn_step(np64(P.cpu()), np64(q), np64(k), np64(v), np64(x["gamma"]), 0.4)
        o = hla.linattn_decode_step(P, q.cuda(), k.cuda(), v.cuda(), gamma=x["gamma"].cuda(), scale=0.4)
        assert np.linalg.norm(np64(P.cpu()) - wP) <= 2.0 ** -23 * np.linalg.norm(wP)
        tol = f32_tol(1, d) + (2.0 ** -8 if dtype == BF else 0)
        assert np.linalg.norm(np64(o.cpu()) - want) <= tol * np.linalg.norm(want)


@pytest.mark.parametrize("dtype, d", [(BF, 64), (F32, 64), (BF, 128)])
def test_prompt_then_steps(dtype, d):
    x = draw(2, 4, 2, 210, d, d, dtype, seed=50)
    c = cuda(x)
    whole = hla.linattn_forward(c["q"], c["k"], c["v"], gamma=c["gamma"], scale=0.2)
    cut = 203
    _, P = hla.linattn_forward(*(c[i][:, :, :cut] for i in ("q", "k", "v")), gamma=c["gamma"], scale=0.2,
                               return_final_state=True)
    want, _ = O.linattn_forward(np64(x["q"]), np64(x["k"]), np64(x["v"]), np64(x["gamma"]), 0.2)
    for t in range(cut, 210):
        o = hla.linattn_decode_step(P, *(c[i][:, :, t] for i in ("q", "k", "v")), gamma=c["gamma"], scale=0.2)
        for got in (o, whole[:, :, t]):
            e = np.linalg.norm(np64(got.cpu()) - want[:, :, t])
            assert e <= ((2.0 ** -8 if dtype == BF else 0) + f32_tol(210, d)) * np.linalg.norm(want[:, :, t])


def test_bindings_refuse():
    q = torch.zeros((1, 4, 8, 16), dtype=BF, device="cuda")
    k = torch.zeros((1, 3, 8, 16), dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        hla.linattn_forward(q, k, k)                       # 4 heads on 3
    with pytest.raises(TypeError):
        hla.linattn_forward(q, q.float(), q)
    with pytest.raises(ValueError):
        hla.linattn_forward(q, q, q, lengths=[1, 2])
    with pytest.raises(ValueError):
        hla.linattn_forward(q, q, q, init_state=torch.zeros((1, 4, 16, 17), device="cuda"))
    with pytest.raises(ValueError):
        hla.linattn_forward(q, q, q, out=torch.zeros((1, 4, 8, 32), dtype=BF, device="cuda"))
    with pytest.raises(hla.HLA2Error):
        hla.linattn_forward(q, q, q, out=q)                # overlaps
    t = torch.zeros((1, 4, 8, 24), dtype=BF, device="cuda")
    with pytest.raises(hla.HLA2Error):
        hla.linattn_forward(t, t, t)                       # d = 24
    with pytest.raises(ValueError):
        hla.linattn_decode_step(torch.zeros((1, 4, 16, 32), device="cuda"), q[:, :, 0], q[:, :, 0], q[:, :, 0])
