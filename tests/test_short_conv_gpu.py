"""The short causal convolution on the GPU against the float64 oracle.

Tolerances: sums of W + 1 products in float32, an approximate SiLU (a few 2^-22) and, in the backward, W more
products, so 2^-18 of the sums over absolute values, of which 1e-5 of the largest output is more than enough; sums over
up to 4000 tokens by 2^-24 a term and partial sums of at most 64: 1e-5 as well.  A bfloat16 output is rounded once."""
import numpy as np
import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from oracle import ssm_oracle as O

from .ssm_cases import BF, F32, close, f64

pytestmark = pytest.mark.gpu


def make(B, n, D, W, dtype, bias=True, state=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    c = dict(x=rand(B, n, D), weight=rand(D, W), bias=rand(D) if bias else None, init_state=rand(B, W - 1, D) if state else None)
    return c, rand(B, n, D), rand(B, W - 1, D) if state else None


def check(c, dout, dfin, lengths=None, act="silu"):
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    kw = dict(bias=f64(c["bias"]), act=act, lengths=lengths, init_state=f64(c["init_state"]))
    out, fin = hla.short_conv_forward(**c, act=act, lengths=lens, return_final_state=True)
    want, wfin = O.conv_forward(f64(c["x"]), f64(c["weight"]), **kw)
    close(out, want, "out", 1e-5)
    assert np.array_equal(f64(fin), wfin)  # inputs, as they are
    g = hla.short_conv_backward(dout=dout, dfinal_state=dfin, act=act, lengths=lens, **c)
    w = O.conv_backward(f64(c["x"]), f64(c["weight"]), f64(dout), dfinal_state=f64(dfin), **kw)
    for name in g._fields:
        source = {"dbias": "bias", "dinit_state": "init_state"}.get(name)
        if source and c[source] is None:
            assert getattr(g, name) is None
        else:
            close(getattr(g, name), w[name], name, 1e-5)
    for s, m in enumerate(lengths or []):
        assert (out[s, max(m, 0):] == 0).all() and (g.dx[s, max(m, 0):] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("n, D", [(1, 8), (2, 24), (3, 1), (9, 131), (100, 64), (67, 257), (200, 40)])
def test_sizes(dtype, W, n, D):
    check(*make(2, n, D, W, dtype, seed=n + W))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("act", ["silu", "none", None])
@pytest.mark.parametrize("bias, state", [(False, False), (True, False), (False, True)])
def test_optional_inputs(dtype, act, bias, state):
    check(*make(2, 30, 48, 4, dtype, bias, state), act=act)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("lengths", [[0, 50, 1], [2, -4, 33], [60, 3, 0]])
def test_lengths(dtype, W, lengths):
    c, dout, dfin = make(3, 50, 32, W, dtype)
    for s, m in enumerate(lengths):  # padding holds anything
        c["x"][s, max(m, 0):] = float("nan") if s % 2 else float("inf")
        dout[s, max(m, 0):] = float("inf") if s % 2 else float("nan")
    check(c, dout, dfin, lengths)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_long(dtype):
    check(*make(3, 4001, 72, 4, dtype), lengths=[4001, 1234, 8])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides(dtype):
    c, dout, dfin = make(2, 40, 32, 4, dtype)
    want = (*hla.short_conv_forward(**c, return_final_state=True), *hla.short_conv_backward(dout=dout, dfinal_state=dfin, **c))
    for off in (0, 1, 8):  # a part of a projection, at odd places too
        wide = torch.empty(2, 40, 100, dtype=dtype, device="cuda")
        first = torch.empty(40, 2, 33, dtype=dtype, device="cuda").transpose(0, 1)  # tokens before sequences
        x, do = wide[..., off:off + 32], first[..., 1:]
        x.copy_(c["x"])
        do.copy_(dout)
        v = {**c, "x": x}
        got = (*hla.short_conv_forward(**v, return_final_state=True), *hla.short_conv_backward(dout=do, dfinal_state=dfin, **v))
        for u, w in zip(got, want):
            if u.dtype == F32:  # another vector width adds the tokens of the sums in another order
                assert torch.allclose(u, w, rtol=1e-5, atol=1e-4)
            else:
                assert torch.equal(u, w)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B, D", [(1, 64), (5, 33), (300, 128)])
def test_step_follows_the_forward(dtype, W, B, D):
    c, _, _ = make(B, 6, D, W, dtype, seed=B)
    want, fin = hla.short_conv_forward(**c, return_final_state=True)
    state = c["init_state"].clone()
    for t in range(6):
        out = hla.short_conv_decode_step(state, c["x"][:, t], c["weight"], bias=c["bias"])
        assert torch.equal(out, want[:, t])
    assert torch.equal(state, fin)


def test_empty():
    c, dout, dfin = make(2, 0, 16, 4, F32)
    out, fin = hla.short_conv_forward(**c, return_final_state=True)
    assert out.shape == (2, 0, 16) and torch.equal(fin, c["init_state"])
    g = hla.short_conv_backward(dout=dout, dfinal_state=dfin, **c)
    assert torch.equal(g.dinit_state, dfin) and not g.dweight.any() and not g.dbias.any()
    assert not hla.short_conv_backward(dout=dout, **c).dinit_state.any()
    c, dout, _ = make(0, 5, 16, 4, F32)
    assert hla.short_conv_forward(**c).shape == (0, 5, 16)
    assert not hla.short_conv_backward(dout=dout, **c).dweight.any()


def test_captured():
    c, dout, dfin = make(2, 300, 64, 4, BF)
    d, _, _ = make(2, 300, 64, 4, BF, seed=9)
    static = {k: v.clone() for k, v in c.items()}
    hla.short_conv_backward(dout=dout, **static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hla.short_conv_forward(**static)
        grads = hla.short_conv_backward(dout=dout, dfinal_state=dfin, **static)
    for case in (d, c):
        for k, v in static.items():
            v.copy_(case[k])
        graph.replay()
        want = (hla.short_conv_forward(**case), *hla.short_conv_backward(dout=dout, dfinal_state=dfin, **case))
        graph.replay()
        for u, w in zip((out, *grads), want):
            assert torch.equal(u, w)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_short_sequences(dtype):
    """More sequences than a grid has rows, and so several to a CTA."""
    c, dout, dfin = make(70_000, 1, 8, 4, dtype)
    g = hla.short_conv_backward(dout=dout, dfinal_state=dfin, **c)
    out, fin = hla.short_conv_forward(**c, return_final_state=True)
    kw = dict(bias=f64(c["bias"]), init_state=f64(c["init_state"]))
    want, wfin = O.conv_forward(f64(c["x"]), f64(c["weight"]), **kw)
    close(out, want, "out", 1e-5)
    assert np.array_equal(f64(fin), wfin)
    w = O.conv_backward(f64(c["x"]), f64(c["weight"]), f64(dout), dfinal_state=f64(dfin), **kw)
    for name in g._fields:  # 70000 terms in 152 * 8 partial sums and more: within the bound of 4000
        close(getattr(g, name), w[name], name, 1e-5)
    state = c["init_state"].clone()
    assert torch.equal(hla.short_conv_decode_step(state, c["x"][:, 0], c["weight"], bias=c["bias"]), out[:, 0])
    assert torch.equal(state, fin)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D", [12, 132])
def test_rows_of_four_channels_alignment(dtype, W, D):
    """Widths and addresses that are multiples of four elements, not of eight."""
    c, dout, dfin = make(2, 45, D, W, dtype, seed=D)
    wide = torch.zeros((2, 45, 2 * D + 4), dtype=dtype, device="cuda")
    wide[..., 4:4 + D] = c["x"]
    check({**c, "x": wide[..., 4:4 + D]}, dout, dfin, lengths=[45, 7])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D", [47, 48])
@pytest.mark.parametrize("m", [3, 16, 17, 40])
def test_an_infinite_input_reaches_its_own_terms_only(dtype, W, D, m):
    """dweight_j = sum_t dout_t x_{t - W + 1 + j}: an input among a sequence's last W - 1 tokens is in fewer than W taps' sums, as
    the tokens after it are padding."""
    c, dout, _ = make(2, 40, D, W, dtype, state=False)
    bad = m - 1  # the last valid token: a term of the last tap alone
    c["x"][1, bad, 5] = float("inf")
    lens = torch.tensor([40, m], dtype=torch.int32, device="cuda")
    g = hla.short_conv_backward(dout=dout, act="none", lengths=lens, **c)
    want = O.conv_backward(f64(c["x"]), f64(c["weight"]), f64(dout), bias=f64(c["bias"]), act="none", lengths=[40, m])
    got = f64(g.dweight)
    assert np.isinf(want["dweight"]).sum() == 1 and np.isinf(want["dweight"][5, W - 1])
    assert got[5, W - 1] == want["dweight"][5, W - 1]
    g.dweight[5, W - 1] = want["dweight"][5, W - 1] = 0.0
    close(g.dweight, want["dweight"], "dweight", 1e-5)
    close(g.dx, want["dx"], "dx", 1e-5)
    close(g.dbias, want["dbias"], "dbias", 1e-5)
