"""The oracle of a selective state space layer's operators: forms that are known, and gradients against differences."""
import numpy as np
import pytest

from oracle import ssm_oracle as O

rng = np.random.default_rng(0)


def ssm_case(B=2, n=5, D=4, N=3, G=2, **kw):
    c = dict(x=rng.normal(size=(B, n, D)), dt=rng.normal(size=(B, n, D)), a=-np.exp(rng.normal(size=(D, N))),
             b=rng.normal(size=(B, n, G, N)), c=rng.normal(size=(B, n, G, N)), skip=rng.normal(size=D),
             gate=rng.normal(size=(B, n, D)), dt_bias=rng.normal(size=D), lengths=[n, 3], init_state=rng.normal(size=(B, D, N)))
    c.update(kw)
    return c


def test_scan_is_its_closed_sum():
    c = ssm_case(lengths=None, skip=None, gate=None, dt_bias=None)
    out, fin = O.ssm_forward(**c)
    delta = np.log1p(np.exp(c["dt"]))
    S = np.cumsum(delta, 1)
    B, n, D = c["x"].shape
    b, cc = np.repeat(c["b"], 2, 2), np.repeat(c["c"], 2, 2)
    for t in range(n):
        h = np.exp(S[:, t, :, None] * c["a"]) * c["init_state"]
        for i in range(t + 1):
            h = h + np.exp((S[:, t] - S[:, i])[..., None] * c["a"]) * (delta[:, i] * c["x"][:, i])[..., None] * b[:, i]
        assert np.allclose(out[:, t], (h * cc[:, t]).sum(-1), rtol=1e-12, atol=1e-12)
    assert np.allclose(fin, h, rtol=1e-12, atol=1e-12)


def test_padding_is_not_read():
    c = ssm_case(lengths=[0, 2])
    full = O.ssm_forward(**c)
    for k in ("x", "dt", "b", "c", "gate"):
        c[k][0] = np.nan
        c[k][1, 2:] = np.inf
    for u, v in zip(full, O.ssm_forward(**c)):
        assert np.array_equal(u, v)
    assert np.array_equal(full[1][0], c["init_state"][0])


def differences(f, v, eps=1e-6):
    g = np.zeros_like(v)
    for i in np.ndindex(*v.shape):
        keep = v[i]
        v[i] = keep + eps
        up = f()
        v[i] = keep - eps
        g[i] = (up - f()) / (2 * eps)
        v[i] = keep
    return g


@pytest.mark.parametrize("kw", [{}, dict(gate=None, dt_softplus=False), dict(skip=None, dt_bias=None, lengths=None)])
def test_scan_gradients(kw):
    c = ssm_case(**kw)
    B, n, D = c["x"].shape
    dout, dfin = rng.normal(size=(B, n, D)), rng.normal(size=c["init_state"].shape)

    def loss():
        out, fin = O.ssm_forward(**c)
        return (out * dout).sum() + (fin * dfin).sum()

    g = O.ssm_backward(dout=dout, dfinal_state=dfin, **c)
    # Without a softplus steps may be negative and the states grow: a loss is the sum of some hundred terms, each of some ten
    # operations, so it is off by up to 2^-53 * 16 of their absolute sum, and a difference by that over the step.
    out, fin = O.ssm_forward(**c)
    atol = 1e-7 + 16 * 2.0 ** -53 * (np.abs(out * dout).sum() + np.abs(fin * dfin).sum()) / 1e-6
    for name in ("x", "dt", "a", "b", "c", "skip", "gate", "dt_bias", "init_state"):
        if c.get(name) is not None:
            assert np.allclose(g["d" + name], differences(loss, c[name]), rtol=1e-6, atol=atol), name


@pytest.mark.parametrize("act", ["silu", None])
@pytest.mark.parametrize("W", [2, 4])
def test_convolution_gradients(act, W):
    B, n, D = 2, 5, 3
    x, w, bias, st = (rng.normal(size=s) for s in ((B, n, D), (D, W), (D,), (B, W - 1, D)))
    dout, dfin = rng.normal(size=x.shape), rng.normal(size=st.shape)
    kw = dict(bias=bias, act=act, lengths=[n, 1], init_state=st)

    def loss():
        out, fin = O.conv_forward(x, w, **kw)
        return (out * dout).sum() + (fin * dfin).sum()

    g = O.conv_backward(x, w, dout, dfinal_state=dfin, **kw)
    for name, v in (("dx", x), ("dweight", w), ("dbias", bias), ("dinit_state", st)):
        assert np.allclose(g[name], differences(loss, v), rtol=1e-6, atol=1e-7), name


def test_convolution_is_a_convolution():
    x, w = rng.normal(size=(1, 7, 1)), rng.normal(size=(1, 3))
    out, fin = O.conv_forward(x, w, act=None)
    assert np.allclose(out[0, :, 0], np.convolve(x[0, :, 0], w[0, ::-1])[:7])
    assert np.array_equal(fin, x[:, 5:])


def test_layer_norm_gradients():
    x, w, b, do = (rng.normal(size=s) for s in ((3, 5), (5,), (5,), (3, 5)))
    y = O.layer_norm(x, np.ones(5), eps=0.0)
    assert np.allclose(y.mean(-1), 0) and np.allclose((y * y).mean(-1), 1)
    loss = lambda: (O.layer_norm(x, w, b) * do).sum()  # noqa: E731
    for got, v in zip(O.layer_norm_backward(x, w, do), (x, w, b)):
        assert np.allclose(got, differences(loss, v), rtol=1e-6, atol=1e-7)
