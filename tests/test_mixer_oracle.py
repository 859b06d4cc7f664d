"""The float64 oracle of the operators around a mixer layer, pinned on the CPU: the recurrence
against the pair sum, the step against the forward, and every gradient against central differences."""
import numpy as np
import pytest

from oracle import mixer_oracle as O


def _inputs(rng, B=2, H=4, Hk=2, n=7, d=3, dv=5):
    q, k, v, do = (rng.standard_normal(s) for s in ((B, H, n, d), (B, Hk, n, d), (B, Hk, n, dv), (B, H, n, dv)))
    return q, k, v, do, np.array([0.9, 0.6])[:Hk], rng.standard_normal((B, Hk, d, dv)), \
        rng.standard_normal((B, Hk, d, dv))


def test_forward_is_the_pair_sum():
    rng = np.random.default_rng(0)
    q, k, v, _, g, P0, _ = _inputs(rng)
    L = [7, 4]
    o, P = O.linattn_forward(q, k, v, g, 0.7, L, P0)
    for b in range(2):
        for h in range(4):
            s = h // 2
            for t in range(7):
                want = np.zeros(5)
                if t < L[b]:
                    want = g[s] ** (t + 1) * q[b, h, t] @ P0[b, s]
                    for i in range(t + 1):
                        want = want + g[s] ** (t - i) * (q[b, h, t] @ k[b, s, i]) * v[b, s, i]
                assert np.allclose(o[b, h, t], 0.7 * want, atol=1e-12)
            want = g[s] ** L[b] * P0[b, s]
            for i in range(L[b]):
                want = want + g[s] ** (L[b] - 1 - i) * np.outer(k[b, s, i], v[b, s, i])
            assert np.allclose(P[b, s], want, atol=1e-12)


def test_steps_are_the_forward():
    rng = np.random.default_rng(1)
    q, k, v, _, g, P, _ = _inputs(rng)
    o, fin = O.linattn_forward(q, k, v, g, 0.7, None, P)
    for t in range(7):
        ot, P = O.linattn_step(P, q[:, :, t], k[:, :, t], v[:, :, t], g, 0.7)
        assert np.allclose(ot, o[:, :, t], atol=1e-12)
    assert np.allclose(P, fin, atol=1e-12)


def _differences(f, arrays, h=1e-5):
    res = []
    for a in arrays:
        d = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = f()
            a[i] = keep - h
            d[i] = (up - f()) / (2 * h)
            a[i] = keep
        res.append(d)
    return res


def test_linattn_gradients_are_differences():
    rng = np.random.default_rng(2)
    q, k, v, do, g, P0, dP = _inputs(rng, B=2, n=4, d=2, dv=3)
    L = [4, 2]

    def loss():
        o, P = O.linattn_forward(q, k, v, g, 0.7, L, P0)
        return (o * do).sum() + (P * dP).sum()

    want = _differences(loss, (q, k, v, P0))
    got = O.linattn_backward(q, k, v, do, g, 0.7, L, P0, dP)
    for a, b in zip(got, want):
        assert np.allclose(a, b, atol=1e-7)


@pytest.mark.parametrize("gate", ["none", "row", "full"])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("scaled, normed", [(True, True), (False, True), (True, False)])
def test_join_gradients_are_differences(gate, act, scaled, normed):
    rng = np.random.default_rng(3)
    D = 5
    x, y, dr, dh = (rng.standard_normal((3, D)) for _ in range(4))
    pw, s, nw = (rng.standard_normal(D) for _ in range(3))
    z = {"none": None, "row": rng.standard_normal((3, 1)), "full": rng.standard_normal((3, D))}[gate]
    s, nw = s if scaled else None, nw if normed else None

    def loss():
        r, h = O.block_join(x, y, pw, z, act, s, nw, 1e-3)
        return (r * dr).sum() + (0.0 if h is None else (h * dh).sum())

    g = O.block_join_backward(x, y, pw, z, act, s, nw, dr, dh if normed else None, 1e-3)
    for name, a in (("dx", x), ("dy", y), ("dgate", z), ("dpost_weight", pw), ("dscale", s), ("dnext_weight", nw)):
        if a is None:
            assert g[name] is None
        else:
            assert np.allclose(g[name], _differences(loss, (a,))[0], atol=1e-7), name


def test_norm_gradients_are_differences():
    rng = np.random.default_rng(4)
    x, dh, w = rng.standard_normal((3, 5)), rng.standard_normal((3, 5)), rng.standard_normal(5)
    dx, dw = O.block_norm_backward(x, w, dh, 1e-3)
    want = _differences(lambda: (O.block_norm(x, w, 1e-3) * dh).sum(), (x, w))
    assert np.allclose(dx, want[0], atol=1e-7) and np.allclose(dw, want[1], atol=1e-7)


def test_w4_is_its_sum():
    rng = np.random.default_rng(5)
    N, K, g = 3, 64, 32
    vals, z = rng.integers(0, 16, (N, K)), rng.integers(0, 16, (N, K // g))
    packed = (vals[:, 0::2] + 16 * vals[:, 1::2]).astype(np.uint8)
    s, x, b = rng.standard_normal((N, K // g)), rng.standard_normal((2, K)), rng.standard_normal(N)
    y = O.w4_matvec(x, packed, s, z, b)
    for m in range(2):
        for n in range(N):
            want = b[n] + sum(x[m, k] * (vals[n, k] - z[n, k // g]) * s[n, k // g] for k in range(K))
            assert abs(y[m, n] - want) < 1e-10
