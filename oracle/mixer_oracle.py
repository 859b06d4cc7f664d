"""Float64 oracle of the operators around a mixer layer (numpy, from the definitions, token by
token): first-order linear attention with a decay for each key head, the block norms with gate and
residual scale, and products with 4-bit weights.  It shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def _lengths(lengths, B, n):
    return np.full(B, n) if lengths is None else np.clip(np.asarray(lengths, dtype=np.int64), 0, n)


def _gamma(gamma, Hk):
    return np.ones(Hk) if gamma is None else np.broadcast_to(np.asarray(gamma, dtype=np.float64), (Hk,))


def linattn_forward(q, k, v, gamma=None, scale=1.0, lengths=None, init=None):
    """(out [B,H,n,dv], state [B,Hk,d,dv]):  P <- g P + k v^T,  out = scale q P, query head h on key
    head h // (H // Hk), sequence b up to lengths[b] tokens."""
    B, H, n, d = q.shape
    Hk, dv = k.shape[1], v.shape[-1]
    rep = H // Hk
    g = _gamma(gamma, Hk)[:, None, None]
    L = _lengths(lengths, B, n)
    P = np.zeros((B, Hk, d, dv)) if init is None else np.array(init, dtype=np.float64)
    out = np.zeros((B, H, n, dv))
    for b in range(B):
        for t in range(L[b]):
            P[b] = g * P[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            out[b, :, t] = scale * np.einsum("hd,hde->he", q[b, :, t], np.repeat(P[b], rep, axis=0))
    return out, P


def linattn_backward(q, k, v, dout, gamma=None, scale=1.0, lengths=None, init=None, dfinal=None):
    """(dq, dk, dv, dinit) by the adjoint of the recurrence, tokens in reverse."""
    B, H, n, d = q.shape
    Hk, dv = k.shape[1], v.shape[-1]
    rep = H // Hk
    g = _gamma(gamma, Hk)[:, None, None]
    L = _lengths(lengths, B, n)
    P0 = np.zeros((B, Hk, d, dv)) if init is None else np.asarray(init, dtype=np.float64)
    dq, dk, dvv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dinit = np.zeros((B, Hk, d, dv)) if dfinal is None else np.array(dfinal, dtype=np.float64)
    for b in range(B):
        P = P0[b].copy()
        for t in range(L[b]):
            P = g * P + k[b, :, t, :, None] * v[b, :, t, None, :]
            dq[b, :, t] = scale * np.einsum("he,hde->hd", dout[b, :, t], np.repeat(P, rep, axis=0))
        R = dinit[b]
        for t in range(L[b] - 1, -1, -1):
            qd = scale * q[b, :, t, :, None] * dout[b, :, t, None, :]
            R = R + qd.reshape(Hk, rep, d, dv).sum(1)
            dk[b, :, t] = np.einsum("hde,he->hd", R, v[b, :, t])
            dvv[b, :, t] = np.einsum("hde,hd->he", R, k[b, :, t])
            R = g * R
        dinit[b] = R
    return dq, dk, dvv, dinit


def linattn_step(state, q, k, v, gamma=None, scale=1.0):
    """(out [N,H,dv], new state [N,Hk,d,dv])"""
    o, P = linattn_forward(q[:, :, None], k[:, :, None], v[:, :, None], gamma, scale, None, state)
    return o[:, :, 0], P


def _norm(t, eps):
    inv = 1.0 / np.sqrt((t * t).mean(-1, keepdims=True) + eps)
    return t * inv, inv


def _norm_adjoint(dn, nt, inv):
    return inv * (dn - nt * (dn * nt).mean(-1, keepdims=True))


def _act(z, act):
    s = 1.0 / (1.0 + np.exp(-z))
    return (s, s * (1.0 - s)) if act == "sigmoid" else (z * s, s * (1.0 + z * (1.0 - s)))


def block_norm(x, w, eps):
    return _norm(x, eps)[0] * w


def block_norm_backward(x, w, dout, eps):
    nx, inv = _norm(x, eps)
    return _norm_adjoint(dout * w, nx, inv), (dout * nx).reshape(-1, x.shape[-1]).sum(0)


def block_join(x, y, pw, gate=None, act="sigmoid", scale=None, nw=None, eps=1e-6):
    a = 1.0 if gate is None else _act(gate, act)[0]
    r = x + (1.0 if scale is None else scale) * a * _norm(y, eps)[0] * pw
    return r, None if nw is None else _norm(r, eps)[0] * nw


def block_join_backward(x, y, pw, gate=None, act="sigmoid", scale=None, nw=None, dr=None, dh=None, eps=1e-6):
    """dict of dx, dy, dgate, dpost_weight, dscale, dnext_weight (None where there is no input)"""
    D = x.shape[-1]
    a, slope = (np.ones(1), None) if gate is None else _act(gate, act)
    s = np.ones(D) if scale is None else scale
    ny, inv = _norm(y, eps)
    u = ny * pw
    R = np.zeros_like(x) if dr is None else np.array(dr)
    out = {"dgate": None, "dscale": None, "dnext_weight": None}
    if nw is not None:
        nr, inv_r = _norm(x + s * a * u, eps)
        R = R + _norm_adjoint(dh * nw, nr, inv_r)
        out["dnext_weight"] = (dh * nr).reshape(-1, D).sum(0)
    if gate is not None:
        dz = R * s * u
        out["dgate"] = (dz if gate.shape[-1] == D else dz.sum(-1, keepdims=True)) * slope
    if scale is not None:
        out["dscale"] = (R * a * u).reshape(-1, D).sum(0)
    out["dx"], out["dy"] = R, _norm_adjoint(R * s * a * pw, ny, inv)
    out["dpost_weight"] = (R * s * a * ny).reshape(-1, D).sum(0)
    return out


def w4_matvec(x, qweight, scales, zeros=None, bias=None):
    N, half = qweight.shape
    w = np.empty((N, 2 * half))
    w[:, 0::2] = qweight % 16
    w[:, 1::2] = qweight // 16
    per = 2 * half // scales.shape[1]
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), per, axis=1)
    y = x @ ((w - z) * np.repeat(scales, per, axis=1)).T
    return y if bias is None else y + bias
