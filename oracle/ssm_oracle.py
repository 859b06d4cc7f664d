"""Float64 CPU oracle of a selective state space layer's operators (include/hla2.h), token by token from their
definitions.  Gradients are written out by hand and pinned by differences (tests/test_ssm_oracle.py)."""
import numpy as np


def softplus(v):
    return np.logaddexp(0.0, v)


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def silu(v):
    return v * sigmoid(v)


def dsilu(v):
    s = sigmoid(v)
    return s + v * s * (1.0 - s)


def _lengths(lengths, B, n):
    return [n] * B if lengths is None else [min(max(int(x), 0), n) for x in lengths]


def _grouped(t, D):
    """[G, N] -> [D, N]"""
    return np.repeat(t, D // t.shape[0], axis=0)


def ssm_step(h, x, dt, a, b, c, skip=None, gate=None, dt_bias=None, dt_softplus=True):
    """(out [D], h after, delta) of one token of one sequence: h [D, N], x, dt [D], b, c [G, N]."""
    D = x.shape[0]
    v = dt if dt_bias is None else dt + dt_bias
    delta = softplus(v) if dt_softplus else v
    h = np.exp(delta[:, None] * a) * h + (delta * x)[:, None] * _grouped(b, D)
    y = (h * _grouped(c, D)).sum(-1) + (0.0 if skip is None else skip * x)
    return (y if gate is None else y * silu(gate)), h, delta


def ssm_forward(x, dt, a, b, c, skip=None, gate=None, dt_bias=None, dt_softplus=True, lengths=None, init_state=None):
    """(out [B, n, D], final state [B, D, N]); b, c [B, n, G, N]."""
    B, n, D = x.shape
    out = np.zeros((B, n, D))
    fin = np.zeros((B, D, a.shape[1])) if init_state is None else init_state.copy()
    for s, m in enumerate(_lengths(lengths, B, n)):
        for t in range(m):
            out[s, t], fin[s], _ = ssm_step(fin[s], x[s, t], dt[s, t], a, b[s, t], c[s, t], skip,
                                            None if gate is None else gate[s, t], dt_bias, dt_softplus)
    return out, fin


def ssm_backward(x, dt, a, b, c, dout, skip=None, gate=None, dt_bias=None, dt_softplus=True, lengths=None,
                 init_state=None, dfinal_state=None):
    """dict of the gradients of sum(out * dout) + sum(final * dfinal_state)"""
    B, n, D = x.shape
    G, N = b.shape[2:]
    per = D // G
    g = {"dx": np.zeros((B, n, D)), "ddt": np.zeros((B, n, D)), "da": np.zeros((D, N)), "db": np.zeros((B, n, G, N)),
         "dc": np.zeros((B, n, G, N)), "dskip": np.zeros(D), "dgate": np.zeros((B, n, D)), "ddt_bias": np.zeros(D),
         "dinit_state": np.zeros((B, D, N))}
    for s, m in enumerate(_lengths(lengths, B, n)):
        h = [np.zeros((D, N)) if init_state is None else init_state[s]]
        deltas = []
        for t in range(m):
            _, after, delta = ssm_step(h[-1], x[s, t], dt[s, t], a, b[s, t], c[s, t], skip, None, dt_bias, dt_softplus)
            h.append(after)
            deltas.append(delta)
        R = np.zeros((D, N)) if dfinal_state is None else dfinal_state[s].copy()
        for t in range(m - 1, -1, -1):
            xt, delta, bt, ct = x[s, t], deltas[t], _grouped(b[s, t], D), _grouped(c[s, t], D)
            dy = dout[s, t]
            if gate is not None:
                y = (h[t + 1] * ct).sum(-1) + (0.0 if skip is None else skip * xt)
                g["dgate"][s, t] = dy * y * dsilu(gate[s, t])
                dy = dy * silu(gate[s, t])
            R = R + ct * dy[:, None]
            g["dc"][s, t] = (h[t + 1] * dy[:, None]).reshape(G, per, N).sum(1)
            g["db"][s, t] = (R * (delta * xt)[:, None]).reshape(G, per, N).sum(1)
            into = (R * bt).sum(-1)
            decay = np.exp(delta[:, None] * a)
            E = R * decay * h[t]
            g["da"] += E * delta[:, None]
            dd = (E * a).sum(-1) + into * xt
            if dt_softplus:
                dd = dd * sigmoid(dt[s, t] if dt_bias is None else dt[s, t] + dt_bias)
            g["ddt"][s, t] = dd
            g["ddt_bias"] += dd
            g["dx"][s, t] = into * delta + (0.0 if skip is None else skip * dy)
            g["dskip"] += dy * xt
            R = R * decay
        g["dinit_state"][s] = R
    return g


def _act(p, act):
    return silu(p) if act == "silu" else p


def conv_forward(x, w, bias=None, act="silu", lengths=None, init_state=None):
    """(out [B, n, D], final state [B, W - 1, D]) of the short causal convolution; x [B, n, D], w [D, W]."""
    B, n, D = x.shape
    W = w.shape[1]
    out, fin = np.zeros((B, n, D)), np.zeros((B, W - 1, D))
    for s, m in enumerate(_lengths(lengths, B, n)):
        line = np.concatenate((np.zeros((W - 1, D)) if init_state is None else init_state[s], x[s, :m]))
        for t in range(m):
            out[s, t] = _act((line[t:t + W] * w.T).sum(0) + (0.0 if bias is None else bias), act)
        fin[s] = line[m:]
    return out, fin


def conv_backward(x, w, dout, bias=None, act="silu", lengths=None, init_state=None, dfinal_state=None):
    B, n, D = x.shape
    W = w.shape[1]
    g = {"dx": np.zeros((B, n, D)), "dweight": np.zeros((D, W)), "dbias": np.zeros(D), "dinit_state": np.zeros((B, W - 1, D))}
    for s, m in enumerate(_lengths(lengths, B, n)):
        line = np.concatenate((np.zeros((W - 1, D)) if init_state is None else init_state[s], x[s, :m]))
        dline = np.zeros_like(line)
        if dfinal_state is not None:
            dline[m:] += dfinal_state[s]
        for t in range(m):
            p = (line[t:t + W] * w.T).sum(0) + (0.0 if bias is None else bias)
            dp = dout[s, t] * (dsilu(p) if act == "silu" else 1.0)
            dline[t:t + W] += w.T * dp
            g["dweight"] += (line[t:t + W] * dp).T
            g["dbias"] += dp
        g["dx"][s, :m] = dline[W - 1:]
        g["dinit_state"][s] = dline[:W - 1]
    return g


def layer_norm(x, w, bias=None, eps=1e-5):
    x = x - x.mean(-1, keepdims=True)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return y if bias is None else y + bias


def layer_norm_backward(x, w, dout, eps=1e-5):
    """(dx, dweight, dbias)"""
    x = x - x.mean(-1, keepdims=True)
    inv = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    nx, g = x * inv, dout * w
    dx = inv * (g - g.mean(-1, keepdims=True) - nx * (g * nx).mean(-1, keepdims=True))
    flat = lambda t: t.reshape(-1, x.shape[-1]).sum(0)  # noqa: E731
    return dx, flat(dout * nx), flat(dout)
