"""Cases, plain forms and exact values of the operators of a selective state space layer.

  ssm    the selective scan, a state of N values for each channel with steps, inputs and outputs that
         depend on the token: forward, backward, and single tokens
  conv   the short causal convolution before it, for each channel on its own: forward, backward, and
         single tokens
  norm   layer norm, forward and backward with the sums of the weight's and the bias's gradients

``own`` selects the framework's calls (True) or the plain form in elementary torch operations in 32
bits (False); both take what ``prepare`` gives.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def _ssm(name, op, B, n, D, N, G, dtype, gate=True, ragged=False, state=False, projected=False):
    return {"name": name, "op": op, "B": B, "n": n, "D": D, "N": N, "G": G, "dtype": dtype, "gate": gate,
            "ragged": ragged, "state": state, "projected": projected}


def _conv(name, op, B, n, D, W, dtype, act="silu", bias=True, ragged=False, state=False):
    return {"name": name, "op": op, "B": B, "n": n, "D": D, "W": W, "dtype": dtype, "act": act, "bias": bias,
            "ragged": ragged, "state": state}


def _norm(name, op, rows, D, dtype, bias=True):
    return {"name": name, "op": op, "rows": rows, "D": D, "dtype": dtype, "bias": bias}


def listed():
    return [
        # a batch of two prompts of different lengths, read as the projections leave them, with the state
        # that decoding goes on from
        _ssm("scan_prompts", "ssm", 2, 2048, 2048, 16, 1, "bf16", True, True, True, True),
        # one long document
        _ssm("scan_long", "ssm", 1, 65536, 2048, 16, 1, "bf16"),
        # a training step of one layer: forward, then every gradient
        _ssm("scan_train", "ssm_train", 4, 4096, 2048, 16, 1, "bf16"),
        # a small training step in float32: odd length and channels, two groups, states of 32, no gate
        _ssm("scan_train_f32", "ssm_train", 2, 1023, 330, 32, 2, "f32", False, True, True),
        # one token for each of 256 running sequences
        _ssm("scan_step_256", "ssm_step", 256, 1, 4096, 16, 1, "bf16"),
        # one token of one sequence: latency
        _ssm("scan_step_one", "ssm_step", 1, 1, 2048, 16, 1, "bf16"),
        # the convolution of one long document
        _conv("conv_long", "conv", 1, 65536, 2048, 4, "bf16"),
        # a small training step in float32 with three taps, odd sizes, a state before and after
        _conv("conv_train_f32", "conv_train", 3, 1021, 777, 3, "f32", "silu", True, True, True),
        # one token for each of 256 running sequences
        _conv("conv_step_256", "conv_step", 256, 1, 4096, 4, "bf16"),
        # the norm of a few running tokens: latency
        _norm("norm_tokens", "norm", 4, 2048, "bf16"),
        # a training step's norm, forward and backward
        _norm("norm_train", "norm_train", 32768, 2048, "bf16"),
        # the same in float32 at an odd width
        _norm("norm_train_f32", "norm_train", 5000, 999, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ssm", "ssm", "ssm_train", "ssm_train", "ssm_step", "conv", "conv_train", "conv_step", "norm",
                     "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_train"):
        D = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            D = max(16, D // 16 * 16)
        rows = _log(rng, 1, max(2, min(32768, 32768 * 2048 // D // (2 if dtype == "f32" else 1))))
        return _norm("", op, rows, D, dtype, rng.random() < 0.7)
    G = rng.choice([1, 1, 1, 2, 4])
    D = G * _log(rng, 48 // G, 4096 // G)
    if rng.random() < 0.6:
        D = max(64, D // 64 * 64)
    if op in ("ssm_step", "conv_step"):
        B = _log(rng, 1, 256)
    else:
        B = _log(rng, 1, 8)
    if op in ("conv", "conv_train", "conv_step"):
        # values: at most the long case's (a quarter of it in training, half of that in float32)
        most = (1 << 27) // (4 if op == "conv_train" else 1) // (2 if dtype == "f32" else 1)
        n = 1 if op == "conv_step" else _log(rng, 1, max(2, min(65536, most // (B * D))))
        return _conv("", op, B, n, D, rng.choice([2, 3, 4, 4]), dtype, rng.choice(["silu", "silu", "none"]),
                     rng.random() < 0.7, rng.random() < 0.4, op == "conv_step" or rng.random() < 0.5)
    N = rng.choice([8, 16, 16, 32, 64])
    if op == "ssm_step":
        return _ssm("", op, max(1, B * 16 // N if N > 16 else B), 1, D, N, G, dtype, rng.random() < 0.7)
    # state updates: at most the long case's (a quarter of it in training, half of that in float32)
    most = (1 << 31) // (4 if op == "ssm_train" else 1) // (2 if dtype == "f32" else 1)
    n = _log(rng, 1, max(2, min(65536, most // (B * D * N))))
    return _ssm("", op, B, n, D, N, G, dtype, rng.random() < 0.7, rng.random() < 0.4, rng.random() < 0.5,
                rng.random() < 0.5)


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 29)
    t = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device=dev, dtype=torch.float32)

    op = case["op"]
    s = {"case": dict(case)}
    if op in ("norm", "norm_train"):
        rows, D = case["rows"], case["D"]
        s["x"] = (0.5 + 2.0 * normal(rows, D)).to(t)
        s["weight"] = uniform(0.5, 1.5, D).to(t)
        s["bias"] = (0.1 * normal(D)).to(t) if case["bias"] else None
        s["dout"] = normal(rows, D).to(t)
        return s
    B, n, D = case["B"], case["n"], case["D"]
    step = op in ("ssm_step", "conv_step")
    s["lengths"] = None
    if not step and case["ragged"]:
        s["lengths"] = torch.randint(0, n + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        s["lengths"][0] = n
    if op in ("conv", "conv_train", "conv_step"):
        W = case["W"]
        s["weight"] = (normal(D, W) / math.sqrt(W)).to(t)
        s["bias"] = (0.1 * normal(D)).to(t) if case["bias"] else None
        s["x"] = normal(*((B, D) if step else (B, n, D))).to(t)
        s["state"] = normal(B, W - 1, D).to(t) if case["state"] or step else None
        if op == "conv_train":
            s["dout"] = normal(B, n, D).to(t)
            s["dfinal"] = normal(B, W - 1, D).to(t) if case["state"] else None
        return s
    N, G = case["N"], case["G"]
    # decays and steps as such layers start with: -1 .. -N for the states, steps from 0.001 to 0.1
    s["a"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(0.2 * normal(D, 1))
    dt = torch.exp(uniform(math.log(1e-3), math.log(1e-1), D))
    s["dt_bias"] = dt + torch.log(-torch.expm1(-dt))
    s["skip"] = uniform(0.5, 1.5, D)
    if step:
        s["x"], s["dt"] = normal(B, D).to(t), (0.5 * normal(B, D)).to(t)
        s["b"], s["c"] = normal(B, G, N).to(t), normal(B, G, N).to(t)
        s["gate"] = normal(B, D).to(t) if case["gate"] else None
        s["state"] = normal(B, D, N)
        return s
    if case["projected"]:  # halves of one projection, and parts of another
        xz = normal(B, n, 2 * D).to(t)
        s["x"], s["gate"] = xz[..., :D], xz[..., D:] if case["gate"] else None
        bc = normal(B, n, 2 * G * N).to(t)
        s["b"], s["c"] = bc[..., :G * N].unflatten(-1, (G, N)), bc[..., G * N:].unflatten(-1, (G, N))
    else:
        s["x"], s["gate"] = normal(B, n, D).to(t), normal(B, n, D).to(t) if case["gate"] else None
        s["b"], s["c"] = normal(B, n, G, N).to(t), normal(B, n, G, N).to(t)
    s["dt"] = (0.5 * normal(B, n, D)).to(t)
    s["init"] = normal(B, D, N) if case["state"] else None
    if op == "ssm_train":
        s["dout"] = normal(B, n, D).to(t)
        s["dfinal"] = normal(B, D, N) if case["state"] else None
    return s


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1: neighbours are joined to pairs, the pairs are scanned, and the
    tokens between them follow."""
    n = a.shape[1]
    if n == 1:
        return b
    even = n // 2 * 2
    a0, a1, b0, b1 = a[:, 0:even:2], a[:, 1:even:2], b[:, 0:even:2], b[:, 1:even:2]
    h1 = _scan(a1 * a0, a1 * b0 + b1)
    h = torch.empty_like(b)
    h[:, 0] = b[:, 0]
    h[:, 1:even:2] = h1
    if n > 2:
        h[:, 2::2] = a[:, 2::2] * h1[:, :(n - 1) // 2] + b[:, 2::2]
    return h


def _valid(s, n):
    """[B, n, 1], whether a token is within its sequence"""
    t = torch.arange(n, device=s["x"].device)
    lengths = s["lengths"] if s["lengths"] is not None else torch.full((s["x"].shape[0],), n, device=t.device)
    return (t[None] < lengths[:, None])[..., None]


def _softplus(v):
    return v.clamp_min(0) + torch.log1p(torch.exp(-v.abs()))


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _channels(t, D):
    """[B, n, G, N] -> [B, n, D, N], each group's values for its channels"""
    return t.repeat_interleave(D // t.shape[2], dim=2)


def _plain_ssm(s):
    c = s["case"]
    B, n, D, N, G = (c[k] for k in ("B", "n", "D", "N", "G"))
    t = s["x"].dtype
    valid = _valid(s, n)
    zero = torch.zeros((), device=s["x"].device)
    x = torch.where(valid, s["x"].float(), zero)
    v = s["dt"].float() + s["dt_bias"]
    delta = torch.where(valid, _softplus(v), zero)
    b, cc = (torch.where(valid[..., None], s[k].float(), zero) for k in ("b", "c"))
    a = torch.exp(delta[..., None] * s["a"])
    u = (delta * x)[..., None] * _channels(b, D)
    if s["init"] is not None:
        u[:, 0] += a[:, 0] * s["init"]
    h = _scan(a, u)
    del u
    y = (h * _channels(cc, D)).sum(-1) + s["skip"] * x
    gate = sig = None
    if s["gate"] is not None:
        z = s["gate"].float()
        sig = _sigmoid(z)
        gate = z * sig
    res = [torch.where(valid, y if gate is None else y * gate, zero).to(t)]
    if c["state"]:
        res.append(h[:, -1].clone())
    if c["op"] == "ssm":
        return res
    do = torch.where(valid, s["dout"].float(), zero)
    dy, dgate = do, None
    if gate is not None:
        dy = torch.where(valid, do * gate, zero)
        dgate = torch.where(valid, do * y * sig * (1.0 + z * (1.0 - sig)), zero)
    dc = (h * dy[..., None]).unflatten(2, (G, D // G)).sum(3)
    g = _channels(cc, D) * dy[..., None]
    if s["dfinal"] is not None:
        g[:, -1] += s["dfinal"]
    after = torch.cat((torch.ones_like(a[:, :1]), a[:, 1:].flip(1)), 1)  # the decay from the token before, in reverse
    dh = _scan(after, g.flip(1)).flip(1)
    del g, after
    db = (dh * (delta * x)[..., None]).unflatten(2, (G, D // G)).sum(3)
    into = (dh * _channels(b, D)).sum(-1)
    dh *= a
    dinit = dh[:, 0].clone() if s["init"] is not None else None
    # the gradient of the exponent
    dh[:, 1:] *= h[:, :-1]
    dh[:, 0] *= s["init"] if s["init"] is not None else zero
    da = (dh * delta[..., None]).sum((0, 1))
    ddelta = (dh * s["a"]).sum(-1) + into * x
    ddt = torch.where(valid, ddelta * _sigmoid(v), zero)
    dx = delta * into + s["skip"] * dy
    res += [dx.to(t), ddt.to(t), da, db.to(t), dc.to(t), (dy * x).sum((0, 1))]
    if gate is not None:
        res.append(dgate.to(t))
    res.append(ddt.sum((0, 1)))
    return res if dinit is None else res + [dinit]


def _plain_ssm_step(s):
    D = s["case"]["D"]
    x = s["x"].float()
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    b, c = (s[k].float().repeat_interleave(D // s[k].shape[1], dim=1) for k in ("b", "c"))
    s["state"].mul_(torch.exp(delta[..., None] * s["a"])).add_((delta * x)[..., None] * b)
    y = (s["state"] * c).sum(-1) + s["skip"] * x
    if s["gate"] is not None:
        z = s["gate"].float()
        y = y * z * _sigmoid(z)
    return [y.to(s["x"].dtype), s["state"]]


def _act(p, act):
    """(act(p), act'(p))"""
    if act == "none":
        return p, torch.ones((), device=p.device)
    sig = _sigmoid(p)
    return p * sig, sig * (1.0 + p * (1.0 - sig))


def _plain_conv(s):
    c = s["case"]
    B, n, D, W = (c[k] for k in ("B", "n", "D", "W"))
    t = s["x"].dtype
    valid = _valid(s, n)
    zero = torch.zeros((), device=s["x"].device)
    before = s["state"].float() if s["state"] is not None else zero.expand(B, W - 1, D)
    xs = torch.cat((before, torch.where(valid, s["x"].float(), zero)), 1)  # token t at t + W - 1
    w = s["weight"].float()
    p = sum(w[:, j] * xs[:, j:j + n] for j in range(W))
    if s["bias"] is not None:
        p = p + s["bias"].float()
    y, slope = _act(p, c["act"])
    res = [torch.where(valid, y, zero).to(t)]
    lengths = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), n, device=w.device)
    last = (lengths[:, None] + torch.arange(W - 1, device=w.device))[..., None].expand(B, W - 1, D)
    if c["state"]:
        res.append(xs.gather(1, last).to(t))
    if c["op"] == "conv":
        return res
    dp = torch.where(valid, s["dout"].float() * slope, zero)
    padded = torch.nn.functional.pad(dp, (0, 0, W - 1, W - 1))  # token t at t + W - 1
    dxs = sum(w[:, j] * padded[:, W - 1 - j:W - 1 - j + n + W - 1] for j in range(W))
    if s["dfinal"] is not None:
        dxs = dxs.scatter_add(1, last, s["dfinal"].float())
    res += [torch.where(valid, dxs[:, W - 1:], zero).to(t),
            torch.stack([(dp * xs[:, j:j + n]).sum((0, 1)) for j in range(W)], -1)]
    if s["bias"] is not None:
        res.append(dp.sum((0, 1)))
    return res + ([dxs[:, :W - 1].to(t)] if s["state"] is not None else [])


def _plain_conv_step(s):
    c = s["case"]
    xs = torch.cat((s["state"].float(), s["x"].float()[:, None]), 1)
    p = (xs * s["weight"].float().t()).sum(1)
    if s["bias"] is not None:
        p = p + s["bias"].float()
    s["state"].copy_(xs[:, 1:])
    return [_act(p, c["act"])[0].to(s["x"].dtype), s["state"]]


def _plain_norm(s):
    x, w = s["x"].float(), s["weight"].float()
    t = s["x"].dtype
    x = x - x.mean(-1, keepdim=True)
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    nx = x * inv
    y = nx * w if s["bias"] is None else nx * w + s["bias"].float()
    if s["case"]["op"] == "norm":
        return [y.to(t)]
    do = s["dout"].float()
    g = do * w
    dx = inv * (g - g.mean(-1, keepdim=True) - nx * (g * nx).mean(-1, keepdim=True))
    return [y.to(t), dx.to(t), (do * nx).sum(0), do.sum(0)]


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def _own(s):
    import chunked_scan_mixer_gb300 as hla

    c = s["case"]
    op = c["op"]
    if op == "norm":
        return [hla.layer_norm(s["x"], s["weight"], bias=s["bias"], eps=EPS)]
    if op == "norm_train":
        y = hla.layer_norm(s["x"], s["weight"], bias=s["bias"], eps=EPS)
        return [y, *hla.layer_norm_backward(s["x"], s["weight"], s["dout"], eps=EPS)]
    if op == "conv_step":
        return [hla.short_conv_decode_step(s["state"], s["x"], s["weight"], bias=s["bias"], act=c["act"]), s["state"]]
    if op in ("conv", "conv_train"):
        kw = dict(bias=s["bias"], act=c["act"], lengths=s["lengths"], init_state=s["state"])
        res = hla.short_conv_forward(s["x"], s["weight"], return_final_state=c["state"], **kw)
        res = list(res) if c["state"] else [res]
        if op == "conv_train":
            g = hla.short_conv_backward(s["x"], s["weight"], s["dout"], dfinal_state=s["dfinal"], **kw)
            res += [g.dx, g.dweight] + ([] if s["bias"] is None else [g.dbias])
            res += [] if s["state"] is None else [g.dinit_state]
        return res
    kw = dict(skip=s["skip"], gate=s["gate"], dt_bias=s["dt_bias"])
    if op == "ssm_step":
        return [hla.ssm_decode_step(s["state"], s["x"], s["dt"], s["a"], s["b"], s["c"], **kw), s["state"]]
    kw.update(lengths=s["lengths"], init_state=s["init"])
    res = hla.ssm_forward(s["x"], s["dt"], s["a"], s["b"], s["c"], return_final_state=c["state"], **kw)
    res = list(res) if c["state"] else [res]
    if op == "ssm_train":
        g = hla.ssm_backward(s["x"], s["dt"], s["a"], s["b"], s["c"], s["dout"], dfinal_state=s["dfinal"], **kw)
        res += [g.dx, g.ddt, g.da, g.db, g.dc, g.dskip]
        res += ([] if s["gate"] is None else [g.dgate]) + [g.ddt_bias]
        res += [] if s["init"] is None else [g.dinit_state]
    return res


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("ssm", "ssm_train"):
        return _plain_ssm(state)
    if op == "ssm_step":
        return _plain_ssm_step(state)
    if op in ("conv", "conv_train"):
        return _plain_conv(state)
    if op == "conv_step":
        return _plain_conv_step(state)
    return _plain_norm(state)


# ---------------------------------------------------------------------------------------
# least work
# ---------------------------------------------------------------------------------------

def work(case):
    e, op = SIZE[case["dtype"]], case["op"]
    if op in ("norm", "norm_train"):
        v = float(case["rows"] * case["D"])
        return {"bytes": e * v * (2 if op == "norm" else 5), "flops": v * (8 if op == "norm" else 22)}
    B, n, D = case["B"], case["n"], case["D"]
    v = float(B * n * D)
    if op in ("conv", "conv_train", "conv_step"):
        W, st = case["W"], e * float(B * (case["W"] - 1) * D) * case["state"]
        if op == "conv_train":
            return {"bytes": e * v * 5 + 4 * st, "flops": v * (6.0 * W + 12)}
        return {"bytes": e * v * 2 + 2 * st, "flops": v * (2.0 * W + 4)}
    N, G = case["N"], case["G"]
    st, bc = 4.0 * B * D * N, e * 2.0 * B * n * G * N
    rows = e * v * (3 + case["gate"])  # x, dt, the gate and the output
    if op == "ssm_step":
        return {"bytes": 2 * st + rows + bc + 4.0 * D * N, "flops": v * (7.0 * N + 20)}
    st *= 2 * case["state"]
    if op == "ssm":
        return {"bytes": rows + bc + st, "flops": v * (7.0 * N + 20)}
    # the backward reads dout beside the inputs, and writes their gradients
    return {"bytes": rows + bc + st + e * v * (3 + 2 + 2 * case["gate"]) + 2 * bc + st,
            "flops": v * (7.0 * N + 20 + 21.0 * N + 40)}


# ---------------------------------------------------------------------------------------
# exact values, in 64 bits from the definitions
# ---------------------------------------------------------------------------------------

def _exact_ssm(s):
    """Token by token: the states forward, and their gradients back."""
    c = s["case"]
    B, n, D, N, G = (c[k] for k in ("B", "n", "D", "N", "G"))
    dev, train, per = s["x"].device, c["op"] == "ssm_train", D // G
    f = torch.float64
    lengths = [n] * B if s["lengths"] is None else s["lengths"].tolist()
    live = torch.zeros(n, B, 1, dtype=torch.bool, device=dev)
    for i in range(B):
        live[:lengths[i], i] = True
    A, skip = s["a"].double(), s["skip"].double()

    def grouped(t, k):  # [B, G, N] of token t, for the channels
        return s[k][:, t].double()[:, :, None, :].expand(B, G, per, N).reshape(B, D, N)

    def delta_of(t):
        return torch.nn.functional.softplus(s["dt"][:, t].double() + s["dt_bias"].double(), threshold=1e9)

    h = s["init"].double().clone() if s["init"] is not None else torch.zeros(B, D, N, dtype=f, device=dev)
    out = torch.zeros(B, n, D, dtype=f, device=dev)
    dgate = torch.zeros_like(out) if train and s["gate"] is not None else None
    kept = torch.empty(max(lengths), B, D, N, dtype=f, device=dev) if train else None  # the state before each token
    for t in range(max(lengths)):
        if train:
            kept[t] = h
        x, d = s["x"][:, t].double(), delta_of(t)
        after = torch.exp(d[..., None] * A) * h + (d * x)[..., None] * grouped(t, "b")
        h = torch.where(live[t, :, :, None], after, h)
        y = torch.einsum("bdn,bdn->bd", h, grouped(t, "c")) + skip * x
        if s["gate"] is not None:
            z = s["gate"][:, t].double()
            if train:
                m = torch.sigmoid(z)
                dgate[:, t] = torch.where(live[t], s["dout"][:, t].double() * y * (m + z * m * (1 - m)), 0.0)
            y = y * torch.nn.functional.silu(z)
        out[:, t] = torch.where(live[t], y, 0.0)
    res = [out, h] if c["state"] else [out]
    if not train:
        return res
    R = s["dfinal"].double().clone() if s["dfinal"] is not None else torch.zeros(B, D, N, dtype=f, device=dev)
    dx, ddt = torch.zeros_like(out), torch.zeros_like(out)
    db = torch.zeros(B, n, G, N, dtype=f, device=dev)
    dc = torch.zeros_like(db)
    da, dskip, dbias = torch.zeros_like(A), torch.zeros_like(skip), torch.zeros_like(skip)
    for t in range(max(lengths) - 1, -1, -1):
        on = live[t].double()
        x, d, prev = s["x"][:, t].double() * on, delta_of(t), kept[t]
        x, d = torch.where(live[t], x, 0.0), torch.where(live[t], d, 0.0)
        bt, ct = (torch.where(live[t, :, :, None], grouped(t, k), 0.0) for k in ("b", "c"))
        dy = torch.where(live[t], s["dout"][:, t].double(), 0.0)
        if s["gate"] is not None:
            dy = torch.where(live[t], dy * torch.nn.functional.silu(s["gate"][:, t].double()), 0.0)
        dec = torch.exp(d[..., None] * A)
        now = dec * prev + (d * x)[..., None] * bt
        dc[:, t] = (now * dy[..., None]).reshape(B, G, per, N).sum(2)
        R = R + ct * dy[..., None]
        db[:, t] = (R * (d * x)[..., None]).reshape(B, G, per, N).sum(2)
        du = (R * bt).sum(-1)
        E = R * dec * prev
        da += torch.einsum("bdn,bd->dn", E, d)
        dd = (E * A).sum(-1) + du * x
        back = torch.where(live[t], dd * torch.sigmoid(s["dt"][:, t].double() + s["dt_bias"].double()), 0.0)
        ddt[:, t] = back
        dbias += back.sum(0)
        dx[:, t] = du * d + skip * dy
        dskip += (dy * x).sum(0)
        R = R * dec
    res += [dx, ddt, da, db, dc, dskip]
    res += ([] if dgate is None else [dgate]) + [dbias]
    return res + ([R] if s["init"] is not None else [])


def _exact_conv(s):
    """The definition sequence by sequence, and its gradients by differentiation."""
    c = s["case"]
    B, n, D, W = (c[k] for k in ("B", "n", "D", "W"))
    p = {k: s[k].double().requires_grad_() for k in ("x", "weight", "bias", "state") if s[k] is not None}
    lengths = [n] * B if s["lengths"] is None else s["lengths"].tolist()
    outs, finals = [], []
    for i in range(B):
        m = lengths[i]
        first = p["state"][i] if "state" in p else torch.zeros(W - 1, D, dtype=torch.float64, device=s["x"].device)
        line = torch.cat((first, p["x"][i, :m]))
        y = torch.nn.functional.conv1d(line.t()[None], p["weight"][:, None], p.get("bias"), groups=D)[0].t() if m else line[:0]
        if c["act"] == "silu":
            y = torch.nn.functional.silu(y)
        outs.append(torch.nn.functional.pad(y, (0, 0, 0, n - m)))
        finals.append(line[m:])
    out, final = torch.stack(outs), torch.stack(finals)
    res = [out.detach()] + ([final.detach()] if c["state"] else [])
    if c["op"] == "conv":
        return res
    total = (out * s["dout"].double()).sum()
    if s["dfinal"] is not None:
        total = total + (final * s["dfinal"].double()).sum()
    return res + list(torch.autograd.grad(total, [p[k] for k in ("x", "weight", "bias", "state") if k in p]))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("ssm", "ssm_train"):
        return _exact_ssm(s)
    if op in ("conv", "conv_train"):
        return _exact_conv(s)
    if op == "ssm_step":
        per = case["D"] // case["G"]
        d = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=1e9)
        b, c = (torch.repeat_interleave(s[k].double(), per, 1) for k in ("b", "c"))
        h = s["state"].double() * torch.exp(d[..., None] * s["a"].double()) + torch.einsum("bd,bdn->bdn", d * s["x"].double(), b)
        y = torch.einsum("bdn,bdn->bd", h, c) + s["skip"].double() * s["x"].double()
        return [y if s["gate"] is None else y * torch.nn.functional.silu(s["gate"].double()), h]
    if op == "conv_step":
        line = torch.cat((s["state"].double(), s["x"].double()[:, None]), 1)
        y = torch.einsum("bwd,dw->bd", line, s["weight"].double())
        y = y if s["bias"] is None else y + s["bias"].double()
        return [torch.nn.functional.silu(y) if case["act"] == "silu" else y, line[:, 1:]]
    p = {k: s[k].double().requires_grad_() for k in ("x", "weight")}
    bias = (s["bias"].double() if s["bias"] is not None else torch.zeros_like(p["weight"])).detach().requires_grad_()
    mean = p["x"].sum(-1, keepdim=True) / case["D"]
    var = ((p["x"] - mean) ** 2).sum(-1, keepdim=True) / case["D"]
    y = (p["x"] - mean) / torch.sqrt(var + EPS) * p["weight"] + bias
    if op == "norm":
        return [y.detach()]
    return [y.detach(), *torch.autograd.grad((y * s["dout"].double()).sum(), [p["x"], p["weight"], bias])]
