"""Cases, plain forms and exact values of the operators around a first-order mixer layer.

  linattn   linear attention with a decay for each head: chunked forward and backward, and
            the recurrent step of single tokens
  join      the norms before and after a block, fused with the block's gate and residual
            scale; norm is the one before a block alone
  w4        matrix-vector products with 4-bit weights and group scales

``own`` selects the framework's calls (True) or the plain form in elementary torch
operations in 32 bits (False); both take what ``prepare`` gives.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6
CHUNK = 128  # width of the plain form's chunks


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def _linattn(name, op, B, H, Hk, n, d, dv, dtype, ragged=False, state=False, tokens_first=False):
    return {"name": name, "op": op, "B": B, "H": H, "Hk": Hk, "n": n, "d": d, "dv": dv, "dtype": dtype,
            "ragged": ragged, "state": state, "tokens_first": tokens_first}


def _step(name, N, H, Hk, d, dv, dtype):
    return {"name": name, "op": "step", "N": N, "H": H, "Hk": Hk, "d": d, "dv": dv, "dtype": dtype}


def _rows(name, op, rows, D, dtype, gate="full", act="sigmoid"):
    return {"name": name, "op": op, "rows": rows, "D": D, "dtype": dtype, "gate": gate, "act": act}


def _w4(name, M, N, K, group, dtype, zeros, bias):
    return {"name": name, "op": "w4", "M": M, "N": N, "K": K, "group": group, "dtype": dtype, "zeros": zeros,
            "bias": bias}


def listed():
    return [
        # a batch of two prompts of different lengths, read as the projections leave them
        # (token-major), with the state that decoding goes on from
        _linattn("prompts", "forward", 2, 8, 8, 2048, 64, 64, "bf16", True, True, True),
        # one long document
        _linattn("long", "forward", 1, 16, 16, 65536, 64, 64, "bf16"),
        # prompts continued from a kept state, four query heads to a key head
        _linattn("shared_heads", "forward", 4, 32, 8, 4096, 128, 128, "bf16", False, True, True),
        # a training step of one layer: forward, then the gradients of q, k and v
        _linattn("train", "train", 4, 16, 16, 8192, 128, 128, "bf16"),
        # a small training step in float32, odd length, values wider than keys, shared heads
        _linattn("train_f32", "train", 1, 4, 2, 1023, 32, 64, "f32", True, True),
        # one token for each of 256 running sequences
        _step("step_256", 256, 32, 32, 128, 128, "bf16"),
        # one token of one sequence: latency
        _step("step_one", 1, 16, 4, 64, 64, "bf16"),
        # the end of a block for a few running tokens: latency
        _rows("join_tokens", "join", 4, 2048, "bf16", "full", "silu"),
        # a training step's block end, forward and backward
        _rows("join_train", "join_train", 32768, 2048, "bf16"),
        # the first norm of a stack in float32, odd width, forward and backward
        _rows("norm_train", "norm_train", 5000, 999, "f32"),
        # a wide projection of one token
        _w4("w4_token", 1, 8192, 2048, 128, "bf16", True, False),
        # a large projection of a dozen tokens, odd number of outputs
        _w4("w4_streams", 12, 10001, 8192, 64, "bf16", False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "train", "train", "step", "join", "join_train", "norm_train", "w4", "w4"])
    if op in ("forward", "train"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        d = rng.choice([16, 32, 64, 64, 128, 128])
        dv = d if rng.random() < 0.7 else rng.choice([16, 32, 64, 128])
        Hk = rng.randint(1, 16)
        H = Hk * rng.choice([1, 1, 2, 4])
        B = _log(rng, 1, 8)
        # tokens of all heads: at most the long case's (a quarter of it in float32 or training)
        most = (1 << 20) // (4 if dtype == "f32" else 1) // (2 if op == "train" else 1) * 64 // max(d, dv)
        n = _log(rng, 1, max(2, min(65536, most // (B * H))))
        return _linattn("", op, B, H, Hk, n, d, dv, dtype, rng.random() < 0.4, rng.random() < 0.5,
                        rng.random() < 0.5)
    if op == "step":
        Hk = rng.randint(1, 32)
        return _step("", _log(rng, 1, 256), Hk * (rng.choice([1, 1, 2, 4]) if Hk <= 8 else 1), Hk,
                     rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "f32"]))
    if op == "w4":
        group = rng.choice([32, 64, 128])
        return _w4("", rng.choice([1, 1, 1, 2, 3, 5, 8, 11, 16]), _log(rng, 17, 10001),
                   group * _log(rng, 1, 8192 // group), group, rng.choice(["bf16", "bf16", "f32"]),
                   rng.random() < 0.5, rng.random() < 0.5)
    D = _log(rng, 16, 8192)
    if rng.random() < 0.6:
        D = max(16, D // 16 * 16)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rows = _log(rng, 1, max(2, min(32768, 32768 * 2048 // D // (2 if dtype == "f32" else 1))))
    return _rows("", op, rows, D, dtype, rng.choice(["full", "full", "row", "none"]), rng.choice(["sigmoid", "silu"]))


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 17)
    t = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device=dev, dtype=torch.float32)

    op = case["op"]
    s = {"case": dict(case)}
    if op in ("forward", "train", "step"):
        H, Hk, d, dv = (case[x] for x in ("H", "Hk", "d", "dv"))
        s["scale"] = 1.0 / math.sqrt(d)
        # memory lengths from tens of tokens to thousands, as a stack of such heads has
        s["gamma"] = 1.0 - torch.exp(uniform(math.log(2e-4), math.log(5e-2), Hk))
        if op == "step":
            N = case["N"]
            s["q"] = normal(N, H, d).to(t)
            s["k"] = (normal(N, Hk, d) / math.sqrt(d)).to(t)
            s["v"] = normal(N, Hk, dv).to(t)
            s["state"] = normal(N, Hk, d, dv)
            return s
        B, n = case["B"], case["n"]

        def tokens(heads, dim, by=1.0):
            if case["tokens_first"]:
                return (normal(B, n, heads, dim) * by).to(t).transpose(1, 2)
            return (normal(B, heads, n, dim) * by).to(t)

        s["q"] = tokens(H, d)
        s["k"] = tokens(Hk, d, 1.0 / math.sqrt(d))
        s["v"] = tokens(Hk, dv)
        s["lengths"] = None
        if case["ragged"]:
            s["lengths"] = torch.randint(0, n + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
            s["lengths"][0] = n
        s["init"] = normal(B, Hk, d, dv) if case["state"] else None
        if op == "train":
            s["dout"] = tokens(H, dv)
            s["dfinal"] = normal(B, Hk, d, dv) if case["state"] else None
        return s
    if op == "w4":
        M, N, K, g = (case[x] for x in ("M", "N", "K", "group"))
        s["x"] = normal(M, K).to(t)
        s["qweight"] = torch.randint(0, 256, (N, K // 2), generator=gen, device=dev, dtype=torch.uint8)
        s["scales"] = (uniform(0.2, 1.0, N, K // g) / math.sqrt(K)).to(t)
        s["zeros"] = (torch.randint(0, 16, (N, K // g), generator=gen, device=dev, dtype=torch.uint8)
                      if case["zeros"] else None)
        s["bias"] = normal(N).to(t) if case["bias"] else None
        return s
    rows, D = case["rows"], case["D"]
    s["x"] = (2.0 * normal(rows, D)).to(t)
    s["next_weight"] = uniform(0.5, 1.5, D).to(t)
    s["dh"] = normal(rows, D).to(t)
    if op == "norm_train":
        return s
    s["y"] = normal(rows, D).to(t)
    s["gate"] = None if case["gate"] == "none" else normal(rows, D if case["gate"] == "full" else 1).to(t)
    s["post_weight"] = uniform(0.5, 1.5, D).to(t)
    s["scale"] = uniform(0.1, 1.0, D).to(t)
    s["dr"] = normal(rows, D).to(t)
    return s


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------

def _powers(gamma, exponents):
    """gamma[h] ** exponents [...] -> [h, ...] float32, formed in 64 bits (far positions)."""
    lg = torch.log(gamma.double())
    return torch.exp(lg.reshape(-1, *([1] * exponents.dim())) * exponents).float()


def _scan(x, k, v, gamma):
    """y_t = sum_{i <= t} gamma^(t-i) (x_t . k_i) v_i by chunks, all float32 [B, H, n, *]."""
    B, H, n, d = x.shape
    dv = v.shape[-1]
    C = max(1, -(-n // CHUNK))
    pad = C * CHUNK - n
    xc, kc, vc = (torch.nn.functional.pad(t, (0, 0, 0, pad)).reshape(B, H, C, CHUNK, -1) for t in (x, k, v))
    r = torch.arange(CHUNK, device=x.device, dtype=torch.float64)
    c = torch.arange(C, device=x.device, dtype=torch.float64)
    inside = _powers(gamma, (r[:, None] - r[None, :]).clamp_min(0)) * (r[:, None] >= r[None, :])
    across = _powers(gamma, (CHUNK * (c[:, None] - 1 - c[None, :])).clamp_min(0)) * (c[:, None] > c[None, :])
    y = torch.matmul(torch.matmul(xc, kc.transpose(-1, -2)) * inside[:, None], vc)
    state = torch.matmul((kc * _powers(gamma, CHUNK - 1 - r)[:, None, :, None]).transpose(-1, -2), vc)
    carry = torch.matmul(across, state.reshape(B, H, C, d * dv)).reshape(B, H, C, d, dv)
    y = y + torch.matmul(xc * _powers(gamma, r + 1)[:, None, :, None], carry)
    return y.reshape(B, H, C * CHUNK, dv)[:, :, :n]


def _lin_common(s):
    c = s["case"]
    rep = c["H"] // c["Hk"]
    n = c["n"]
    t = torch.arange(n, device=s["q"].device)
    lengths = s["lengths"] if s["lengths"] is not None else torch.full((c["B"],), n, device=t.device)
    lengths = lengths.long()
    valid = (t[None] < lengths[:, None])[:, None, :, None]
    # decay from a token to the end, and from the start to a token, [B, Hk, n]
    lg = torch.log(s["gamma"].double())[None, :, None]
    to_end = torch.exp(lg * (lengths[:, None, None] - 1 - t).clamp_min(0)).float()
    from_start = torch.exp(lg * (t + 1.0)).float().expand(c["B"], -1, -1)
    whole = torch.exp(lg[..., None] * lengths[:, None, None, None]).float()
    return rep, valid, to_end, from_start, whole


def _heads(t, rep):
    return t if rep == 1 else t.repeat_interleave(rep, dim=1)


def _group_sum(t, rep):
    return t if rep == 1 else t.reshape(t.shape[0], t.shape[1] // rep, rep, *t.shape[2:]).sum(2)


def _plain_linattn(s):
    c = s["case"]
    rep, valid, to_end, from_start, whole = _lin_common(s)
    t = s["q"].dtype
    zero = torch.zeros((), device=s["q"].device)
    q, k, v = (torch.where(valid, s[x].float(), zero) for x in ("q", "k", "v"))
    gam = s["gamma"] if rep == 1 else s["gamma"].repeat_interleave(rep)
    kh, vh = _heads(k, rep), _heads(v, rep)
    scale = s["scale"]
    start = _heads(from_start, rep)[..., None]
    o = _scan(q, kh, vh, gam)
    if s["init"] is not None:
        o = o + torch.matmul(q * start, _heads(s["init"], rep))
    res = [torch.where(valid, scale * o, zero).to(t)]
    if c["state"]:
        final = torch.matmul((k * to_end[..., None]).transpose(-1, -2), v)
        if s["init"] is not None:
            final = final + whole * s["init"]
        res.append(final)
    if c["op"] == "forward":
        return res
    do = torch.where(valid, s["dout"].float(), zero) * scale
    dq = _scan(do, vh, kh, gam)
    if s["init"] is not None:
        dq = dq + torch.matmul(do * start, _heads(s["init"], rep).transpose(-1, -2))
    qf, kf, vf, dof = (x.flip(2) for x in (q, kh, vh, do))
    dk = _group_sum(_scan(vf, dof, qf, gam).flip(2), rep)
    dv = _group_sum(_scan(kf, qf, dof, gam).flip(2), rep)
    if s["dfinal"] is not None:
        dk = dk + torch.matmul(v * to_end[..., None], s["dfinal"].transpose(-1, -2))
        dv = dv + torch.matmul(k * to_end[..., None], s["dfinal"])
    res += [torch.where(valid, g, zero).to(t) for g in (dq, dk, dv)]
    if s["init"] is not None:
        dinit = _group_sum(torch.matmul((q * start).transpose(-1, -2), do), rep)
        if s["dfinal"] is not None:
            dinit = dinit + whole * s["dfinal"]
        res.append(dinit)
    return res


def _plain_step(s):
    c = s["case"]
    N, Hk, rep = c["N"], c["Hk"], c["H"] // c["Hk"]
    k, v, q = s["k"].float(), s["v"].float(), s["q"].float()
    s["state"].mul_(s["gamma"].reshape(1, Hk, 1, 1)).add_(k[..., :, None] * v[..., None, :])
    o = torch.matmul(q.reshape(N, Hk, rep, c["d"]), s["state"]).reshape(N, c["H"], c["dv"])
    return [(s["scale"] * o).to(s["q"].dtype), s["state"]]


def _rms(t):
    return torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)


def _norm_back(dn, n, inv):
    """Gradient of n = t * inv(t) for the gradient dn of n."""
    return inv * (dn - n * (dn * n).mean(-1, keepdim=True))


def _plain_rows(s):
    c = s["case"]
    t = s["x"].dtype
    x, w = s["x"].float(), s["next_weight"].float()
    if c["op"] == "norm_train":
        inv = _rms(x)
        nx, dh = x * inv, s["dh"].float()
        return [(nx * w).to(t), _norm_back(dh * w, nx, inv).to(t), (dh * nx).sum(0)]
    y, pw, scale = s["y"].float(), s["post_weight"].float(), s["scale"].float()
    inv = _rms(y)
    ny = y * inv
    u = ny * pw
    if s["gate"] is None:
        a, slope = torch.ones((), device=x.device), None
    else:
        z = s["gate"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        a = sig if c["act"] == "sigmoid" else z * sig
        slope = sig * (1.0 - sig) if c["act"] == "sigmoid" else sig * (1.0 + z * (1.0 - sig))
    r = x + scale * a * u
    inv_r = _rms(r)
    nr = r * inv_r
    res = [r.to(t), (nr * w).to(t)]
    if c["op"] == "join":
        return res
    dh = s["dh"].float()
    dr = s["dr"].float() + _norm_back(dh * w, nr, inv_r)
    du = dr * scale * a
    res += [dr.to(t), _norm_back(du * pw, ny, inv).to(t)]
    if s["gate"] is not None:
        dz = dr * scale * u
        dz = (dz if c["gate"] == "full" else dz.sum(-1, keepdim=True)) * slope
        res.append(dz.to(t))
    return res + [(du * ny).sum(0), (dr * a * u).sum(0), (dh * nr).sum(0)]


def _plain_w4(s):
    c = s["case"]
    N, K, g = c["N"], c["K"], c["group"]
    w = torch.stack((s["qweight"] & 15, s["qweight"] >> 4), dim=-1).reshape(N, K // g, g).float()
    w = w - (8.0 if s["zeros"] is None else s["zeros"].float()[..., None])
    w = (w * s["scales"].float()[..., None]).reshape(N, K)
    y = torch.matmul(s["x"].float(), w.transpose(0, 1))
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def _own(s):
    import chunked_scan_mixer_gb300 as hla

    c = s["case"]
    op = c["op"]
    if op == "step":
        o = hla.linattn_decode_step(s["state"], s["q"], s["k"], s["v"], gamma=s["gamma"], scale=s["scale"])
        return [o, s["state"]]
    if op in ("forward", "train"):
        res = hla.linattn_forward(s["q"], s["k"], s["v"], gamma=s["gamma"], scale=s["scale"], lengths=s["lengths"],
                                  init_state=s["init"], return_final_state=c["state"])
        res = list(res) if c["state"] else [res]
        if op == "train":
            res += hla.linattn_backward(s["q"], s["k"], s["v"], s["dout"], gamma=s["gamma"], scale=s["scale"],
                                        lengths=s["lengths"], init_state=s["init"], dfinal_state=s["dfinal"])
        return res
    if op == "w4":
        return hla.w4_matvec(s["x"], s["qweight"], s["scales"], zeros=s["zeros"], bias=s["bias"])
    if op == "norm_train":
        h = hla.block_norm(s["x"], s["next_weight"], eps=EPS)
        return [h, *hla.block_norm_backward(s["x"], s["next_weight"], s["dh"], eps=EPS)]
    r, h = hla.block_join(s["x"], s["y"], s["post_weight"], gate=s["gate"], gate_act=c["act"], scale=s["scale"],
                          next_weight=s["next_weight"], eps=EPS)
    if op == "join":
        return [r, h]
    g = hla.block_join_backward(s["x"], s["y"], s["post_weight"], gate=s["gate"], gate_act=c["act"],
                                scale=s["scale"], next_weight=s["next_weight"], dr=s["dr"], dh=s["dh"], eps=EPS)
    return [r, h, g.dx, g.dy] + ([] if s["gate"] is None else [g.dgate]) + [g.dpost_weight, g.dscale, g.dnext_weight]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "step":
        return _plain_step(state)
    if op in ("forward", "train"):
        return _plain_linattn(state)
    if op == "w4":
        return _plain_w4(state)
    return _plain_rows(state)


# ---------------------------------------------------------------------------------------
# least work
# ---------------------------------------------------------------------------------------

def work(case):
    e, op = SIZE[case["dtype"]], case["op"]
    if op == "w4":
        M, N, K, g = (case[x] for x in ("M", "N", "K", "group"))
        return {"bytes": N * K / 2 + N * (K // g) * (e + case["zeros"]) + e * (M * K + M * N + case["bias"] * N),
                "flops": 2.0 * M * N * K}
    if op in ("forward", "train", "step"):
        H, Hk, d, dv = (case[x] for x in ("H", "Hk", "d", "dv"))
        if op == "step":
            N = case["N"]
            return {"bytes": N * (8.0 * Hk * d * dv + e * (H * (d + dv) + Hk * (d + dv))),
                    "flops": N * (2.0 * Hk + 2.0 * H) * d * dv}
        rows = case["B"] * case["n"]
        qo, kv, st = e * H * (d + dv), e * Hk * (d + dv), 4.0 * case["B"] * Hk * d * dv * case["state"]
        nbytes = rows * (qo + kv) + 2 * st
        flops = rows * (2.0 * Hk + 2.0 * H) * d * dv
        if op == "train":
            nbytes += rows * (2 * kv + qo + e * H * d) + 3 * st
            # two states (forward and reverse), and three outputs read from them
            flops += rows * (2.0 * Hk + 2.0 * H + 2.0 * H + 4.0 * Hk) * d * dv
        return {"bytes": nbytes, "flops": flops}
    rows, D = case["rows"], case["D"]
    full = {"full": D, "row": 1, "none": 0}[case["gate"]]
    if op == "norm_train":
        return {"bytes": e * rows * D * 5.0, "flops": 12.0 * rows * D}
    nbytes = e * rows * (4.0 * D + full)
    if op == "join":
        return {"bytes": nbytes, "flops": 12.0 * rows * D}
    return {"bytes": nbytes + e * rows * (6.0 * D + 2 * full), "flops": 40.0 * rows * D}


# ---------------------------------------------------------------------------------------
# exact values, in 64 bits from the definitions (token by token)
# ---------------------------------------------------------------------------------------

def _exact_linattn(s):
    c = s["case"]
    B, H, Hk, n, d, dv = (c[x] for x in ("B", "H", "Hk", "n", "d", "dv"))
    rep, dev = H // Hk, s["q"].device
    g = s["gamma"].double().reshape(1, Hk, 1, 1)
    q = s["q"].double().reshape(B, Hk, rep, n, d)
    k, v = s["k"].double(), s["v"].double()
    lengths = [n] * B if s["lengths"] is None else s["lengths"].tolist()
    live = torch.zeros(n, B, 1, 1, 1, dtype=torch.bool, device=dev)
    for b in range(B):
        live[:lengths[b], b] = True
    P = torch.zeros(B, Hk, d, dv, dtype=torch.float64, device=dev)
    if s["init"] is not None:
        P += s["init"].double()
    train = c["op"] == "train"
    do = s["dout"].double().reshape(B, Hk, rep, n, dv) if train else None
    o = torch.zeros(B, Hk, rep, n, dv, dtype=torch.float64, device=dev)
    dq = torch.zeros(B, Hk, rep, n, d, dtype=torch.float64, device=dev) if train else None
    for t in range(max(lengths)):
        P = torch.where(live[t], g * P + k[:, :, t, :, None] * v[:, :, t, None, :], P)
        o[:, :, :, t] = torch.where(live[t], s["scale"] * (q[:, :, :, t] @ P), 0.0)
        if train:
            dq[:, :, :, t] = torch.where(live[t], s["scale"] * (do[:, :, :, t] @ P.transpose(-1, -2)), 0.0)
    res = [o.reshape(B, H, n, dv)]
    if c["state"]:
        res.append(P)
    if not train:
        return res
    R = torch.zeros(B, Hk, d, dv, dtype=torch.float64, device=dev)  # gradient of the state after token t
    if s["dfinal"] is not None:
        R += s["dfinal"].double()
    dk, dvv = torch.zeros_like(k), torch.zeros_like(v)
    for t in range(max(lengths) - 1, -1, -1):
        at = R + s["scale"] * (q[:, :, :, t].transpose(-1, -2) @ do[:, :, :, t])
        dk[:, :, t] = torch.where(live[t, :, :, 0], (at @ v[:, :, t, :, None])[..., 0], 0.0)
        dvv[:, :, t] = torch.where(live[t, :, :, 0], (k[:, :, t, None, :] @ at)[..., 0, :], 0.0)
        R = torch.where(live[t], g * at, R)
    res += [dq.reshape(B, H, n, d), dk, dvv]
    return res + [R] if s["init"] is not None else res


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("forward", "train"):
        return _exact_linattn(s)
    if op == "step":
        rep = case["H"] // case["Hk"]
        P = (s["state"].double() * s["gamma"].double()[None, :, None, None]
             + torch.einsum("nhd,nhe->nhde", s["k"].double(), s["v"].double()))
        o = torch.einsum("nhrd,nhde->nhre", s["q"].double().unflatten(1, (case["Hk"], rep)), P)
        return [s["scale"] * o.flatten(1, 2), P]
    if op == "w4":
        low, high = (s["qweight"] % 16).double(), (s["qweight"] // 16).double()
        each = case["group"] // 2
        z = 8.0 if s["zeros"] is None else s["zeros"].double().repeat_interleave(each, 1)
        sc = s["scales"].double().repeat_interleave(each, 1)
        x = s["x"].double()
        y = x[:, 0::2] @ ((low - z) * sc).T + x[:, 1::2] @ ((high - z) * sc).T
        return y if s["bias"] is None else y + s["bias"].double()
    # rows: the forward in 64 bits, the gradients by differentiation of it
    names = ["x", "next_weight"] if op == "norm_train" else ["x", "y", "gate", "post_weight", "scale", "next_weight"]
    p = {k: s[k].double().requires_grad_() for k in names if s[k] is not None}

    def norm(t):
        return t / torch.sqrt(t.square().sum(-1, keepdim=True) / t.shape[-1] + EPS)

    r = p["x"]
    if op != "norm_train":
        a = 1.0
        if "gate" in p:
            a = torch.sigmoid(p["gate"])
            a = a if case["act"] == "sigmoid" else a * p["gate"]
        r = r + p["scale"] * (a * (norm(p["y"]) * p["post_weight"]))
    h = norm(r) * p["next_weight"]
    if op == "join":
        return [r.detach(), h.detach()]
    total = (h * s["dh"].double()).sum()
    if op != "norm_train":
        total = total + (r * s["dr"].double()).sum()
    grads = torch.autograd.grad(total, [p[k] for k in names if k in p])
    return ([] if op == "norm_train" else [r.detach()]) + [h.detach(), *grads]
