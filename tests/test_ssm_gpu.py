"""The selective scan on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from oracle import ssm_oracle as O

from .ssm_cases import BF, F32, close, f64, make_ssm

pytestmark = pytest.mark.gpu


def oracle_args(c, **kw):
    d = {k: f64(v) for k, v in c.items()}
    d.update(kw)
    return d


def check_forward(c, lengths=None, **kw):
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, fin = hla.ssm_forward(**c, lengths=lens, return_final_state=True, **kw)
    want, wfin = O.ssm_forward(**oracle_args(c, lengths=lengths, **kw))
    assert out.dtype == c["x"].dtype and fin.dtype == F32
    close(out, want, "out")
    close(fin, wfin, "final state")
    if lengths is not None:
        for s, m in enumerate(lengths):
            assert (out[s, max(m, 0):] == 0).all()
    return out, fin


def check_backward(c, lengths=None, dfinal=True, seed=1, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dout = torch.randn(c["x"].shape, generator=g, device="cuda").to(c["x"].dtype)
    B, n, D = c["x"].shape
    dfin = torch.randn((B, D, c["a"].shape[1]), generator=g, device="cuda") if dfinal else None
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got = hla.ssm_backward(dout=dout, dfinal_state=dfin, lengths=lens, **c, **kw)
    want = O.ssm_backward(**oracle_args(c, dout=f64(dout), dfinal_state=f64(dfin), lengths=lengths, **kw))
    for name in got._fields:
        t = getattr(got, name)
        source = {"dskip": "skip", "dgate": "gate", "ddt_bias": "dt_bias", "dinit_state": "init_state"}.get(name)
        if source and c[source] is None:
            assert t is None
        else:
            close(t, want[name], name)
    return got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 100])
def test_forward(dtype, N, n):
    check_forward(make_ssm(2, n, 72, N, dtype=dtype, seed=n))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D, G", [(1, 1), (7, 1), (63, 1), (65, 1), (128, 2), (66, 2), (12, 4), (200, 1)])
def test_channels_and_groups(dtype, D, G):
    c = make_ssm(2, 37, D, 16, G, dtype=dtype, seed=D)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("n", [1, 4, 16, 33, 100])
def test_backward(dtype, N, n):
    check_backward(make_ssm(2, n, 72, N, dtype=dtype, seed=n))


@pytest.mark.parametrize("have", ["", "gate", "skip", "bias", "state"])
@pytest.mark.parametrize("softplus", [True, False])
def test_optional_inputs(have, softplus):
    c = make_ssm(2, 40, 24, 16, **{k: k == have for k in ("gate", "skip", "bias", "state")})
    if not softplus:
        c["dt"] = c["dt"].abs() * 0.1
        if c["dt_bias"] is not None:  # about -5, for the softplus: as a step it would grow past 64 bits, e^80 a token
            c["dt_bias"] = c["dt_bias"].abs() * 0.01
    check_forward(c, dt_softplus=softplus)
    check_backward(c, dt_softplus=softplus, dfinal=have == "state")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lengths", [[0, 40, 17], [40, -3, 1], [99, 16, 0]])
def test_lengths(dtype, lengths):
    c = make_ssm(3, 40, 24, 16, dtype=dtype, seed=5)
    for s, m in enumerate(lengths):  # padding holds anything
        for k in ("x", "dt", "b", "c", "gate"):
            c[k][s, max(m, 0):] = float("nan") if s % 2 else float("inf")
    out, fin = check_forward(c, lengths)
    g = check_backward(c, lengths)
    for t in (g.dx, g.ddt, g.dgate, g.db, g.dc):
        for s, m in enumerate(lengths):
            assert (t[s, max(m, 0):] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [700, 1500])
def test_segments(dtype, n):
    """Few channels and many tokens: the sequence is cut into segments."""
    c = make_ssm(1, n, 24, 16, dtype=dtype, seed=n)
    assert hla.lib().hla2_ssm_workspace_bytes  # the plan is the library's own
    check_forward(c)
    check_forward(c, [n // 3])
    check_backward(c)
    check_backward(c, [n - n // 3])


def test_fast_and_slow_steps():
    """Steps from next to nothing, where softplus is e^x, to ones that forget at once."""
    c = make_ssm(1, 64, 32, 16, dt_scale=8.0, seed=9)
    c["dt"][:, :, 0] = -30.0
    c["dt"][:, :, 1] = 60.0
    c["dt"][:, :, 2] = -200.0
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("B, D, G", [(1, 64, 1), (3, 50, 2), (300, 96, 1)])
def test_step_follows_the_forward(dtype, N, B, D, G):
    c = make_ssm(B, 3, D, N, G, dtype=dtype, seed=B)
    state = c.pop("init_state")
    want, wst = O.ssm_forward(**oracle_args(c, init_state=f64(state)))
    for t in range(3):
        one = {k: c[k][:, t] if k in ("x", "dt", "b", "c", "gate") else c[k] for k in c}
        close(hla.ssm_decode_step(state, **one), want[:, t], f"token {t}")
    close(state, wst, "state")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides(dtype):
    """Parts of a projection, tokens before sequences, odd offsets and a broadcast: the values of contiguous copies."""
    B, n, D, G, N = 2, 50, 40, 2, 16
    c = make_ssm(B, n, D, N, G, dtype=dtype, seed=3)
    want = hla.ssm_forward(**c, return_final_state=True)
    dout = torch.randn(B, n, D, device="cuda").to(dtype)
    grads = hla.ssm_backward(dout=dout, **c)
    xz = torch.empty(B, n, 2 * D + 1, device="cuda", dtype=dtype)
    odd = torch.empty(n, B, 3 + D + 2 * G * N, device="cuda", dtype=dtype).transpose(0, 1)
    v = dict(c)
    v["x"], v["gate"], v["dt"] = xz[..., :D], xz[..., D + 1:], odd[..., 3:3 + D]
    v["b"] = odd[..., 3 + D:3 + D + G * N].unflatten(-1, (G, N))
    v["c"] = odd[..., 3 + D + G * N:].unflatten(-1, (G, N))
    for k in ("x", "gate", "dt", "b", "c"):
        v[k].copy_(c[k])
    got = hla.ssm_forward(**v, return_final_state=True)
    dv = torch.empty(B, D, n, device="cuda", dtype=dtype).transpose(1, 2)  # copied: the last dimension is strided
    dv.copy_(dout)
    for u, w in zip((*got, *hla.ssm_backward(dout=dv, **v)), (*want, *grads)):
        assert torch.equal(u, w)
    # one gate row for all tokens, one b for all sequences
    v["gate"] = c["gate"][:, :1].expand(B, n, D)
    v["b"] = c["b"][:1].expand(B, n, G, N)
    same = {**c, "gate": v["gate"].contiguous(), "b": v["b"].contiguous()}
    for u, w in zip(hla.ssm_backward(dout=dout, **v), hla.ssm_backward(dout=dout, **same)):
        assert torch.equal(u, w)


def test_three_dimensional_b_and_c():
    c = make_ssm(2, 20, 24, 8)
    flat = {**c, "b": c["b"][:, :, 0], "c": c["c"][:, :, 0]}
    assert torch.equal(hla.ssm_forward(**c), hla.ssm_forward(**flat))
    dout = torch.randn(2, 20, 24, device="cuda")
    u, v = hla.ssm_backward(dout=dout, **c), hla.ssm_backward(dout=dout, **flat)
    assert v.db.shape == flat["b"].shape and torch.equal(u.db[:, :, 0], v.db) and torch.equal(u.dc[:, :, 0], v.dc)


def test_empty():
    c = make_ssm(2, 0, 24, 16)
    out, fin = hla.ssm_forward(**c, return_final_state=True)
    assert out.shape == (2, 0, 24) and torch.equal(fin, c["init_state"])
    dfin = torch.randn_like(fin)
    g = hla.ssm_backward(dout=out, dfinal_state=dfin, **c)
    assert torch.equal(g.dinit_state, dfin) and not g.da.any() and not g.dskip.any() and not g.ddt_bias.any()
    c = make_ssm(0, 5, 24, 16)
    assert hla.ssm_forward(**c).shape == (0, 5, 24)
    g = hla.ssm_backward(dout=c["x"], **c)
    assert g.db.shape == (0, 5, 1, 16) and not g.da.any() and not g.ddt_bias.any()


def test_gradients_are_differences():
    """The kernels' own forward, differenced in float32 along a few directions: the truncation is of second order and the
    rounding of the loss, about 1e-6 of its terms, is divided by the step 1e-2."""
    c = make_ssm(1, 30, 16, 8, seed=11)
    dout = torch.randn(1, 30, 16, device="cuda")
    g = hla.ssm_backward(dout=dout, **c)

    def loss(d):
        return (hla.ssm_forward(**d).double() * dout.double()).sum().item()

    eps = 1e-2
    for name in ("x", "dt", "a", "b", "c", "skip", "gate", "dt_bias", "init_state"):
        u = torch.randn_like(c[name])
        u = u / u.norm()
        diff = (loss({**c, name: c[name] + eps * u}) - loss({**c, name: c[name] - eps * u})) / (2 * eps)
        want = (getattr(g, "d" + name).double() * u.double()).sum().item()
        terms = (hla.ssm_forward(**c).abs().double() * dout.abs().double()).sum().item()
        assert abs(diff - want) <= 1e-6 * terms / eps + 1e-3 * abs(want) + 1e-3, (name, diff, want)


def test_repeatable_and_on_another_stream():
    c = make_ssm(2, 600, 64, 16, dtype=BF)
    dout = torch.randn_like(c["x"])
    want = (*hla.ssm_forward(**c, return_final_state=True), *hla.ssm_backward(dout=dout, **c))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = (*hla.ssm_forward(**c, return_final_state=True), *hla.ssm_backward(dout=dout, **c))
    side.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u, v)


def test_captured():
    """Forward, backward and step in one graph, replayed on other values, with eager calls of the same sizes between."""
    c = make_ssm(1, 900, 64, 16, dtype=BF)
    d = make_ssm(1, 900, 64, 16, dtype=BF, seed=7)
    dout = torch.randn_like(c["x"])
    static = {k: v.clone() for k, v in c.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hla.ssm_forward(**static)
        hla.ssm_backward(dout=dout, **static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, fin = hla.ssm_forward(**static, return_final_state=True)
        grads = hla.ssm_backward(dout=dout, **static)
    for case in (d, c):
        for k, v in static.items():
            v.copy_(case[k])
        graph.replay()
        want = (*hla.ssm_forward(**case, return_final_state=True), *hla.ssm_backward(dout=dout, **case))
        graph.replay()
        for u, v in zip((out, fin, *grads), want):
            assert torch.equal(u, v)


def test_many_short_sequences():
    """More sequences than a grid has rows."""
    c = make_ssm(70_000, 1, 4, 8, gate=False)
    out, fin = check_forward(c)
    check_backward(c)
    state = c["init_state"].clone()
    one = {k: c[k][:, 0] for k in ("x", "dt", "b", "c")}
    y = hla.ssm_decode_step(state, a=c["a"], skip=c["skip"], dt_bias=c["dt_bias"], **one)
    close(y, f64(out[:, 0]), "step", 1e-5)
    close(state, f64(fin), "state", 1e-5)
    # and more than four to a CTA's sequences in one launch
    c = make_ssm(4 * 65_535 + 3, 1, 64, 8, gate=False, state=False, seed=2)
    one = {k: c[k][:, 0] for k in ("x", "dt", "b", "c")}
    state = torch.zeros(4 * 65_535 + 3, 64, 8, device="cuda")
    y = hla.ssm_decode_step(state, a=c["a"], skip=c["skip"], dt_bias=c["dt_bias"], **one)
    tail = {k: v[-5:] for k, v in one.items()}
    last = torch.zeros(5, 64, 8, device="cuda")
    w = hla.ssm_decode_step(last, a=c["a"], skip=c["skip"], dt_bias=c["dt_bias"], **tail)
    close(y[-5:], f64(w), "step", 1e-5)
    close(state[-5:], f64(last), "state", 1e-5)


@pytest.mark.parametrize("n, step, steps_of", [(8192, 1e-3, "scan"), (8192, 1e-5, "scan"), (2048, 1e-3, "tokens")])
def test_slow_decays_keep_their_rate(n, step, steps_of):
    """A state that nothing enters decays by exp(a sum of the steps).  Each token's rounded decay is within 2^-23 of it at
    worst, but what counts over thousands of tokens is the mean: it has to stay below 4e-9, an eighth of the decay's half
    step of 2^-25.  Of the roundings to nearest, of the decays and the products, each token adds at most 2^-24.  They
    change sign from channel to channel, so that the mean of 64 channels x 8 states has 2^-24 sqrt(2 n / 512), below
    4e-9 n from n = 100 on."""
    D, N = 64, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    dt = step * (0.5 + torch.rand((1, n, D), generator=g, device="cuda"))
    a = -0.05 - 0.1 * torch.rand((D, N), generator=g, device="cuda")
    h0 = 1.0 + torch.rand((1, D, N), generator=g, device="cuda")
    x, b = torch.zeros((1, n, D), device="cuda"), torch.zeros((1, n, 1, N), device="cuda")
    if steps_of == "scan":
        fin = hla.ssm_forward(x, dt, a, b, b, dt_softplus=False, init_state=h0, return_final_state=True)[1]
    else:
        fin = h0.clone()
        for t in range(n):
            hla.ssm_decode_step(fin, x[:, t], dt[:, t], a, b[:, t], b[:, t], dt_softplus=False)
    want = h0.double() * torch.exp(dt.double().sum(1)[..., None] * a.double())
    assert abs(((fin.double() - want) / want).mean().item()) <= 4e-9 * n
    # no decay: a product with 1
    none = hla.ssm_forward(x, dt, 0 * a, b, b, dt_softplus=False, init_state=h0, return_final_state=True)[1]
    assert torch.equal(none, h0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D, G", [(12, 1), (68, 1), (204, 3)])
def test_rows_of_four_channels_alignment(dtype, D, G):
    """Widths and addresses that are multiples of four elements, not of eight."""
    c = make_ssm(2, 37, D, 16, G, dtype=dtype, seed=D)
    wide = torch.zeros((2, 37, 2 * D + 4), dtype=dtype, device="cuda")
    wide[..., 4:4 + D], wide[..., 4 + D:] = c["x"], c["gate"]
    c["x"], c["gate"] = wide[..., 4:4 + D], wide[..., 4 + D:]
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_channels(dtype):
    """Without channels the sums over a group's channels are zeros."""
    c = make_ssm(2, 5, 0, 16, dtype=dtype)
    out, fin = hla.ssm_forward(**c, return_final_state=True)
    assert out.shape == (2, 5, 0) and fin.shape == (2, 0, 16)
    dirty = [torch.full((2, 5, 1, 16), float("nan"), device="cuda", dtype=dtype) for _ in range(64)]
    del dirty  # what the allocator hands out next
    g = hla.ssm_backward(dout=out, **c)
    assert g.db.shape == g.dc.shape == (2, 5, 1, 16) and g.da.shape == (0, 16) and g.dx.shape == (2, 5, 0)
    assert (g.db == 0).all() and (g.dc == 0).all()


def small_steps(n, dtype=F32):
    """Channels with steps softplus(v) of about e^-30 to e^-3, and positive values throughout, so that no sum cancels; each channel is a
    group of its own, so that b's and c's gradients are its alone."""
    v = torch.linspace(-30.0, -3.0, 28, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: 0.9 + 0.2 * torch.rand(s, generator=g, device="cuda")  # noqa: E731
    D, N = len(v), 8
    c = dict(x=rand(1, n, D), dt=v.expand(1, n, D).clone(), b=rand(1, n, D, N), c=rand(1, n, D, N))
    c = {k: t.to(dtype) for k, t in c.items()}
    c["a"] = -0.1 * torch.arange(1, N + 1, device="cuda", dtype=F32).repeat(D, 1)
    return c, rand(1, n, D).to(dtype), v.double().cpu().numpy()


def relative(got, want, tol, what):
    """Every element within tol of its own value; tol over the channels, the dimension of size 28."""
    g = f64(got)
    assert g.shape == want.shape and (want != 0).all(), what
    shape = [1] * g.ndim
    shape[list(g.shape).index(len(tol))] = len(tol)
    err = np.abs(g / want - 1.0) / tol.reshape(shape)
    assert (err <= 1.0).all(), f"{what}: {err.max():.3g} of the tolerance at {np.unravel_index(err.argmax(), err.shape)}"


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("softplus", [True, False])
def test_small_steps_keep_their_relative_accuracy(n, softplus):
    """Nothing here but terms that are proportional to a step, each compared with its own value.

    e^-|v| by the unit is good to 2^-22; its argument |v| log2 e is rounded twice, to half a step of the product and of the constant,
    together 1.25 2^-24 |v| of the result.  A reciprocal (2^-23), the polynomial (1e-8) and six roundings give the step
    (4 + 2 + 1 + 6) 2^-24; delta x, its product with b or c, a decay (4 and 1) for each of up to three tokens, and eight terms' sums
    another 2 + 15 + 8.  With the decays, whose share of a gradient of the step is of the other sign and at most 2 tokens x 0.8 x
    softplus(-3) x (1.1 / 0.9)^2 = 0.12 of it, 1.3 times that: 50 + 1.7 |v|.  da is a product of two steps: twice."""
    c, dout, v = small_steps(n)
    if not softplus:
        c["dt"] = torch.exp(c["dt"])
    tol = (50 + 1.7 * np.abs(v)) * 2.0 ** -24
    out, fin = hla.ssm_forward(**c, dt_softplus=softplus, return_final_state=True)
    args = oracle_args(c, dt_softplus=softplus)
    want, wfin = O.ssm_forward(**args)
    relative(out, want, tol, "out")
    relative(fin, wfin, tol, "final state")
    got, w = hla.ssm_backward(dout=dout, dt_softplus=softplus, **c), O.ssm_backward(dout=f64(dout), **args)
    for name in ("dx", "ddt", "db", "dc"):
        relative(getattr(got, name), w[name], tol, name)
    if n > 1:  # one token from a zero state has no decay to differentiate
        relative(got.da, w["da"], 2 * tol, "da")
    state = torch.zeros_like(fin)
    for t in range(n):
        y = hla.ssm_decode_step(state, c["x"][:, t], c["dt"][:, t], c["a"], c["b"][:, t], c["c"][:, t], dt_softplus=softplus)
        relative(y, want[:, t], tol, f"step {t}")
    relative(state, wfin, tol, "state of the steps")


def test_small_steps_in_bfloat16():
    """States are float32 whatever the tensors' type: the bounds above, and one rounding more for what is bfloat16."""
    c, dout, v = small_steps(3, BF)
    tol = (50 + 1.7 * np.abs(f64(c["dt"])[0, 0])) * 2.0 ** -24
    out, fin = hla.ssm_forward(**c, return_final_state=True)
    want, wfin = O.ssm_forward(**oracle_args(c))
    relative(fin, wfin, tol, "final state")
    relative(out, want, tol + 2.0 ** -8, "out")
    got, w = hla.ssm_backward(dout=dout, **c), O.ssm_backward(dout=f64(dout), **oracle_args(c))
    relative(got.da, w["da"], 2 * tol, "da")
    for name in ("dx", "ddt", "db", "dc"):
        relative(getattr(got, name), w[name], tol + 2.0 ** -8, name)


@pytest.mark.parametrize("N", [16, 64])
def test_gradients_of_fast_states(N):
    """The decays' gradients and the states fall off with the state's index, -1 .. -N; each index is held against its own
    size (the bound of `close` is per state: a rounding of each token that it remembers)."""
    c = make_ssm(2, 100, 72, N, seed=21)
    dout = torch.randn_like(c["x"])
    out, fin = hla.ssm_forward(**c, return_final_state=True)
    wfin = O.ssm_forward(**oracle_args(c))[1]
    g, w = hla.ssm_backward(dout=dout, **c), O.ssm_backward(dout=f64(dout), **oracle_args(c))
    for k in range(N):
        close(fin[..., k], wfin[..., k], f"state {k}")
        close(g.da[:, k], w["da"][:, k], f"da {k}")
        close(g.dinit_state[..., k], w["dinit_state"][..., k], f"dinit {k}")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("n, lengths", [(5, None), (16, None), (37, [37, 20]), (700, [1, 699])])
def test_states_that_forget_at_once(dtype, N, n, lengths):
    """a = -inf (or so low that a log2 e is): the state is the last token's input alone.  The tokens that fill up a tile, with steps of
    zero, leave it as it is."""
    c = make_ssm(2, n, 40, N, dtype=dtype, seed=n)
    far = {**c, "a": c["a"].clone()}
    far["a"][3], far["a"][7, 1::2] = -1e30, -1e30  # finite, so that the oracle's gradients are
    out, fin = check_forward(far, lengths)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    dout, dfin = torch.randn_like(c["x"]), torch.randn_like(c["init_state"])
    grads = hla.ssm_backward(dout=dout, dfinal_state=dfin, lengths=lens, **far)
    if n < 100:
        check_backward(far, lengths)
    for low in (-float("inf"), torch.finfo(F32).min):
        v = {**c, "a": far["a"].masked_fill(far["a"] == -1e30, low)}
        got = hla.ssm_forward(**v, lengths=lens, return_final_state=True)
        assert torch.equal(got[0], out) and torch.equal(got[1], fin)
        for name, a, b in zip(grads._fields, hla.ssm_backward(dout=dout, dfinal_state=dfin, lengths=lens, **v), grads):
            assert torch.equal(a, b), name
        one = {k: v[k][:, 0] if k in ("x", "dt", "b", "c", "gate") else v[k] for k in v if k != "init_state"}
        s, t = c["init_state"].clone(), c["init_state"].clone()
        assert torch.equal(hla.ssm_decode_step(s, **one), hla.ssm_decode_step(t, **{**one, "a": far["a"]})) and torch.equal(s, t)
