"""The norms before and after a block with its gate and residual scale, on the GPU against the
float64 oracle.

Tolerances.  Every output is computed in float32 from the exact inputs and rounded once: half a step of
its type (bf16 2^-8, float32 2^-24 relative) plus float32 arithmetic.  The latter: a row statistic is a sum
of D squares by a tree, off by a few 2^-24 relative, and every value is a sum of two or three terms (they
may cancel, for one: at D = 1 a norm's gradient is nearly 0); 2^-24 * 64 of the absolute terms, plus as much of
the row's scale of them for the statistics they share, covers it.  Weight gradients are float32 sums over
the rows: 2^-24 (32 + 2 sqrt(rows)) relative in norm.
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


def draw(rows, D, dtype, gate="full", seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = {"x": 2 * r(rows, D), "y": r(rows, D), "gate": None if gate == "none" else r(rows, D if gate == "full" else 1),
         "pw": 1 + 0.3 * r(D), "scale": 0.5 + 0.2 * r(D), "nw": 1 + 0.3 * r(D), "dr": r(rows, D), "dh": r(rows, D)}
    return {k: None if t is None else t.to(dtype) for k, t in x.items()}


def terms(n, gate, act, eps):
    """Sums of absolute terms of r, h, dx, dy, dgate."""
    a, slope = (np.ones(1), None) if gate is None else O._act(gate, act)
    ny, inv = O._norm(n["y"], eps)
    t = {"r": np.abs(n["x"]) + np.abs(n["scale"] * a * ny * n["pw"])}
    r = n["x"] + n["scale"] * a * ny * n["pw"]
    nr, inv_r = O._norm(r, eps)
    t["h"] = np.abs(n["nw"]) * inv_r * t["r"]
    dn = np.abs(n["dh"] * n["nw"])
    t["dx"] = np.abs(n["dr"]) + inv_r * (dn + np.abs(nr) * (dn * np.abs(nr)).mean(-1, keepdims=True)) \
        * (1 + t["r"] / np.maximum(np.abs(r), 1e-3 * t["r"]))
    dm = t["dx"] * np.abs(n["scale"] * a * n["pw"])
    t["dy"] = inv * (dm + np.abs(ny) * (dm * np.abs(ny)).mean(-1, keepdims=True))
    if gate is not None:
        t["dgate"] = t["dx"] * np.abs(n["scale"] * ny * n["pw"] * slope)
    return t


def close(got, want, dtype, what, scale=None):
    got, want = np64(got.cpu()), np.asarray(want)
    assert got.shape == want.shape, what
    if not want.size:
        return
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    scale = np.abs(want) if scale is None else scale
    lim = half * np.abs(want) + 2.0 ** -24 * 64 * (scale + np.sqrt((scale * scale).mean(-1, keepdims=True))) + 1e-30
    bad = np.abs(got - want) / lim
    assert (bad <= 1).all(), (what, float(bad.max()))


def close_sum(got, want, rows, what):
    got = np64(got.cpu())
    assert got.shape == want.shape, what
    n = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= 2.0 ** -24 * (32 + 2 * math.sqrt(rows)) * n * 4 + 1e-30, what


SIZES = [(1, 1), (3, 5), (2, 16), (9, 24), (7, 100), (5, 255), (4, 256), (6, 257), (3, 999), (2, 2048), (3, 2050),
         (2, 2056), (2, 4095), (2, 4096), (3, 5000), (2, 8191), (2, 8192)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, D", SIZES)
@pytest.mark.parametrize("gate, act", [("full", "silu"), ("row", "sigmoid"), ("none", "sigmoid")])
def test_join_and_gradients(dtype, rows, D, gate, act):
    x = draw(rows, D, dtype, gate, seed=D)
    c = {k: None if t is None else t.cuda() for k, t in x.items()}
    n = {k: None if t is None else np64(t) for k, t in x.items()}
    r, h = hla.block_join(c["x"], c["y"], c["pw"], gate=c["gate"], gate_act=act, scale=c["scale"], next_weight=c["nw"],
                          eps=1e-5)
    wr, wh = O.block_join(n["x"], n["y"], n["pw"], n["gate"], act, n["scale"], n["nw"], 1e-5)
    t = terms(n, n["gate"], act, 1e-5)
    close(r, wr, dtype, "r", t["r"])
    close(h, wh, dtype, "h", t["h"])
    g = hla.block_join_backward(c["x"], c["y"], c["pw"], gate=c["gate"], gate_act=act, scale=c["scale"],
                                next_weight=c["nw"], dr=c["dr"], dh=c["dh"], eps=1e-5)
    w = O.block_join_backward(n["x"], n["y"], n["pw"], n["gate"], act, n["scale"], n["nw"], n["dr"], n["dh"], 1e-5)
    close(g.dx, w["dx"], dtype, "dx", t["dx"])
    close(g.dy, w["dy"], dtype, "dy", t["dy"])
    if gate == "full":
        close(g.dgate, w["dgate"], dtype, "dgate", t["dgate"])
    elif gate == "row":  # a sum over the row: against the sum of its absolute terms
        a = t["dgate"].sum(-1, keepdims=True)
        lim = (2.0 ** -8 if dtype == BF else 2.0 ** -24) * np.abs(w["dgate"]) + 2.0 ** -24 * 128 * a
        assert (np.abs(np64(g.dgate.cpu()) - w["dgate"]) <= lim).all()
    else:
        assert g.dgate is None
    for name in ("dpost_weight", "dscale", "dnext_weight"):
        assert getattr(g, name).dtype == F32
        close_sum(getattr(g, name), w[name], rows, name)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, D", [(1, 1), (40, 16), (700, 64), (3, 999), (2000, 256), (1300, 2048), (9, 8192)])
def test_norm_and_gradients(dtype, rows, D):
    x = draw(rows, D, dtype, seed=rows)
    h = hla.block_norm(x["x"].cuda(), x["nw"].cuda(), eps=1e-6)
    close(h, O.block_norm(np64(x["x"]), np64(x["nw"]), 1e-6), dtype, "h")
    dx, dw = hla.block_norm_backward(x["x"].cuda(), x["nw"].cuda(), x["dh"].cuda(), eps=1e-6)
    wx, ww = O.block_norm_backward(np64(x["x"]), np64(x["nw"]), np64(x["dh"]), 1e-6)
    nx, inv = O._norm(np64(x["x"]), 1e-6)
    dn = np.abs(np64(x["dh"]) * np64(x["nw"]))
    close(dx, wx, dtype, "dx", inv * (dn + np.abs(nx) * (dn * np.abs(nx)).mean(-1, keepdims=True)))
    close_sum(dw, ww, rows, "dw")


def test_parts_left_out():
    x = draw(6, 320, BF, seed=9)
    c = {k: t.cuda() for k, t in x.items()}
    n = {k: np64(t) for k, t in x.items()}
    r, h = hla.block_join(c["x"], c["y"], c["pw"])
    assert h is None
    big = np.full(c["x"].shape, 16.0)  # every term here is a few units
    close(r, O.block_join(n["x"], n["y"], n["pw"])[0], BF, "r", big)
    g = hla.block_join_backward(c["x"], c["y"], c["pw"], dr=c["dr"])
    w = O.block_join_backward(n["x"], n["y"], n["pw"], dr=n["dr"])
    close(g.dx, w["dx"], BF, "dx", big)
    close(g.dy, w["dy"], BF, "dy", big)
    assert g.dscale is None and g.dnext_weight is None and g.dgate is None
    g = hla.block_join_backward(c["x"], c["y"], c["pw"], gate=c["gate"], next_weight=c["nw"], dh=c["dh"])
    w = O.block_join_backward(n["x"], n["y"], n["pw"], n["gate"], nw=n["nw"], dh=n["dh"])
    for k in ("dx", "dy", "dgate"):
        close(getattr(g, k), w[k], BF, k, big)


def test_rows_of_zeros_and_strided_rows():
    x = draw(5, 64, F32, seed=10)
    x["y"][2] = 0
    x["x"][2] = 0
    wide = torch.zeros((5, 3, 64), device="cuda")
    for i, k in enumerate(("x", "y", "gate")):
        wide[:, i] = x[k].cuda()
    c = {k: t.cuda() for k, t in x.items()}
    a = hla.block_join(wide[:, 0], wide[:, 1], c["pw"], gate=wide[:, 2], scale=c["scale"], next_weight=c["nw"])
    b = hla.block_join(c["x"], c["y"], c["pw"], gate=c["gate"], scale=c["scale"], next_weight=c["nw"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert not a[0][2].any() and torch.isfinite(a[1]).all()
    g = hla.block_join_backward(wide[:, 0], wide[:, 1], c["pw"], gate=wide[:, 2], scale=c["scale"], next_weight=c["nw"],
                                dr=c["dr"], dh=c["dh"])
    assert all(torch.isfinite(t).all() for t in g)
    # leading dimensions, and none
    three = hla.block_join(c["x"].view(5, 1, 64), c["y"].view(5, 1, 64), c["pw"])[0]
    one = hla.block_join(c["x"][0], c["y"][0], c["pw"])[0]
    assert three.shape == (5, 1, 64) and torch.equal(three[0, 0], one)
    # rows at odd addresses take the single-element kernels
    flat = torch.randn(5 * 65 + 1, device="cuda")
    odd = flat[1:1 + 5 * 65].view(5, 65)[:, :64]
    assert torch.equal(hla.block_norm(odd, c["nw"]), hla.block_norm(odd.contiguous(), c["nw"])) or \
        (hla.block_norm(odd, c["nw"]) - hla.block_norm(odd.contiguous(), c["nw"])).abs().max() < 1e-5


def test_closed_gates_and_empty():
    x = draw(3, 128, BF, seed=12)
    c = {k: t.cuda() for k, t in x.items()}
    gate = torch.full((3, 1), float("-inf"), dtype=BF, device="cuda")
    r, _ = hla.block_join(c["x"], c["y"], c["pw"], gate=gate)
    assert torch.equal(r, c["x"])
    lowest = torch.full((3, 128), torch.finfo(BF).min, dtype=BF, device="cuda")
    r, _ = hla.block_join(c["x"], c["y"], c["pw"], gate=lowest, gate_act="silu")
    assert torch.equal(r, c["x"])
    e = torch.zeros((0, 128), dtype=BF, device="cuda")
    r, h = hla.block_join(e, e, c["pw"], next_weight=c["nw"])
    assert r.shape == h.shape == (0, 128)
    g = hla.block_join_backward(e, e, c["pw"], next_weight=c["nw"], dh=e)
    assert g.dx.shape == (0, 128) and not g.dpost_weight.any() and not g.dnext_weight.any()


def test_same_bits_every_time():
    x = draw(3000, 512, BF, seed=13)
    c = {k: t.cuda() for k, t in x.items()}
    kw = dict(gate=c["gate"], scale=c["scale"], next_weight=c["nw"], dr=c["dr"], dh=c["dh"])
    a = hla.block_join_backward(c["x"], c["y"], c["pw"], **kw)
    b = hla.block_join_backward(c["x"], c["y"], c["pw"], **kw)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, D", [(3000, 256), (2003, 439), (45001, 7), (600, 4096)])
def test_norm_in_place(dtype, rows, D):
    x = torch.randn((rows, D), device="cuda").to(dtype)
    w = torch.randn(D, device="cuda").to(dtype)
    want = hla.block_norm(x, w)
    assert hla.block_norm(x, w, out=x) is x and torch.equal(x, want)
    both = torch.randn((rows + 1, D), device="cuda").to(dtype)
    with pytest.raises(hla.HLA2Error):
        hla.block_norm(both[1:], w, out=both[:-1])
    with pytest.raises(hla.HLA2Error):
        hla.block_norm(x, x[1], out=x)


def test_refusals():
    x = torch.zeros((2, 64), device="cuda")
    w = torch.zeros(64, device="cuda")
    with pytest.raises(TypeError):
        hla.block_join(x, x.to(BF), w)
    with pytest.raises(ValueError):
        hla.block_join(x, x, w, gate=x, gate_act="relu")
    with pytest.raises(ValueError):
        hla.block_join(x, x, torch.zeros(63, device="cuda"))
    with pytest.raises(ValueError):
        hla.block_join(x, x, w, gate=torch.zeros((2, 2), device="cuda"))
    with pytest.raises(ValueError):
        hla.block_join_backward(x, x, w)
    with pytest.raises(hla.HLA2Error):
        hla.block_norm(torch.zeros((1, 8193), device="cuda"), torch.zeros(8193, device="cuda"))
