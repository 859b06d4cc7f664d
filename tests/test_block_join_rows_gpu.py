"""The block norms on the GPU at enough rows for several rounds of every CTA, so that the ring's slots and the sums
over rows are used again: sub-warps of 8 and of 32, pairs, single elements (held and not), the 256-thread shape,
one and two vectors above 2048.

Tolerances are those of test_block_join_gpu.py, but for the gradient of a row's gate.  That is act'(z) times a sum, and
act' = s (t p + e), with s = sigmoid(z), t = 1 - s (SiLU: p = z, e = 1; sigmoid: p = 1, e = 0), is itself a sum whose
terms cancel, wholly at the SiLU's minimum (z = -1.278): its error is counted against s ((1 + s) |p| + e).
"""
import numpy as np
import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from oracle import mixer_oracle as O

from .helpers import np64
from .test_block_join_gpu import BF, F32, close, close_sum, draw, terms, test_norm_and_gradients

pytestmark = pytest.mark.gpu

MANY = [(45001, 7), (30011, 24), (9001, 96), (6007, 33), (2003, 439), (2003, 999), (1999, 1002), (2500, 2048), (777, 2050),
        (777, 2051), (503, 5001), (480, 8192)]
norm_of = test_norm_and_gradients
del test_norm_and_gradients  # collected where it stands


def slope_terms(z, act):
    s = 1.0 / (1.0 + np.exp(-z))
    return s * ((1 + s) * np.abs(z) + 1) if act == "silu" else s * (1 + s)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, D", MANY)
@pytest.mark.parametrize("gate, act", [("full", "sigmoid"), ("row", "silu"), ("none", "sigmoid")])
def test_join_and_gradients(dtype, rows, D, gate, act):
    x = draw(rows, D, dtype, gate, seed=D)
    c = {k: None if t is None else t.cuda() for k, t in x.items()}
    n = {k: None if t is None else np64(t) for k, t in x.items()}
    kw = dict(gate=c["gate"], gate_act=act, scale=c["scale"], next_weight=c["nw"], eps=1e-5)
    r, h = hla.block_join(c["x"], c["y"], c["pw"], **kw)
    g = hla.block_join_backward(c["x"], c["y"], c["pw"], dr=c["dr"], dh=c["dh"], **kw)
    wr, wh = O.block_join(n["x"], n["y"], n["pw"], n["gate"], act, n["scale"], n["nw"], 1e-5)
    w = O.block_join_backward(n["x"], n["y"], n["pw"], n["gate"], act, n["scale"], n["nw"], n["dr"], n["dh"], 1e-5)
    t = terms(n, n["gate"], act, 1e-5)
    close(r, wr, dtype, "r", t["r"])
    close(h, wh, dtype, "h", t["h"])
    close(g.dx, w["dx"], dtype, "dx", t["dx"])
    close(g.dy, w["dy"], dtype, "dy", t["dy"])
    if gate == "full":
        close(g.dgate, w["dgate"], dtype, "dgate", t["dgate"])
    elif gate == "row":
        slope = np.abs(O._act(n["gate"], act)[1])
        a = (t["dgate"] / slope).sum(-1, keepdims=True) * slope_terms(n["gate"], act)
        lim = (2.0 ** -8 if dtype == BF else 2.0 ** -24) * np.abs(w["dgate"]) + 2.0 ** -24 * 128 * a
        assert (np.abs(np64(g.dgate.cpu()) - w["dgate"]) <= lim).all()
    for name in ("dpost_weight", "dscale", "dnext_weight"):
        close_sum(getattr(g, name), w[name], rows, name)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, D", MANY)
def test_norm_and_gradients_of_many_rows(dtype, rows, D):
    norm_of(dtype, rows, D)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, D", [(2003, 439), (2500, 512), (777, 2051)])
def test_strided_rows_of_many_rounds(dtype, rows, D):
    """Rows at odd distances and addresses give the bits of packed ones that take the same vectors."""
    x = draw(rows, D, dtype, seed=D + 1)
    c = {k: t.cuda() for k, t in x.items()}
    wide = torch.zeros((rows, 3, D + 1), dtype=dtype, device="cuda")
    flat = {k: torch.zeros(rows * D + 1, dtype=dtype, device="cuda")[1:].view(rows, D).copy_(c[k]) for k in ("x", "y", "gate", "dr", "dh")}
    for i, k in enumerate(("x", "y", "gate")):
        wide[:, i, 1:] = c[k]
    kw = dict(scale=c["scale"], next_weight=c["nw"])
    got = [*hla.block_join(*(wide[:, i, 1:] for i in (0, 1)), c["pw"], gate=wide[:, 2, 1:], **kw),
           *hla.block_join_backward(*(wide[:, i, 1:] for i in (0, 1)), c["pw"], gate=wide[:, 2, 1:], dr=flat["dr"], dh=flat["dh"], **kw)]
    want = [*hla.block_join(flat["x"], flat["y"], c["pw"], gate=flat["gate"], **kw),
            *hla.block_join_backward(flat["x"], flat["y"], c["pw"], gate=flat["gate"], dr=flat["dr"], dh=flat["dh"], **kw)]
    for a, b in zip(got, want):
        assert torch.equal(a, b)
