"""Linear attention on the GPU where a segment has many chunks, so that slots, barriers and the state go round:
more heads than SMs (the plan then gives each one long segment), or a few long segments a head.

The float64 oracle runs on a sample of the heads; the tolerances are those of test_linattn_gpu.py.
"""
import numpy as np
import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from oracle import mixer_oracle as O

from .test_linattn_gpu import BF, F32, absolute, check, cuda, draw, n64

pytestmark = pytest.mark.gpu


def sampled(x, keys):
    """The key heads ``keys`` of every sequence, with their queries, in float64."""
    rep = x["q"].shape[1] // x["k"].shape[1]
    queries = [k * rep + r for k in keys for r in range(rep)]
    at = {"q": queries, "dout": queries, "k": keys, "v": keys, "init": keys, "dfinal": keys}
    z = {n: None if x[n] is None else n64(x[n][:, h]) for n, h in at.items()}
    z["gamma"] = None if x["gamma"] is None else n64(x["gamma"][keys])
    z["lengths"] = None if x["lengths"] is None else x["lengths"].numpy()
    return z, queries


def run_sampled(x, scale, dtype, keys, states=True):
    n, d, dv = x["q"].shape[2], x["q"].shape[3], x["v"].shape[3]
    rep = x["q"].shape[1] // x["k"].shape[1]
    c = cuda(x)
    kw = dict(gamma=c["gamma"], scale=scale, lengths=c["lengths"], init_state=c["init"])
    if states:
        o, fin = hla.linattn_forward(c["q"], c["k"], c["v"], return_final_state=True, **kw)
    else:
        o, fin = hla.linattn_forward(c["q"], c["k"], c["v"], **kw), None
    grads = hla.linattn_backward(c["q"], c["k"], c["v"], c["dout"], dfinal_state=c["dfinal"], **kw)
    hla.check_status()
    z, queries = sampled(x, keys)
    a = absolute(z)
    fwd = lambda s: O.linattn_forward(s["q"], s["k"], s["v"], s["gamma"], scale, s["lengths"], s["init"])  # noqa: E731
    bwd = lambda s: O.linattn_backward(s["q"], s["k"], s["v"], s["dout"], s["gamma"], scale, s["lengths"],  # noqa: E731
                                       s["init"], s["dfinal"])
    (wo, wP), (bo, _), want, bound = fwd(z), fwd(a), bwd(z), bwd(a)
    check(o[:, queries], wo, bo, dtype, n, max(d, dv), "out")
    if states:
        check(fin[:, keys], wP, None, F32, n, 1, "final state")
    for name, g, h, w, b in zip(("dq", "dk", "dv"), grads, (queries, keys, keys), want, bound):
        check(g[:, h], w, b, dtype, n * rep, max(d, dv), name)
    if x["init"] is not None:
        check(grads[3][:, keys], want[3], None, F32, n * rep, 1, "dinit")
    for b, L in enumerate([] if x["lengths"] is None else x["lengths"].tolist()):
        for t in (o, *grads[:3]):
            assert not t[b, :, max(0, min(n, L)):].any()


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("gamma", [(0.9, 0.9995), (0.1, 0.9)])
def test_two_queries_a_key_head_over_many_chunks(ragged, gamma):
    """At 64 dimensions the Gram product of a chunk's last query is issued before the state that enters the chunk
    is there."""
    x = draw(3, 128, 64, 1200, 64, 64, BF, seed=61, ragged=ragged, state=ragged, gamma=gamma)
    run_sampled(x, 0.125, BF, [0, 31, 63], states=ragged)
