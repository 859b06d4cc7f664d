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


# 160 or 192 state heads on 152 SMs: one segment of 6 to 11 chunks each
LONG_SEGMENTS = [
    # B, Hk, queries a key head, n, d, dv, ragged, state, gamma
    (1, 160, 1, 1300, 64, 64, False, False, (0.9, 0.9995)),
    (3, 64, 1, 1150, 64, 64, True, True, (0.05, 0.9)),
    (3, 64, 3, 700, 64, 64, True, True, (0.3, 0.999)),
    (2, 80, 4, 650, 32, 64, True, False, (0.9, 0.999)),
    (1, 160, 1, 900, 128, 128, False, True, (0.05, 0.9995)),
    (3, 64, 1, 1150, 128, 128, True, True, (0.9, 0.9995)),
    (3, 64, 2, 700, 128, 128, True, True, (0.3, 0.999)),
    (3, 56, 3, 650, 128, 64, True, False, (0.9, 0.999)),
    (2, 80, 1, 800, 16, 128, True, True, None),
]


@pytest.mark.parametrize("B, Hk, rep, n, d, dv, ragged, state, gamma", LONG_SEGMENTS)
def test_long_segments(B, Hk, rep, n, d, dv, ragged, state, gamma):
    x = draw(B, Hk * rep, Hk, n, d, dv, BF, seed=n + d, ragged=ragged, state=state, gamma=gamma)
    run_sampled(x, 0.2, BF, [0, Hk // 2, Hk - 1], states=state)


# Few heads: several segments of 3 to 8 chunks, joined by the output pass (up to sixteen segments and 512 KB of
# states) or by the scan
@pytest.mark.parametrize("B, Hk, rep, n, d, ragged", [
    (1, 40, 1, 3000, 64, False),    # 3 segments of 8 chunks, joined
    (4, 10, 2, 3000, 64, True),
    (1, 6, 1, 8000, 64, False),     # 22 segments of 3 chunks, scanned
    (2, 3, 3, 8000, 64, True),
    (1, 10, 1, 5000, 128, False),   # 14 segments of 3 chunks, scanned
    (2, 20, 2, 2900, 128, True),    # 3 segments of 8 chunks, joined
])
def test_several_segments_of_several_chunks(B, Hk, rep, n, d, ragged):
    x = draw(B, Hk * rep, Hk, n, d, d, BF, seed=n + Hk, tokens_first=True, ragged=ragged, state=True, gamma=(0.4, 0.9995))
    run_sampled(x, 0.2, BF, [0, Hk - 1], states=True)


@pytest.mark.parametrize("B, Hk, rep, n, d, dv, ragged", [(3, 64, 1, 700, 64, 64, True), (3, 64, 3, 333, 32, 128, True),
                                                          (1, 20, 2, 2000, 128, 64, False)])
def test_float32_over_many_chunks(B, Hk, rep, n, d, dv, ragged):
    x = draw(B, Hk * rep, Hk, n, d, dv, F32, seed=n, ragged=ragged, state=True, gamma=(0.3, 0.9995))
    run_sampled(x, 0.2, F32, [0, Hk // 2, Hk - 1])


@pytest.mark.parametrize("dtype, chunk", [(BF, 128), (F32, 64)])
def test_a_bad_value_reaches_no_earlier_chunk_and_no_other_head(dtype, chunk):
    """A NaN or infinity in a valid row spreads to its chunk and onwards (backwards in the reverse passes), not further."""
    x = cuda(draw(2, 4, 2, 900, 64, 64, dtype, seed=71))
    kw = dict(gamma=x["gamma"])
    run = lambda c: (hla.linattn_forward(c["q"], c["k"], c["v"], **kw),  # noqa: E731
                     *hla.linattn_backward(c["q"], c["k"], c["v"], c["dout"], **kw))
    clean = run(x)
    for name, row, bad in (("v", 700, float("nan")), ("k", 530, float("inf")), ("q", 400, float("-inf")),
                           ("dout", 300, float("nan"))):
        c = dict(x)
        c[name] = x[name].clone()
        c[name][1, 0, row] = bad
        got = run(c)
        lo, hi = row // chunk * chunk, (row // chunk + 1) * chunk
        for a, b in zip(clean, got):
            assert torch.equal(a[0], b[0])                      # the other sequence
            assert torch.equal(a[1, -1], b[1, -1])              # the other key head, and its queries
        for i in (0, 1):                                        # out and dq look back
            assert torch.equal(clean[i][1, :, :lo], got[i][1, :, :lo]), name
        for i in (2, 3):                                        # dk and dv look ahead
            assert torch.equal(clean[i][1, :, hi:], got[i][1, :, hi:]), name
        touched = {"v": (0, 1, 2), "k": (0, 1, 3), "q": (0, 2, 3), "dout": (1, 2, 3)}[name]
        assert all(not torch.isfinite(got[i][1]).all() for i in touched), name
