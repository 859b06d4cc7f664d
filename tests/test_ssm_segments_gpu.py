"""The selective scan where the sequence is one segment of many marks, a few segments, or more than a CTA joins itself: the count of
segments is read from the workspace's size, so that each path is known to run."""
import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from chunked_scan_mixer_gb300.hla2 import _SSM_ARGS

from .ssm_cases import BF, F32, close, f64, make_ssm
from .test_ssm_gpu import check_backward, check_forward

pytestmark = pytest.mark.gpu
CHANNELS, TOKENS, JOIN = 64, 16, 32  # of a CTA, between marks, and segments that a CTA joins itself


def up(x):
    return (x + 255) // 256 * 256


def segments(c, backward):
    """Segments of the call's plan: the only count with the workspace's size."""
    B, n, D = c["x"].shape
    G, N = c["b"].shape[2:]
    dtype = 1 if c["x"].dtype == BF else 0
    size = hla.lib().hla2_ssm_workspace_bytes(_SSM_ARGS.pack(dtype, B, n, D, N, G, 1, *[0] * 24), int(backward))
    tiles, steps, found = G * -(-(D // G) // CHANNELS), -(-n // TOKENS), set()
    for each in range(1, steps + 1):
        nseg = -(-steps // each)
        slots, state, more = B * tiles * nseg, CHANNELS * N * 4, nseg > 1
        total = more * (up(slots * state) + up(slots * CHANNELS * 4))
        if backward:
            total += up(slots * each * state) + more * (up(slots * each * CHANNELS * 4) + up(slots * state))
            total += up(B * n * tiles * 2 * N * 4) + up(B * nseg * D * (N + 2) * 4)
        if total == size:
            found.add(nseg)
    assert len(found) == 1, (size, found)
    return found.pop()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_few_segments(dtype, N):
    """Joined by the CTAs themselves; two groups of an odd width, ragged."""
    c = make_ssm(2, 290, 2 * 33, N, 2, dtype=dtype, seed=N)
    assert 1 < segments(c, False) <= JOIN and 1 < segments(c, True) <= JOIN
    check_forward(c)
    check_backward(c)
    check_forward(c, [130, 283])
    check_backward(c, [130, 283])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("B, per", [(2, 33), (1, 68)])
def test_many_segments(dtype, N, B, per):
    """Joined by a scan of their own, forward and in reverse: more than one batch of 32; two groups of one tile or of two."""
    c = make_ssm(B, 1190, 2 * per, N, 2, dtype=dtype, seed=N)
    assert segments(c, False) > JOIN and segments(c, True) > JOIN
    check_forward(c)
    check_backward(c, [1190, 707][-B:])
    check_backward(c, [0, 1181][-B:], dfinal=False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("ragged", [False, True])
def test_one_segment_of_many_marks(dtype, N, ragged):
    """A call that fills the GPU by itself, against differentiation in float64.  The sums over 640 sequences are added as 64000 terms
    in partial sums, at most 2^-24 sqrt(64000) off: within the bound of `close`."""
    B, n, D = 640, 100, 64
    c = make_ssm(B, n, D, N, dtype=dtype, seed=N)
    assert segments(c, False) == segments(c, True) == 1
    g = torch.Generator(device="cuda").manual_seed(8)
    dout = torch.randn((B, n, D), generator=g, device="cuda").to(dtype)
    dfin = torch.randn((B, D, N), generator=g, device="cuda")
    lengths = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if ragged else None
    out, fin = hla.ssm_forward(**c, lengths=lengths, return_final_state=True)
    got = hla.ssm_backward(dout=dout, dfinal_state=dfin, lengths=lengths, **c)

    p = {k: v.double().requires_grad_() for k, v in c.items()}
    live = torch.arange(n, device="cuda")[None] < (torch.full((B,), n, device="cuda") if lengths is None else lengths)[:, None]
    h, ys = p["init_state"], []
    for t in range(n):
        delta = torch.nn.functional.softplus(p["dt"][:, t] + p["dt_bias"], threshold=1e9)
        after = torch.exp(delta[..., None] * p["a"]) * h + (delta * p["x"][:, t])[..., None] * p["b"][:, t]
        h = torch.where(live[:, t, None, None], after, h)
        y = (h * p["c"][:, t]).sum(-1) + p["skip"] * p["x"][:, t]
        ys.append(torch.where(live[:, t, None], y * torch.nn.functional.silu(p["gate"][:, t]), 0.0))
    want = torch.stack(ys, 1)
    names = ("x", "dt", "a", "b", "c", "skip", "gate", "dt_bias", "init_state")
    grads = torch.autograd.grad((want * dout.double()).sum() + (h * dfin.double()).sum(), [p[k] for k in names])
    close(out, f64(want), "out")
    close(fin, f64(h), "final state")
    for k, w in zip(names, grads):
        close(getattr(got, "d" + k), f64(w), "d" + k)
