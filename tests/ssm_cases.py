"""Inputs and comparisons of the tests of a selective state space layer's operators."""
import numpy as np
import torch

BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def make_ssm(B, n, D, N, G=1, dtype=F32, gate=True, skip=True, bias=True, state=True, seed=0, dt_scale=0.5):
    """Inputs of ssm_forward as such layers have them: steps from 0.001 to 0.1, decays -1 .. -N."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    dt0 = torch.exp(torch.rand(D, generator=g, device="cuda") * 4.6 - 6.9)
    c = dict(x=rand(B, n, D).to(dtype), dt=(dt_scale * rand(B, n, D)).to(dtype),
             a=-torch.arange(1, N + 1, device="cuda") * torch.exp(0.2 * rand(D, 1)),
             b=rand(B, n, G, N).to(dtype), c=rand(B, n, G, N).to(dtype))
    c["skip"] = 0.5 + rand(D) if skip else None
    c["gate"] = rand(B, n, D).to(dtype) if gate else None
    c["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0)) if bias else None
    c["init_state"] = rand(B, D, N) if state else None
    return c


def close(got, want, what="", f32_tol=1e-4, terms=0.0):
    """The arithmetic is float32: a state's error is at most the tokens that it remembers, a few hundred here, times the
    rounding of a decay, an input and a sum, 2^-21.5 together, so 1e-4 of the largest value; sums over channels and tokens
    are of that kind.  An output in bfloat16 is rounded once: 2^-8 of the value.  ``terms``: the size of the terms of
    outputs that are their difference, where it says more than that of the outputs."""
    g, want = f64(got), np.asarray(want)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    if want.size == 0:
        return
    top = np.abs(want).max()
    tol = f32_tol * np.maximum(top, terms) + 1e-30 + (2.0 ** -8 * np.abs(want) if got.dtype == BF else 0.0)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(g - want)):.3g} of {top:.3g}, " \
                          f"first at {np.argwhere(bad)[0].tolist()}"
