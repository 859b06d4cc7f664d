"""Layer norm on the GPU against the float64 oracle.

Tolerances: a mean and a variance of D values are sums in float32, good to 2^-24 sqrt(D) and about 4 2^-24 relative with the
roundings of the elements; a value is centred, scaled and shifted with a rounding each.  1e-5 of the largest output
covers D = 8192, and sums over up to 40000 rows, which are added in partial sums of a few hundred.  A mean far from zero
costs its own rounding, 2^-24 of it, against the spread.  A bfloat16 output is rounded once.

dx = inv (g - mean(g) - nx mean(g nx)) is a difference of three terms, each at most max|g| sqrt(D) and rounded to 2^-24 of
itself; in rows of two values nx is (1, -1) but for eps, so that they cancel to 1e-4 of themselves.  An error is
therefore held against the largest term, inv max|g| of the row (found at D = 2, where all of dx is what the terms leave)."""
import numpy as np
import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from oracle import ssm_oracle as O

from .ssm_cases import BF, F32, close, f64

pytestmark = pytest.mark.gpu


def make(shape, dtype, seed=0, mean=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    D = shape[-1]
    return ((mean + 2 * rand(*shape)).to(dtype), (1 + 0.3 * rand(D)).to(dtype), (0.2 * rand(D)).to(dtype), rand(*shape).to(dtype))


def check(x, w, b, do, eps=1e-5, tol=1e-5):
    close(hla.layer_norm(x, w, bias=b, eps=eps), O.layer_norm(f64(x), f64(w), f64(b) if b is not None else None, eps), "out", tol)
    x64, g64 = f64(x), f64(do) * f64(w)
    terms = (np.abs(g64).max(-1, keepdims=True) / np.sqrt(x64.var(-1, keepdims=True) + eps)) if x.numel() else 0.0
    for name, got, want in zip(("dx", "dweight", "dbias"), hla.layer_norm_backward(x, w, do, eps=eps),
                               O.layer_norm_backward(f64(x), f64(w), f64(do), eps)):
        assert got.dtype == (x.dtype if name == "dx" else F32)
        close(got, want, name, tol, terms if name == "dx" else 0.0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows, D", [(1, 1), (3, 2), (5, 7), (100, 8), (64, 33), (9, 64), (300, 100), (17, 255), (33, 256), (12, 513),
                                     (40, 999), (1000, 1024), (7, 2047), (77, 2048), (9, 2050), (5, 4096), (6, 5001), (3, 8192)])
def test_sizes(dtype, rows, D):
    x, w, b, do = make((rows, D), dtype, seed=D)
    check(x, w, b, do)
    check(x, w, None, do)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_rows(dtype):
    check(*make((40000, 40), dtype))


def test_rows_far_from_zero():
    """A mean of 1000 beside a spread of 2: off by 1000 2^-24, 3e-5 of the spread, where a difference of sums would have lost 8
    bits of the variance more."""
    check(*make((50, 500), F32, mean=1000.0), tol=1e-4)


def test_constant_rows():
    x = torch.full((4, 96), 3.0, device="cuda")
    w, b = torch.ones(96, device="cuda"), torch.full((96,), 0.25, device="cuda")
    assert torch.equal(hla.layer_norm(x, w, bias=b), torch.full_like(x, 0.25))
    dx, dw, db = hla.layer_norm_backward(x, w, torch.ones_like(x))
    assert not dx.any() and not dw.any() and torch.equal(db, torch.full_like(db, 4.0))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_leading_dimensions_strides_and_in_place(dtype):
    x, w, b, do = make((3, 5, 96), dtype)
    want, grads = hla.layer_norm(x, w, bias=b), hla.layer_norm_backward(x, w, do)
    assert want.shape == x.shape and grads[0].shape == x.shape
    flat = hla.layer_norm(x.view(15, 96), w, bias=b)
    assert torch.equal(want.view(15, 96), flat)
    for off in (0, 1, 8):
        wide = torch.empty(15, 200, dtype=dtype, device="cuda")
        v = wide[:, off:off + 96]
        v.copy_(x.view(15, 96))
        assert torch.allclose(hla.layer_norm(v, w, bias=b).float(), flat.float(), rtol=2 ** -7, atol=1e-6)
        close(hla.layer_norm_backward(v, w, do.view(15, 96))[0], f64(grads[0]).reshape(15, 96), "dx", 2 ** -8 if dtype == BF else 1e-5)
    y = x.clone()
    assert hla.layer_norm(y, w, bias=b, out=y) is y and torch.equal(y, want)


@pytest.mark.parametrize("D", [64, 2048, 4096])
def test_a_bad_row_stays_alone(D):
    x, w, b, do = make((20, D), BF)
    want, dx = hla.layer_norm(x, w, bias=b), hla.layer_norm_backward(x, w, do)[0]
    x[7, 3] = float("nan")
    x[11, 0] = float("inf")
    got, gx = hla.layer_norm(x, w, bias=b), hla.layer_norm_backward(x, w, do)[0]
    rest = [i for i in range(20) if i not in (7, 11)]
    assert torch.equal(got[rest], want[rest]) and torch.equal(gx[rest], dx[rest])
    assert got[7].isnan().all() and gx[7].isnan().all()


def test_no_rows():
    x, w, b, do = make((0, 64), F32)
    assert hla.layer_norm(x, w, bias=b).shape == (0, 64)
    dx, dw, db = hla.layer_norm_backward(x, w, do)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_captured():
    x, w, b, do = make((500, 256), BF)
    x2 = make((500, 256), BF, seed=3)[0]
    s = x.clone()
    hla.layer_norm_backward(s, w, do)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = hla.layer_norm(s, w, bias=b)
        grads = hla.layer_norm_backward(s, w, do)
    for v in (x2, x):
        s.copy_(v)
        graph.replay()
        want = (hla.layer_norm(v, w, bias=b), *hla.layer_norm_backward(v, w, do))
        graph.replay()
        for u, t in zip((y, *grads), want):
            assert torch.equal(u, t)
