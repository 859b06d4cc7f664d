"""Products with 4-bit weights on the GPU against the float64 oracle.

Tolerances.  The products are exact; the float32 sums over K terms are off by at most
2^-24 (16 + 2 sqrt(K)) of the sum of absolute terms, element by element; then one rounding to the output's type
(bf16 2^-8, float32 2^-24, relative)."""
import math

import numpy as np
import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from oracle import mixer_oracle as O

from .helpers import np64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def draw(M, N, K, group, dtype, zeros=True, bias=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g).to(dtype)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = (0.01 + torch.rand((N, K // group), generator=g)).to(dtype)
    z = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8) if zeros else None
    b = torch.randn(N, generator=g).to(dtype) if bias else None
    return x, w, s, z, b


def check(x, w, s, z, b, dtype, y):
    n = lambda t: None if t is None else np64(t)  # noqa: E731
    zz = None if z is None else z.numpy()
    want = O.w4_matvec(n(x), w.numpy().astype(np.int64), n(s), zz, n(b))
    # |q - z| <= 15: the absolute terms
    big = O.w4_matvec(np.abs(n(x)), np.full(w.shape, 0xFF, dtype=np.int64), n(s), np.zeros(s.shape)) + np.abs(want)
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    lim = half * np.abs(want) + 2.0 ** -24 * (16 + 2 * math.sqrt(x.shape[1])) * big
    got = np64(y.cpu())
    assert got.shape == want.shape
    assert (np.abs(got - want) <= lim).all(), float((np.abs(got - want) / lim).max())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M, N, groups", [(1, 1, 1), (1, 16, 2), (1, 17, 7), (2, 100, 9), (3, 33, 16), (5, 50, 3), (8, 64, 5),
                                          (9, 31, 33), (11, 160, 8), (16, 47, 20), (1, 2000, 16)])
def test_shapes(dtype, group, M, N, groups):
    x, w, s, z, b = draw(M, N, group * groups, group, dtype, zeros=M % 2 == 1, bias=N % 2 == 0, seed=M + N)
    y = hla.w4_matvec(x.cuda(), w.cuda(), s.cuda(), zeros=None if z is None else z.cuda(),
                      bias=None if b is None else b.cuda())
    check(x, w, s, z, b, dtype, y)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_value_and_zero_point(dtype):
    """One nonzero x at a time reads a column back: exact values, scale 1."""
    K, N = 64, 256
    w = torch.arange(256, dtype=torch.uint8).reshape(N, 1).expand(N, K // 2).contiguous()
    s = torch.ones((N, 1), dtype=dtype)
    for zp in (0, 7, 15):
        z = torch.full((N, 1), zp, dtype=torch.uint8)
        for k in (0, 1, 5, 30, 33, 63):
            x = torch.zeros((1, K), dtype=dtype)
            x[0, k] = 1
            y = hla.w4_matvec(x.cuda(), w.cuda(), s.cuda(), zeros=z.cuda()).cpu().float()[0]
            want = (w[:, 0] // 16 if k % 2 else w[:, 0] % 16).float() - zp
            assert torch.equal(y, want)


def test_large_values_and_float32_digits():
    """float32 x keeps its 24 bits: a sum of two values that differ in the last ones."""
    K = 32
    x = torch.zeros((2, K))
    x[0, 0], x[0, 1] = 1.0 + 2.0 ** -23, -1.0
    x[1, 3] = 3.0e38
    w = torch.full((1, K // 2), 0x99, dtype=torch.uint8)  # q = 9, so q - 8 = 1
    y = hla.w4_matvec(x.cuda(), w.cuda(), torch.ones((1, 1)).cuda()).cpu()
    assert y[0, 0] == 2.0 ** -23 and y[1, 0] == x[1, 3]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 8, 12])
def test_weights_at_their_zero_point(dtype, group, M):
    """Nearly every weight is zero and x has a mean: the sums count against |q - z| |x| s, not against |q| or |x|."""
    K, N = 8192, 64
    g = torch.Generator().manual_seed(M + group)
    x = (1 + 0.5 * torch.randn((M, K), generator=g)).to(dtype)
    z = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8)
    q = z.repeat_interleave(group, 1)
    at = torch.randint(0, K, (N, 3), generator=g)
    q.scatter_(1, at, torch.randint(0, 16, (N, 3), generator=g, dtype=torch.uint8))
    w = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    s = (0.01 + torch.rand((N, K // group), generator=g)).to(dtype)
    n = [np64(x), w.numpy().astype(np.int64), np64(s), z.numpy()]
    want = O.w4_matvec(*n)
    terms = np.abs(n[0]) @ (np.abs(q.numpy().astype(np.float64) - z.repeat_interleave(group, 1).numpy())
                            * np.repeat(n[2], group, axis=1)).T
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    lim = half * np.abs(want) + 2.0 ** -24 * (16 + 2 * math.sqrt(K)) * terms
    y = np64(hla.w4_matvec(x.cuda(), w.cuda(), s.cuda(), zeros=z.cuda()).cpu())
    assert (np.abs(y - want) <= lim).all(), float((np.abs(y - want) / np.maximum(lim, 1e-300)).max())
    # without any zero point given, and all weights at 8: exactly nothing
    eights = torch.full((N, K // 2), 0x88, dtype=torch.uint8)
    assert not hla.w4_matvec(x.cuda(), eights.cuda(), s.cuda()).any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M", [1, 9])
def test_infinite_and_large_values(dtype, M):
    """An infinity goes to its outputs with the sign of its weight (NaN where that is zero), and to no other row;
    values whose products by 16 and more would pass float32 stay finite where the output is."""
    K, N, group = 256, 6, 64
    q = torch.full((N, K), 8, dtype=torch.uint8)
    q[0, 70], q[1, 70], q[2, 70] = 11, 3, 8
    q[3, 130], q[4, 131] = 9, 7
    w = q[:, 0::2] | (q[:, 1::2] << 4)
    s = torch.ones((N, K // group), dtype=dtype)
    x = torch.zeros((M, K), dtype=dtype)
    x[0, 70] = float("inf")
    y = hla.w4_matvec(x.cuda(), w.cuda(), s.cuda()).cpu().float()
    assert y[0, 0] == float("inf") and y[0, 1] == float("-inf") and y[0, 2:].isnan().all()
    assert not y[1:].any()
    x[0, 70] = 0
    x[0, 130] = x[0, 131] = torch.tensor(3.0e38, dtype=dtype)
    y = hla.w4_matvec(x.cuda(), w.cuda(), s.cuda()).cpu()
    assert y[0, 3] == x[0, 130] and y[0, 4] == -x[0, 131] and not y[0, [0, 1, 2, 5]].any()


def test_views_and_leading_dimensions():
    x, w, s, z, b = (t.cuda() for t in draw(6, 40, 256, 64, BF))
    want = hla.w4_matvec(x, w, s, zeros=z, bias=b)
    wide = torch.zeros((6, 300), dtype=BF, device="cuda")
    wide[:, :256] = x
    assert torch.equal(hla.w4_matvec(wide[:, :256], w, s, zeros=z, bias=b), want)  # rows of 600 bytes: copied
    wide = torch.zeros((6, 320), dtype=BF, device="cuda")
    wide[:, 8:264] = x
    assert torch.equal(hla.w4_matvec(wide[:, 8:264], w, s, zeros=z, bias=b), want)
    assert torch.equal(hla.w4_matvec(x.view(2, 3, 256), w, s, zeros=z, bias=b), want.view(2, 3, 40))
    assert torch.equal(hla.w4_matvec(x[2], w, s, zeros=z, bias=b), want[2])
    out = torch.empty((6, 40), dtype=BF, device="cuda")
    assert hla.w4_matvec(x, w, s, zeros=z, bias=b, out=out) is out and torch.equal(out, want)
    assert hla.w4_matvec(x[:0], w, s).shape == (0, 40)
    assert hla.w4_matvec(x, w[:0], s[:0]).shape == (6, 0)


def test_rows_do_not_touch_each_other():
    x, w, s, z, b = (t.cuda() for t in draw(5, 70, 512, 128, BF, seed=4))
    want = hla.w4_matvec(x, w, s, zeros=z, bias=b)
    x2 = x.clone()
    x2[3] = float("nan")
    got = hla.w4_matvec(x2, w, s, zeros=z, bias=b)
    assert torch.equal(got[[0, 1, 2, 4]], want[[0, 1, 2, 4]]) and got[3].isnan().all()
    for m in range(5):
        assert torch.equal(hla.w4_matvec(x[m], w, s, zeros=z, bias=b), want[m])


def test_refusals():
    x, w, s, z, b = (t.cuda() for t in draw(2, 8, 128, 64, BF))
    for bad in (lambda: hla.w4_matvec(x[:, :64], w, s), lambda: hla.w4_matvec(x, w, s[:, :0]),
                lambda: hla.w4_matvec(x, w, s, zeros=z[:, :1]), lambda: hla.w4_matvec(x, w, s, bias=b[:3]),
                lambda: hla.w4_matvec(x, w.to(torch.int32), s)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        hla.w4_matvec(x.float(), w, s)
    with pytest.raises(hla.HLA2Error):
        hla.w4_matvec(torch.zeros((17, 128), dtype=BF, device="cuda"), w, s)
    with pytest.raises(hla.HLA2Error):
        hla.w4_matvec(x, w, s.repeat(1, 4))  # groups of 16


def test_output_over_the_input_is_refused():
    x = torch.zeros((2, 128), dtype=BF, device="cuda")
    square = torch.randint(0, 256, (128, 64), device="cuda", dtype=torch.uint8)
    with pytest.raises(hla.HLA2Error):
        hla.w4_matvec(x, square, torch.ones((128, 2), dtype=BF, device="cuda"), out=x)  # other CTAs still read x
