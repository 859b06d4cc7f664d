"""A selective state space layer's operators on tensors whose offsets pass 32 bits, in elements or in bytes: the far end
gives what the same sequences or rows give by themselves."""
import pytest
import torch

import chunked_scan_mixer_gb300 as hla

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def randn(*shape, dtype=BF, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_scan():
    B, n, D, N = 3, 180_000, 4096, 8  # 2.2e9 elements, 4.4 GB a tensor
    x, dt, dout = randn(B, n, D, seed=1), randn(B, n, D, seed=2), randn(B, n, D, seed=3)
    assert x.numel() > 2 ** 31
    b, c = randn(B, n, N, seed=4), randn(B, n, N, seed=5)
    a = -torch.arange(1.0, N + 1, device="cuda").repeat(D, 1)
    kw = dict(dt_bias=torch.full((D,), -4.0, device="cuda"), skip=torch.ones(D, device="cuda"))
    lengths = torch.tensor([n, n - 1000, n - 77], dtype=torch.int32, device="cuda")
    out, fin = hla.ssm_forward(x, dt, a, b, c, lengths=lengths, return_final_state=True, **kw)
    one = lambda t: t[2:3]  # noqa: E731
    w, wf = hla.ssm_forward(one(x), one(dt), a, one(b), one(c), lengths=lengths[2:], return_final_state=True, **kw)
    # the segments differ, and with them the order of the float32 sums; a bfloat16 output may round the other way
    assert rel(out[2], w[0]) <= 2.0 ** -8 and rel(fin[2], wf[0]) <= 2.0 ** -18
    assert not out[2, n - 77:].any() and out[2, n - 78].any()
    del out, w
    g = hla.ssm_backward(x, dt, a, b, c, dout, lengths=lengths, **kw)
    v = hla.ssm_backward(one(x), one(dt), a, one(b), one(c), one(dout), lengths=lengths[2:], **kw)
    for name in ("dx", "ddt", "db", "dc"):
        assert rel(getattr(g, name)[2], getattr(v, name)[0]) <= 2.0 ** -8, name
        assert not getattr(g, name)[2, n - 77:].any()


def test_scan_step():
    B, D, N = 8400, 4096, 64  # 2.2e9 state elements, 8.8 GB
    state = randn(B, D, N, dtype=F32)
    assert state.numel() > 2 ** 31
    x, dt, b, c = randn(B, D, seed=1), randn(B, D, seed=2), randn(B, N, seed=3), randn(B, N, seed=4)
    a = -torch.arange(1.0, N + 1, device="cuda").repeat(D, 1)
    last = state[-1:].clone()
    out = hla.ssm_decode_step(state, x, dt, a, b, c)
    w = hla.ssm_decode_step(last, x[-1:], dt[-1:], a, b[-1:], c[-1:])
    assert rel(out[-1:], w) <= 2.0 ** -8 and rel(state[-1:], last) <= 2.0 ** -20  # four sequences a thread, and one


@pytest.mark.parametrize("D, n", [(4096, 180_000), (4099, 180_000)])
def test_convolution(D, n):
    x, dout, w = randn(3, n, D, seed=1), randn(3, n, D, seed=2), randn(D, 4, seed=3)
    assert x.numel() > 2 ** 31
    out = hla.short_conv_forward(x, w)
    tail = slice(n - 40, n)
    want = hla.short_conv_forward(x[2:, tail].contiguous(), w, init_state=x[2:, n - 43:n - 40].contiguous())
    assert torch.equal(out[2:, tail], want)
    del out
    g = hla.short_conv_backward(x, w, dout)
    v = hla.short_conv_backward(x[2:, tail].contiguous(), w, dout[2:, tail].contiguous(), init_state=x[2:, n - 43:n - 40].contiguous())
    assert torch.equal(g.dx[2:, tail], v.dx)


@pytest.mark.parametrize("D", [2048, 2051])
def test_norm(D):
    rows = 1_060_000
    x, do, w = randn(rows, D, seed=1), randn(rows, D, seed=2), randn(D, seed=3)
    assert x.numel() > 2 ** 31
    tail = slice(rows - 40, rows)
    # forty rows take another number of warps, and so another order of the sums: a bfloat16 value may round the other way
    assert rel(hla.layer_norm(x, w)[tail], hla.layer_norm(x[tail], w)) <= 2.0 ** -8
    assert rel(hla.layer_norm_backward(x, w, do)[0][tail], hla.layer_norm_backward(x[tail], w, do[tail])[0]) <= 2.0 ** -8
