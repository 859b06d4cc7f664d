"""The operators around a layer on tensors whose offsets pass 32 bits, in elements or in bytes: the far end gives what
the same rows or heads give by themselves."""
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


@pytest.mark.parametrize("tokens_first", [False, True])
def test_linear_attention(tokens_first):
    B, H, n, d = 3, 48, 117000, 128  # 2.2e9 elements, 4.3 GB a tensor
    make = lambda s: (randn(B, n, H, d, seed=s).transpose(1, 2) if tokens_first else randn(B, H, n, d, seed=s))  # noqa: E731
    q, k, v = make(1), make(2), make(3)
    assert q.numel() > 2 ** 31
    gamma = torch.full((H,), 0.99, device="cuda")
    lengths = torch.tensor([n, n - 1000, n - 77], dtype=torch.int32, device="cuda")
    o, fin = hla.linattn_forward(q, k, v, gamma=gamma, scale=0.1, lengths=lengths, return_final_state=True)
    hla.check_status()
    for b, h in ((2, 47), (0, 0), (1, 24)):
        one = lambda t: t[b:b + 1, h:h + 1].contiguous()  # noqa: E731, B023
        w, wf = hla.linattn_forward(one(q), one(k), one(v), gamma=gamma[:1], scale=0.1, lengths=lengths[b:b + 1],
                                    return_final_state=True)
        # the segments differ, and with them the rounding of the carried states: two half steps of bf16 each side
        assert (o[b, h].double() - w[0, 0].double()).norm() <= 2.0 ** -7 * w.double().norm()
        assert (fin[b, h].double() - wf[0, 0].double()).norm() <= 2.0 ** -18 * wf.double().norm()
        L = int(lengths[b])
        assert not o[b, h, L:].any() and o[b, h, L - 1].any()


def test_step():
    N, H, d = 4200, 32, 128  # 2.2e9 state elements, 8.8 GB
    state = randn(N, H, d, d, dtype=F32)
    assert state.numel() > 2 ** 31
    q, k, v = (randn(N, H, d, seed=s) for s in (1, 2, 3))
    last = state[-1:].clone()
    o = hla.linattn_decode_step(state, q, k, v, gamma=0.9, scale=0.1)
    w = hla.linattn_decode_step(last, q[-1:], k[-1:], v[-1:], gamma=0.9, scale=0.1)
    assert torch.equal(o[-1:], w) and torch.equal(state[-1:], last)


@pytest.mark.parametrize("D, rows", [(2048, 1_060_000), (2051, 1_060_000)])
def test_join_and_gradients(D, rows):
    x, y, z, dr = (randn(rows, D, seed=s) for s in range(4))
    assert x.numel() > 2 ** 31
    pw, sc, nw = (randn(D, seed=s) for s in (7, 8, 9))
    kw = dict(scale=sc, next_weight=nw, gate_act="silu")
    tail = slice(rows - 40, rows)
    r, h = hla.block_join(x, y, pw, gate=z, **kw)
    wr, wh = hla.block_join(x[tail], y[tail], pw, gate=z[tail], **kw)
    assert torch.equal(r[tail], wr) and torch.equal(h[tail], wh)
    del r, h
    g = hla.block_join_backward(x, y, pw, gate=z, dr=dr, dh=dr, **kw)
    w = hla.block_join_backward(x[tail], y[tail], pw, gate=z[tail], dr=dr[tail], dh=dr[tail], **kw)
    for name in ("dx", "dy", "dgate"):
        assert torch.equal(getattr(g, name)[tail], getattr(w, name)), name


@pytest.mark.parametrize("dtype", [BF, F32])
def test_products(dtype):
    N, K, group = 530_001, 8192, 64  # 2.2e9 bytes of weights
    w = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8)
    assert w.numel() > 2 ** 31
    x, s = randn(3, K, dtype=dtype), randn(N, K // group, dtype=dtype, seed=1)
    tail = slice(N - 33, N)
    assert torch.equal(hla.w4_matvec(x, w, s)[:, tail], hla.w4_matvec(x, w[tail].clone(), s[tail].clone()))
