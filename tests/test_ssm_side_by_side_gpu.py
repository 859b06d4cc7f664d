"""The C entry points on tensors that lie side by side in one buffer: what separate tensors give, and nothing beside them written."""
import ctypes

import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from chunked_scan_mixer_gb300.hla2 import Rows, View

from .ssm_cases import BF, F32, make_ssm
from .test_ssm_abi import ConvArgs, SsmArgs, SsmGradArgs

pytestmark = pytest.mark.gpu


def rows(t):
    return Rows(t.data_ptr(), *t.stride()[:2])


def view(t):
    return View(t.data_ptr(), t.stride(0), t.stride(2), t.stride(1))


def run(rc):
    assert rc == 0, hla.lib().hla2_last_error().decode()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D, G", [(64, 1), (66, 2), (200, 2)])
@pytest.mark.parametrize("n", [37, 900])
def test_scan(dtype, D, G, n):
    L, B, N = hla.lib(), 2, 16
    c = make_ssm(B, n, D, N, G, dtype=dtype, seed=D)
    dout = torch.randn(B, n, D, device="cuda").to(dtype)
    want_out, want_fin = hla.ssm_forward(**c, return_final_state=True)
    want = hla.ssm_backward(dout=dout, **c)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")

    def args(x):
        a = SsmArgs(1 if dtype == BF else 0, B, n, D, N, G, 1, rows(x), rows(c["dt"]), rows(c["gate"]), view(c["b"]), view(c["c"]),
                    *(c[k].data_ptr() for k in ("a", "skip", "dt_bias")), None, c["init_state"].data_ptr(), ws.data_ptr(), ws.numel())
        return ctypes.byref(a)

    stream = torch.cuda.current_stream().cuda_stream
    # the output beside the input
    buf = torch.full((B, n, 3 * D), 7.0, device="cuda", dtype=dtype)
    x, out, free = buf.split(D, -1)
    x.copy_(c["x"])
    fin = torch.empty_like(want_fin)
    run(L.hla2_ssm_forward(args(x), rows(out), fin.data_ptr(), stream))
    assert torch.equal(out, want_out) and torch.equal(fin, want_fin) and torch.equal(x, c["x"]) and (free == 7).all()
    # the gradients of a projection's halves and of its parts, as the projection's own gradients
    dxz = torch.full((B, n, 2 * D + 3), 7.0, device="cuda", dtype=dtype)
    dbc = torch.full((B, n, 2 * G * N), 7.0, device="cuda", dtype=dtype)
    dx, dgate, free = dxz.split((D, D, 3), -1)
    db, dc = (t.unflatten(-1, (G, N)) for t in dbc.split(G * N, -1))
    ddt, da, dinit = torch.empty_like(want.ddt), torch.empty_like(want.da), torch.empty_like(want.dinit_state)
    dskip, dbias = torch.empty_like(want.dskip), torch.empty_like(want.ddt_bias)
    g = SsmGradArgs(rows(dx), rows(ddt), rows(dgate), view(db), view(dc), *(t.data_ptr() for t in (da, dskip, dbias, dinit)))
    run(L.hla2_ssm_backward(args(c["x"]), rows(dout), None, ctypes.byref(g), stream))
    for t, w in zip((dx, ddt, da, db, dc, dskip, dgate, dbias, dinit), want):
        assert torch.equal(t, w)
    assert (free == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D", [64, 33])
def test_convolution(dtype, D):
    L, B, n, W = hla.lib(), 2, 45, 4
    x0, dout = (torch.randn(B, n, D, device="cuda").to(dtype) for _ in range(2))
    w = torch.randn(D, W, device="cuda").to(dtype)
    want, grads = hla.short_conv_forward(x0, w), hla.short_conv_backward(x0, w, dout)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    buf = torch.full((B, n, 4 * D), 7.0, device="cuda", dtype=dtype)
    x, out, dx, free = buf.split(D, -1)
    x.copy_(x0)
    a = ConvArgs(1 if dtype == BF else 0, B, n, D, W, 1, rows(x), w.data_ptr(), None, None, None, ws.data_ptr(), ws.numel())
    dw, stream = torch.empty_like(grads.dweight), torch.cuda.current_stream().cuda_stream
    run(L.hla2_short_conv_forward(ctypes.byref(a), rows(out), None, stream))
    run(L.hla2_short_conv_backward(ctypes.byref(a), rows(dout), None, rows(dx), dw.data_ptr(), None, None, stream))
    assert torch.equal(out, want) and torch.equal(dx, grads.dx) and torch.equal(x, x0) and (free == 7).all()
    assert torch.allclose(dw, grads.dweight, rtol=1e-5, atol=1e-4)  # another vector width may add the tokens in another order
    # a step, in and out of one buffer
    a.lengths = None
    one = torch.full((B, 2 * D), 7.0, device="cuda", dtype=dtype)
    one[:, :D] = x0[:, 0]
    s, t = (torch.randn(B, W - 1, D, device="cuda").to(dtype) for _ in range(2))
    t.copy_(s)
    a.x = Rows(one.data_ptr(), 2 * D, 0)
    run(L.hla2_short_conv_decode_step(ctypes.byref(a), s.data_ptr(), Rows(one[:, D:].data_ptr(), 2 * D, 0), stream))
    assert torch.equal(one[:, D:], hla.short_conv_decode_step(t, x0[:, 0], w)) and torch.equal(s, t)
    assert torch.equal(one[:, :D], x0[:, 0])
