"""Host-side checks of a selective state space layer's entry points (no GPU): bad arguments are refused with a message before
any launch, empty calls succeed, and the packed arguments have the header's layout.

Addresses are made up and never dereferenced: a call that passes the checks would be launched, so those are made only where
there is no device to launch on (-4)."""
import ctypes
import random

import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from chunked_scan_mixer_gb300.hla2 import _CONV_ARGS, _NORM_ARGS, _SSM_ARGS, _SSM_GRADS, Rows, View, _length_tensor

NO_GPU = not torch.cuda.is_available()
I, P, Q, Z = ctypes.c_int, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_size_t


@pytest.fixture(scope="module")
def L():
    return hla.lib()


class SsmArgs(ctypes.Structure):
    """hla2_ssm_args, field by field."""
    _fields_ = [(n, I) for n in ("dtype", "B", "n", "D", "N", "G", "softplus")] + [
        ("x", Rows), ("dt", Rows), ("gate", Rows), ("b", View), ("c", View), ("a", P), ("skip", P), ("dt_bias", P), ("lengths", P),
        ("init_state", P), ("workspace", P), ("workspace_bytes", Z)]


class SsmGradArgs(ctypes.Structure):
    """hla2_ssm_grads, field by field."""
    _fields_ = [("dx", Rows), ("ddt", Rows), ("dgate", Rows), ("db", View), ("dc", View), ("da", P), ("dskip", P), ("ddt_bias", P),
                ("dinit_state", P)]


class ConvArgs(ctypes.Structure):
    """hla2_conv_args, field by field."""
    _fields_ = [(n, I) for n in ("dtype", "B", "n", "D", "W", "silu")] + [
        ("x", Rows), ("weight", P), ("bias", P), ("lengths", P), ("init_state", P), ("workspace", P), ("workspace_bytes", Z)]


class NormArgs(ctypes.Structure):
    """hla2_norm_args, field by field."""
    _fields_ = [("dtype", I), ("rows", Q), ("D", I), ("eps", ctypes.c_float), ("x", P), ("x_stride", Q), ("weight", P), ("bias", P)]


def test_packed_argument_blocks_have_the_c_layout():
    r = lambda k: Rows(k, k + 1, k + 2)  # noqa: E731
    v = lambda k: View(k, k + 1, k + 2, k + 3)  # noqa: E731
    a = SsmArgs(1, 2, 3, 4, 16, 2, 1, r(10), r(13), r(16), v(19), v(23), *range(27, 34))
    assert _SSM_ARGS.pack(1, 2, 3, 4, 16, 2, 1, *range(10, 34)) == bytes(a)
    g = SsmGradArgs(r(1), r(4), r(7), v(10), v(14), 18, 19, 20, 21)
    assert _SSM_GRADS.pack(*range(1, 22)) == bytes(g)
    c = ConvArgs(1, 2, 3, 4, 4, 1, r(7), *range(10, 16))
    assert _CONV_ARGS.pack(1, 2, 3, 4, 4, 1, *range(7, 16)) == bytes(c)
    n = NormArgs(1, 3, 64, 0.25, 4, 64, 5, 6)
    assert _NORM_ARGS.pack(1, 3, 64, 0.25, 4, 64, 5, 6) == bytes(n)


B, N, D, G = 2, 5000, 48, 2  # tokens enough for segments, which need a workspace
SIZE = B * N * D * 2         # bytes of x
BC = B * N * G * 16 * 2      # of b
ST = B * D * 16 * 4          # of a state


def rows(p, n=N, d=D):
    return Rows(p, n * d, d)


def states(p, n=N):
    return View(p, n * G * 16, 16, G * 16)


def ssm(**kw):
    c = dict(dtype=1, B=B, n=N, D=D, N=16, G=G, softplus=1, x=rows(0x10000000), dt=rows(0x11000000), gate=rows(0x12000000),
             b=states(0x13000000), c=states(0x14000000), a=0x15000000, skip=0x15100000, dt_bias=0x15200000, lengths=0x15300000,
             init_state=0x15400000, workspace=None, workspace_bytes=0)
    c.update(kw)
    return SsmArgs(*c.values())


BAD_SSM = [dict(dtype=2), dict(B=-1), dict(n=-1), dict(D=-1), dict(N=12), dict(N=128), dict(N=0), dict(G=0), dict(G=5), dict(softplus=2),
           dict(x=rows(None)), dict(dt=rows(None)), dict(b=states(None)), dict(c=states(None)), dict(a=None), dict(x=rows(0x10000001)),
           dict(gate=rows(0x12000001)), dict(x=Rows(0x10000000, -1, D)), dict(dt=Rows(0x11000000, N * D, -D)),
           dict(b=View(0x13000000, 0, -16, 0)), dict(a=0x15000004), dict(init_state=0x15400008), dict(skip=0x15100002),
           dict(dt_bias=0x15200001), dict(lengths=0x15300002)]


def forward(L, a, out=rows(0x20000000), fin=0x21000000):
    return L.hla2_ssm_forward(ctypes.byref(a), out, fin, None)


def grads(**kw):
    c = dict(dx=rows(0x30000000), ddt=rows(0x31000000), dgate=rows(0x32000000), db=states(0x33000000), dc=states(0x34000000), da=0x35000000,
             dskip=0x35100000, ddt_bias=0x35200000, dinit_state=0x35300000)
    c.update(kw)
    return SsmGradArgs(*c.values())


def backward(L, a, g=None, dout=rows(0x22000000), dfin=0x23000000):
    return L.hla2_ssm_backward(ctypes.byref(a), dout, dfin, ctypes.byref(grads() if g is None else g), None)


@pytest.mark.parametrize("kw", BAD_SSM)
def test_scan_refuses(L, kw):
    for call in (forward, backward):
        assert call(L, ssm(**kw)) == -1, call
        assert L.hla2_last_error().decode()
    step = ssm(**{"lengths": None, "init_state": None, **kw})
    token_stride = "dt" in kw and kw["dt"].sn < 0  # a step does not look at it
    if "lengths" not in kw and "init_state" not in kw and "n" not in kw and not token_stride:
        assert L.hla2_ssm_decode_step(ctypes.byref(step), 0x21000000, rows(0x20000000), None) == -1
    if kw.keys() & {"dtype", "B", "n", "D", "N", "G", "softplus"}:
        assert L.hla2_ssm_workspace_bytes(ctypes.byref(ssm(**kw)), 1) == Z(-1).value


def test_scan_needs_its_workspace(L):
    a = ssm()
    need = [L.hla2_ssm_workspace_bytes(ctypes.byref(a), back) for back in (0, 1)]
    assert 0 < need[0] < need[1]
    for call, size in zip((forward, backward), need):
        assert call(L, a) == -3
        assert call(L, ssm(workspace=0x60000000, workspace_bytes=size - 1)) == -3
        assert call(L, ssm(workspace=0x60000008, workspace_bytes=size)) == -3
        if NO_GPU:
            assert call(L, ssm(workspace=0x60000000, workspace_bytes=size)) == -4
    assert L.hla2_ssm_forward(None, rows(0x20000000), None, None) == -1
    assert L.hla2_ssm_backward(ctypes.byref(a), rows(0x22000000), None, None, None) == -1


def test_scan_refuses_sizes_past_its_indices(L):
    assert forward(L, ssm(B=1 << 20, D=1 << 12)) == -2
    assert forward(L, ssm(n=(1 << 30) + 1)) == -2


def test_scan_refuses_overlaps(L):
    for out in (rows(0x10000000), rows(0x11000000 + SIZE - 2), rows(0x12000000 - SIZE + 2), rows(0x13000000 + BC - 2), rows(0x14000000),
                rows(0x15000000 + 16), rows(0x15100000), rows(0x21000000), rows(None), rows(0x20000001), Rows(0x20000000, N * D, D - 1),
                Rows(0x20000000, 0, D), Rows(0x20000000, D, D)):
        assert forward(L, ssm(), out) == -1, hex(out.p or 0)
    for fin in (0x15400000, 0x15400000 + ST - 16, 0x10000000, 0x21000004):
        assert forward(L, ssm(), fin=fin) == -1, hex(fin)
    # tokens before sequences do not overlap; adjacent tensors do not
    assert forward(L, ssm(), Rows(0x20000000, D, B * D)) == -3
    assert forward(L, ssm(), rows(0x10000000 + SIZE)) == -3
    bad = [dict(dx=rows(0x10000000)), dict(dx=rows(0x22000000)), dict(ddt=rows(0x30000000)), dict(dgate=rows(0x31000000 + 16)), dict(db=states(0x33000000 + 2 * BC), dc=states(0x33000000 + 2 * BC)),
           dict(db=states(0x13000000)), dict(da=0x15000000), dict(dskip=0x35000000 + 32), dict(ddt_bias=0x15200000),
           dict(dinit_state=0x23000000), dict(dinit_state=0x15400000), dict(dx=rows(None)), dict(da=None), dict(dskip=None),
           dict(ddt_bias=None), dict(dgate=rows(None)), dict(db=View(0x33000000, N * G * 16, 8, G * 16)), dict(da=0x35000002), dict(dinit_state=0x35300004)]
    for kw in bad:
        assert backward(L, ssm(), grads(**kw)) == -1, kw
        assert L.hla2_last_error().decode()
    assert backward(L, ssm(skip=None)) == -1 and backward(L, ssm(gate=rows(None))) == -1 and backward(L, ssm(dt_bias=None)) == -1
    assert backward(L, ssm(), dout=rows(None)) == -1 and backward(L, ssm(), dfin=0x23000002) == -1
    assert backward(L, ssm(), grads(dinit_state=None)) == -3


def test_scan_step_refuses(L):
    a = ssm(lengths=None, init_state=None)
    step = lambda a=a, st=0x21000000, out=Rows(0x20000000, D, 0): L.hla2_ssm_decode_step(ctypes.byref(a), st, out, None)  # noqa: E731
    assert step(ssm(init_state=None)) == -1 and step(ssm(lengths=None)) == -1
    for st in (None, 0x21000008, 0x15000000, 0x10000000, 0x20000000):
        assert step(st=st) == -1, st
    for out in (Rows(None, D, 0), Rows(0x10000000, D, 0), Rows(0x20000000, D - 1, 0), Rows(0x20000001, D, 0), Rows(0x15100000, D, 0)):
        assert step(out=out) == -1
    assert step(ssm(B=0, lengths=None, init_state=None)) == 0


def test_empty_scans_succeed(L):
    assert forward(L, ssm(B=0)) == 0 and forward(L, ssm(D=0)) == 0 and backward(L, ssm(D=0)) == 0
    none = dict(x=rows(None), dt=rows(None), gate=rows(None), b=states(None), c=states(None))
    assert forward(L, ssm(n=0, **none), rows(None), None) == 0


def conv(**kw):
    c = dict(dtype=1, B=B, n=N, D=D, W=4, silu=1, x=rows(0x10000000), weight=0x15000000, bias=0x15100000, lengths=0x15300000,
             init_state=0x15400000, workspace=None, workspace_bytes=0)
    c.update(kw)
    return ConvArgs(*c.values())


BAD_CONV = [dict(dtype=2), dict(B=-1), dict(n=-1), dict(D=-1), dict(W=1), dict(W=5), dict(silu=2), dict(x=rows(None)), dict(x=rows(0x10000001)),
            dict(x=Rows(0x10000000, -D, D)), dict(weight=None), dict(weight=0x15000001), dict(bias=0x15100001), dict(init_state=0x15400001),
            dict(lengths=0x15300001)]


def conv_forward(L, a, out=rows(0x20000000), fin=0x21000000):
    return L.hla2_short_conv_forward(ctypes.byref(a), out, fin, None)


def conv_backward(L, a, **kw):
    c = dict(dout=rows(0x22000000), dfin=0x23000000, dx=rows(0x30000000), dw=0x35000000, db=0x35100000, dinit=0x35300000)
    c.update(kw)
    return L.hla2_short_conv_backward(ctypes.byref(a), *c.values(), None)


@pytest.mark.parametrize("kw", BAD_CONV)
def test_convolution_refuses(L, kw):
    assert conv_forward(L, conv(**kw)) == -1 and conv_backward(L, conv(**kw)) == -1
    assert L.hla2_last_error().decode()
    if "n" not in kw:
        a = conv(**{"lengths": None, "init_state": None, **kw})
        assert L.hla2_short_conv_decode_step(ctypes.byref(a), 0x21000000, rows(0x20000000), None) == -1


def test_convolution_refuses_overlaps(L):
    st = B * 3 * D * 2
    for out in (rows(0x10000000), rows(0x10000000 + SIZE - 2), rows(0x15000000), rows(0x15400000 - 16), rows(0x21000000), rows(None),
                Rows(0x20000000, N * D, D - 1)):
        assert conv_forward(L, conv(), out) == -1
    for fin in (0x15400000, 0x15400000 + st - 2, 0x10000000, 0x21000001):
        assert conv_forward(L, conv(), fin=fin) == -1
    for kw in (dict(dx=rows(0x10000000)), dict(dx=rows(0x22000000 + 2)), dict(dw=0x15000000), dict(dw=None), dict(db=None), dict(db=0x35000000),
               dict(dinit=0x15400000), dict(dinit=0x23000000), dict(dinit=0x30000000), dict(dx=rows(None)), dict(dout=rows(None)),
               dict(dw=0x35000002), dict(dfin=0x23000001)):
        assert conv_backward(L, conv(), **kw) == -1, kw
        assert L.hla2_last_error().decode()
    assert conv_backward(L, conv(bias=None)) == -1 and conv_backward(L, conv()) == -3
    need = L.hla2_short_conv_backward_workspace_bytes(ctypes.byref(conv()))
    assert need > 0 and conv_backward(L, conv(workspace=0x60000000, workspace_bytes=need - 1)) == -3
    assert L.hla2_short_conv_backward_workspace_bytes(ctypes.byref(conv(W=7))) == Z(-1).value
    a = conv(lengths=None, init_state=None)
    step = lambda st, out: L.hla2_short_conv_decode_step(ctypes.byref(a), st, out, None)  # noqa: E731
    ok = Rows(0x20000000, D, 0)
    assert step(None, ok) == -1 and step(0x10000000, ok) == -1 and step(0x20000000, ok) == -1 and step(0x21000001, ok) == -1
    assert step(0x21000000, Rows(0x15000000, D, 0)) == -1
    assert L.hla2_short_conv_decode_step(ctypes.byref(conv()), 0x21000000, ok, None) == -1  # lengths and a state


def test_empty_convolutions_succeed(L):
    assert conv_forward(L, conv(B=0)) == 0 and conv_forward(L, conv(D=0)) == 0 and conv_backward(L, conv(D=0)) == 0
    assert conv_forward(L, conv(n=0, x=rows(None)), rows(None), None) == 0


def norm(**kw):
    c = dict(dtype=1, rows=3, D=64, eps=1e-5, x=0x10000, x_stride=64, weight=0x20000, bias=0x30000)
    c.update(kw)
    return NormArgs(*c.values())


BAD_NORM = [dict(dtype=3), dict(D=0), dict(rows=-1), dict(x=None), dict(weight=None), dict(x=0x10001), dict(bias=0x30001), dict(x_stride=-64)]


def norm_backward(L, a, **kw):
    c = dict(dout=0x40000, dx=0x50000, dw=0x60000, db=0x70000, ws=None, size=0)
    c.update(kw)
    return L.hla2_layer_norm_backward(ctypes.byref(a), *c.values(), None)


@pytest.mark.parametrize("kw", BAD_NORM)
def test_norm_refuses(L, kw):
    assert L.hla2_layer_norm(ctypes.byref(norm(**kw)), 0x50000, None) == -1
    assert norm_backward(L, norm(**kw), ws=0x80000, size=1 << 30) == -1
    assert L.hla2_last_error().decode()


def test_norm_refuses_overlaps_but_rows_in_place(L):
    size = 3 * 64 * 2
    call = lambda out, a=norm(): L.hla2_layer_norm(ctypes.byref(a), out, None)  # noqa: E731
    assert call(None) == -1 and call(0x50001) == -1 and call(0x20000) == -1 and call(0x30000 - size + 2) == -1
    assert call(0x10000 + 128) == -1 and call(0x10000, norm(x_stride=128)) == -1 and call(0x10000 - 2) == -1
    assert L.hla2_layer_norm(ctypes.byref(norm(D=8193)), 0x50000, None) == -2
    if NO_GPU:
        assert call(0x10000) == -4 and call(0x50000) == -4
    assert norm_backward(L, norm()) == -3
    assert norm_backward(L, norm(), dx=0x10000) == -3 and norm_backward(L, norm(), dx=0x40000) == -3 and norm_backward(L, norm(), db=None) == -3
    for kw in (dict(dx=0x10000 + 128), dict(dx=0x40000 - 128), dict(dx=0x20000), dict(dw=0x70000), dict(dw=0x10000), dict(db=0x50000), dict(dw=None),
               dict(db=0x40000 + 64), dict(dw=0x20000), dict(dout=None), dict(dx=None), dict(dw=0x60002), dict(dx=0x50001)):
        assert norm_backward(L, norm(), **kw) == -1, kw
    need = L.hla2_layer_norm_backward_workspace_bytes(ctypes.byref(norm()))
    assert need > 0 and norm_backward(L, norm(), ws=0x80000, size=need - 1) == -3
    assert L.hla2_layer_norm_backward_workspace_bytes(ctypes.byref(norm(D=0))) == Z(-1).value
    assert L.hla2_layer_norm(ctypes.byref(norm(rows=0, x=None)), None, None) == 0


def test_bindings_refuse_host_tensors_and_bad_shapes():
    t, a, b = torch.zeros(1, 4, 16), torch.zeros(16, 8), torch.zeros(1, 4, 8)
    with pytest.raises(TypeError):
        hla.ssm_forward(t, t, a, b, b)
    with pytest.raises(TypeError):
        hla.ssm_backward(t, t, a, b, b, t)
    with pytest.raises(TypeError):
        hla.ssm_decode_step(torch.zeros(1, 16, 8), t[:, 0], t[:, 0], a, b[:, 0], b[:, 0])
    with pytest.raises(TypeError):
        hla.short_conv_forward(t, torch.zeros(16, 4))
    with pytest.raises(TypeError):
        hla.short_conv_backward(t, torch.zeros(16, 4), t)
    with pytest.raises(TypeError):
        hla.short_conv_decode_step(torch.zeros(1, 3, 16), t[:, 0], torch.zeros(16, 4))
    with pytest.raises(TypeError):
        hla.layer_norm(t, torch.zeros(16))
    with pytest.raises(TypeError):
        hla.layer_norm_backward(t, torch.zeros(16), t)


@pytest.mark.gpu
def test_bindings_refuse_what_does_not_fit():
    z = lambda *s, dtype=torch.float32: torch.zeros(s, device="cuda", dtype=dtype)  # noqa: E731
    x, a, b = z(2, 5, 16), z(16, 8), z(2, 5, 8)
    half = lambda t: t.to(torch.bfloat16)  # noqa: E731
    for bad in (dict(dt=z(2, 5, 15)), dict(dt=half(x)), dict(a=z(15, 8)), dict(a=z(16, 8, 1)), dict(b=z(2, 4, 8)), dict(c=z(2, 5, 1, 8)),
                dict(b=z(2, 5, 3, 8), c=z(2, 5, 3, 8)), dict(skip=z(15)), dict(gate=z(2, 5, 1)), dict(dt_bias=z(16, 1)), dict(lengths=[1]),
                dict(lengths=z(2)), dict(init_state=z(2, 16, 9)), dict(init_state=half(z(2, 16, 8))), dict(x=z(5, 16)), dict(skip=torch.zeros(16))):
        args = {**dict(x=x, dt=x, a=a, b=b, c=b), **bad}
        with pytest.raises((ValueError, TypeError)):
            hla.ssm_forward(**args)
        with pytest.raises((ValueError, TypeError)):
            hla.ssm_backward(dout=x, **args)
    with pytest.raises(hla.HLA2Error):
        hla.ssm_forward(x, x, z(16, 12), z(2, 5, 12), z(2, 5, 12))
    for bad in (z(2, 5, 15), half(x), z(1, 5, 16)):
        with pytest.raises((ValueError, TypeError)):
            hla.ssm_backward(x, x, a, b, b, bad)
    for state in (z(2, 16, 9), half(z(2, 16, 8)), z(2, 8, 16).transpose(1, 2), z(1, 16, 8)):
        with pytest.raises((ValueError, TypeError)):
            hla.ssm_decode_step(state, x[:, 0], x[:, 0], a, b[:, 0], b[:, 0])
    w = z(16, 4)
    for bad in (dict(weight=z(15, 4)), dict(weight=half(w)), dict(bias=z(15)), dict(act="tanh"), dict(init_state=z(2, 4, 16)), dict(lengths=[1, 2, 3])):
        with pytest.raises((ValueError, TypeError)):
            hla.short_conv_forward(**{**dict(x=x, weight=w), **bad})
    with pytest.raises(hla.HLA2Error):
        hla.short_conv_forward(x, z(16, 5))
    with pytest.raises(ValueError):
        hla.short_conv_decode_step(z(2, 4, 16), x[:, 0], w)
    for args in ((x, z(15)), (x, half(z(16)))):
        with pytest.raises((ValueError, TypeError)):
            hla.layer_norm(*args)
    with pytest.raises(hla.HLA2Error):
        hla.layer_norm(z(2, 8200), z(8200))
    with pytest.raises(ValueError):
        hla.layer_norm(x, z(16), out=z(2, 5, 15))
    with pytest.raises(ValueError):
        hla.layer_norm_backward(x, z(16), z(2, 5, 15))


@pytest.mark.parametrize("n", [0, 1, -1, (1 << 30) + 1, -(1 << 31)])
def test_steps_do_not_look_at_n(L, n):
    out, state = Rows(0x20000000, D, 0), 0x21000000
    none = dict(lengths=None, init_state=None, n=n)
    steps = ((L.hla2_ssm_decode_step, ssm), (L.hla2_short_conv_decode_step, conv))
    for step, args in steps:
        assert step(ctypes.byref(args(B=0, **none)), state, out, None) == 0
        assert step(ctypes.byref(args(D=0, **none)), state, out, None) == 0
        assert step(ctypes.byref(args(**none)), None, out, None) == -1  # what it does look at
        assert "state" in L.hla2_last_error().decode()
        assert step(None, state, out, None) == -1
        if NO_GPU:
            assert step(ctypes.byref(args(**none)), state, out, None) == -4


def test_gradients_may_lie_side_by_side(L):
    """Parts of the rows of one buffer share no element, though their address ranges meet."""
    wide = lambda p, at=0, d=2 * D: Rows(p + 2 * at, N * d, d)  # noqa: E731
    both = lambda p, at, each=16, d=2 * G * 16: View(p + 2 * at, N * d, each, d)  # noqa: E731
    ok = [dict(dx=wide(0x40000000), dgate=wide(0x40000000, D)),
          dict(dx=wide(0x40000000, D), dgate=wide(0x40000000)),
          dict(dx=wide(0x40000000, 0, 3 * D), ddt=wide(0x40000000, D, 3 * D), dgate=wide(0x40000000, 2 * D, 3 * D)),
          dict(db=both(0x40000000, 0), dc=both(0x40000000, G * 16)),
          dict(db=both(0x40000000, 0, 32), dc=both(0x40000000, 16, 32)),  # group by group
          dict(dx=Rows(0x40000000, 2 * D, 2 * B * D), dgate=Rows(0x40000000 + 2 * D, 2 * D, 2 * B * D))]  # tokens before sequences
    for kw in ok:
        assert backward(L, ssm(), grads(**kw)) == -3, kw
    bad = [dict(dx=wide(0x40000000), dgate=wide(0x40000000, D - 1)), dict(dx=wide(0x40000000, 1), dgate=wide(0x40000000, D + 2)),
           dict(dx=wide(0x40000000), dgate=wide(0x40000000)), dict(dx=wide(0x40000000), dgate=wide(0x40000000, D, 2 * D + 1)),
           dict(db=both(0x40000000, 0), dc=both(0x40000000, G * 16 - 1)), dict(db=both(0x40000000, 0, 32), dc=both(0x40000000, 24, 32)),
           dict(dx=wide(0x40000000), da=0x40000000 + 16 * D)]  # the sums have no place in a row
    for kw in bad:
        assert backward(L, ssm(), grads(**kw)) == -1, kw
    # outputs beside inputs
    assert forward(L, ssm(x=wide(0x40000000)), wide(0x40000000, D)) == -3
    assert forward(L, ssm(x=wide(0x40000000)), wide(0x40000000, D + 1)) == -1
    assert backward(L, ssm(x=wide(0x40000000)), grads(dx=wide(0x40000000, D))) == -3
    assert conv_backward(L, conv(x=wide(0x40000000)), dx=wide(0x40000000, D)) == -3
    assert conv_backward(L, conv(x=wide(0x40000000)), dx=wide(0x40000000, D // 2)) == -1
    assert conv_backward(L, conv(), dx=wide(0x40000000), dw=0x40000000 + 4 * D) == -1
    if NO_GPU:
        assert conv_forward(L, conv(x=wide(0x40000000)), wide(0x40000000, D)) == -4
        a = conv(lengths=None, init_state=None, x=Rows(0x40000000, 2 * D, 0))
        assert L.hla2_short_conv_decode_step(ctypes.byref(a), 0x21000000, Rows(0x40000000 + 2 * D, 2 * D, 0), None) == -4
        a = ssm(lengths=None, init_state=None, x=Rows(0x40000000, 2 * D, 0))
        assert L.hla2_ssm_decode_step(ctypes.byref(a), 0x21000000, Rows(0x40000000 + 2 * D, 2 * D, 0), None) == -4


def test_no_shared_element_passes(L):
    """Random layouts of two gradients in one buffer: those that share an element are refused, whatever their strides."""
    rng = random.Random(3)
    seen = {-1: 0, -3: 0}
    for _ in range(4000):
        b, n, d = rng.randint(1, 3), rng.randint(1, 4), rng.choice([4, 6])
        unit = rng.choice([d, d + 2, 2 * d, 3 * d])
        sn = rng.choice([unit, unit * rng.randint(1, 3), unit + rng.randint(0, 3)])
        sb = rng.choice([sn * n, sn * n + unit, sn * n + rng.randint(0, 5)])
        first = Rows(0x40000000, sb, sn)
        if rng.random() < 0.3:
            sn, sb = sn * 2, sb * rng.choice([1, 2])
        second = Rows(0x40000000 + 2 * rng.randint(0, 3 * unit), sb, sn)

        def places(r):
            return [r.p + 2 * (i * r.sb + t * r.sn + k) for i in range(b) for t in range(n) for k in range(d)]

        one, two = places(first), places(second)
        args = ssm(B=b, n=n, D=d, G=1, gate=rows(0x12000000, n, d), x=rows(0x10000000, n, d), dt=rows(0x11000000, n, d),
                   b=View(0x13000000, n * 16, 16, 16), c=View(0x14000000, n * 16, 16, 16))
        g = grads(dx=first, dgate=second, ddt=rows(0x31000000, n, d), db=View(0x33000000, n * 16, 16, 16),
                  dc=View(0x34000000, n * 16, 16, 16))
        rc = backward(L, args, g, dout=rows(0x22000000, n, d))
        seen[rc] += 1
        shared = len(set(one + two)) < len(one) + len(two)
        assert rc == -1 or not shared, (b, n, d, first.sb, first.sn, second.p - first.p, second.sb, second.sn)
    assert min(seen.values()) > 300, seen


def test_lengths_of_no_sequences():
    none = _length_tensor([], 0, 5, torch.device("cpu"))
    assert none.dtype == torch.int32 and none.shape == (0,)
    assert _length_tensor([7, -1, 1 << 40], 3, 5, torch.device("cpu")).tolist() == [5, 0, 5]
    for bad in ([1.0], [True], torch.zeros(1), torch.zeros(0), [], [1, 2], torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            _length_tensor(bad, 1, 5, torch.device("cpu"))
