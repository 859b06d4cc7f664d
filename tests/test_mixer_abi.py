"""Host-side checks of the entry points around a mixer layer (no GPU): bad arguments are refused
with a message before any launch, empty calls succeed, and the structures match the header."""
import ctypes

import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from chunked_scan_mixer_gb300.hla2 import _BLOCK_ARGS, _LINATTN_ARGS, View


@pytest.fixture(scope="module")
def L():
    return hla.lib()


class LinattnArgs(ctypes.Structure):
    """hla2_linattn_args, field by field."""
    _fields_ = [
        ("dtype", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int), ("Hk", ctypes.c_int), ("n", ctypes.c_int),
        ("d", ctypes.c_int), ("dv", ctypes.c_int), ("scale", ctypes.c_float), ("gamma", ctypes.c_void_p),
        ("lengths", ctypes.c_void_p), ("q", View), ("k", View), ("v", View), ("init_state", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class BlockArgs(ctypes.Structure):
    """hla2_block_args, field by field."""
    _fields_ = [
        ("dtype", ctypes.c_int), ("gate_act", ctypes.c_int), ("gate_cols", ctypes.c_int),
        ("rows", ctypes.c_longlong), ("D", ctypes.c_int), ("eps", ctypes.c_float),
        ("x", ctypes.c_void_p), ("x_stride", ctypes.c_longlong), ("y", ctypes.c_void_p), ("y_stride", ctypes.c_longlong),
        ("gate", ctypes.c_void_p), ("gate_stride", ctypes.c_longlong), ("post_weight", ctypes.c_void_p),
        ("scale", ctypes.c_void_p), ("next_weight", ctypes.c_void_p),
    ]


def test_packed_argument_blocks_have_the_c_layout():
    a = LinattnArgs(1, 2, 6, 3, 5, 16, 32, 0.5, 8, 9, View(10, 11, 12, 13), View(14, 15, 16, 17), View(18, 19, 20, 21),
                    22, 23, 24)
    assert _LINATTN_ARGS.pack(1, 2, 6, 3, 5, 16, 32, 0.5, *range(8, 25)) == bytes(a)
    b = BlockArgs(1, 0, 64, 3, 64, 0.25, 6, 7, 8, 9, 10, 11, 12, 13, 14)
    assert _BLOCK_ARGS.pack(1, 0, 64, 3, 64, 0.25, *range(6, 15)) == bytes(b)


def view(p, B, H, n, D):
    return View(p, H * n * D, n * D, D)


def lin(**kw):
    c = dict(dtype=1, B=2, H=4, Hk=2, n=9, d=16, dv=32, scale=1.0, gamma=None, lengths=None, init_state=None,
             workspace=None, workspace_bytes=0)
    c.update({k: x for k, x in kw.items() if k in c})
    B, H, Hk, n, d, dv = (c[k] for k in ("B", "H", "Hk", "n", "d", "dv"))
    # distinct addresses that are never dereferenced
    q = kw.get("q", view(0x10000000, B, H, n, d))
    k = kw.get("k", view(0x20000000, B, Hk, n, d))
    v = kw.get("v", view(0x30000000, B, Hk, n, dv))
    a = LinattnArgs(c["dtype"], B, H, Hk, n, d, dv, c["scale"], None, None, q, k, v, c["init_state"], c["workspace"],
                    c["workspace_bytes"])
    return a, kw.get("out", view(0x40000000, B, H, n, dv))


BAD_LIN = [
    (dict(dtype=2), -1), (dict(B=-1), -1), (dict(n=-1), -1), (dict(d=48), -1), (dict(dv=8), -1), (dict(d=256), -1),
    (dict(H=3), -1), (dict(H=0), -1), (dict(Hk=0), -1), (dict(Hk=3), -1),
    (dict(q=view(None, 2, 4, 9, 16)), -1), (dict(k=view(0x20000008, 2, 2, 9, 16)), -1),
    (dict(q=View(0x10000000, 4 * 9 * 16, 9 * 16, 12)), -1),      # token stride not of 16 bytes
    (dict(v=View(0x30000000, 2 * 9 * 32, 9 * 32, 16)), -1),      # rows overlap
    (dict(k=View(0x20000000, 2 * 9 * 16, 0, 16)), -1),           # broadcast head
    (dict(out=view(0x30000000 + 64, 2, 4, 9, 32)), -1),          # out overlaps v
    (dict(init_state=0x50000004), -1),
    (dict(n=5000, init_state=0x50000000), -3),                   # no workspace
    (dict(n=5000, init_state=0x50000000, workspace=0x60000000, workspace_bytes=64), -3),
]


@pytest.mark.parametrize("kw, code", BAD_LIN)
def test_linattn_forward_refuses(L, kw, code):
    a, out = lin(**kw)
    assert L.hla2_linattn_forward(ctypes.byref(a), out, None, None) == code
    assert L.hla2_last_error().decode()


@pytest.mark.parametrize("kw, code", [x for x in BAD_LIN if "out" not in x[0]])
def test_linattn_backward_refuses(L, kw, code):
    a, dout = lin(**kw)
    B, H, Hk, n, d, dv = a.B, a.H, a.Hk, a.n, a.d, a.dv
    g = [view(0x70000000, B, H, n, d), view(0x80000000, B, Hk, n, d), view(0x90000000, B, Hk, n, dv)]
    assert L.hla2_linattn_backward(ctypes.byref(a), dout, *g, None, None, None) == code
    assert L.hla2_last_error().decode()


def test_linattn_backward_refuses_shared_outputs(L):
    a, dout = lin()
    dq, dk, dv = view(0x70000000, 2, 4, 9, 16), view(0x80000000, 2, 2, 9, 16), view(0x90000000, 2, 2, 9, 32)
    call = lambda *g: L.hla2_linattn_backward(ctypes.byref(a), dout, *g, None, None, None)  # noqa: E731
    assert call(dq, dq, dv) == -1
    assert call(view(0x10000000, 2, 4, 9, 16), dk, dv) == -1  # dq on q
    assert call(dq, dk, View(0x90000000, 2 * 9 * 32, 9 * 32, 30)) == -1


def test_linattn_refuses_states_in_place(L):
    """The state is read by CTAs that run beside the one that writes it."""
    size = 2 * 2 * 16 * 32 * 4  # bytes of [B, Hk, d, dv]
    init = 0x50000000
    a, out = lin(init_state=init)
    for at in (init, init + size - 16, init - size + 16):
        assert L.hla2_linattn_forward(ctypes.byref(a), out, at, None) == -1
        assert b"overlaps" in L.hla2_last_error()
    assert L.hla2_linattn_forward(ctypes.byref(a), out, init + size, None) == -3  # only the workspace is missing
    g = [view(0x70000000, 2, 4, 9, 16), view(0x80000000, 2, 2, 9, 16), view(0x90000000, 2, 2, 9, 32)]
    dout = view(0x40000000, 2, 4, 9, 32)
    back = lambda dfinal, dinit: L.hla2_linattn_backward(ctypes.byref(a), dout, *g, dfinal, dinit, None)  # noqa: E731
    for dinit in (init, init + size - 16, 0xA0000000, 0xA0000000 - size + 16):
        assert back(0xA0000000, dinit) == -1
        assert b"overlaps" in L.hla2_last_error()
    assert back(0xA0000000, 0xA0000000 + size) == -3
    assert back(None, init) == -1 and back(None, 0xA0000000) == -3


def test_linattn_empty_calls_succeed(L):
    for kw in (dict(B=0), dict(H=0, Hk=0), dict(n=0, q=view(None, 2, 4, 0, 16), k=view(None, 2, 2, 0, 16),
                                                v=view(None, 2, 2, 0, 32), out=view(None, 2, 4, 0, 32))):
        a, out = lin(**kw)
        assert L.hla2_linattn_forward(ctypes.byref(a), out, None, None) == 0, L.hla2_last_error()
        assert L.hla2_linattn_workspace_bytes(ctypes.byref(a), 0, 0) == 0


def test_linattn_workspace_grows_with_what_is_asked(L):
    a, _ = lin(n=1 << 20, d=64, dv=64)
    sizes = [L.hla2_linattn_workspace_bytes(ctypes.byref(a), *x) for x in ((0, 0), (1, 0))]
    assert 0 < sizes[0] < sizes[1]
    a, _ = lin(d=17)
    assert L.hla2_linattn_workspace_bytes(ctypes.byref(a), 0, 0) == ctypes.c_size_t(-1).value


def test_linattn_step_refuses(L):
    ok = dict(state=0x10000, q=0x20000, k=0x30000, v=0x40000, out=0x50000, N=2, H=4, Hk=2, d=16, dv=16, gamma=None,
              scale=1.0, dtype=1, stream=None)

    def call(**kw):
        c = {**ok, **kw}
        return L.hla2_linattn_decode_step(*(c[x] for x in ok))

    for kw in (dict(state=None), dict(q=None), dict(state=0x10004), dict(v=0x40002), dict(out=0x20000), dict(d=24),
               dict(dtype=5), dict(H=5), dict(N=-1)):
        assert call(**kw) == -1, kw
        assert L.hla2_last_error().decode()
    assert call(N=0) == 0


def block(**kw):
    c = dict(dtype=1, gate_act=0, gate_cols=64, rows=3, D=64, eps=1e-6, x=0x10000, x_stride=64, y=0x20000, y_stride=64,
             gate=0x30000, gate_stride=64, post_weight=0x40000, scale=0x50000, next_weight=0x60000)
    c.update(kw)
    return BlockArgs(*c.values())


BAD_BLOCK = [dict(dtype=3), dict(D=0), dict(rows=-1), dict(x=None), dict(y=None), dict(post_weight=None),
             dict(gate_act=2), dict(gate_cols=2), dict(x=0x10001), dict(gate=0x30001), dict(x_stride=-64),
             dict(y=None, next_weight=None)]


@pytest.mark.parametrize("kw", BAD_BLOCK)
def test_block_join_refuses(L, kw):
    assert L.hla2_block_join(ctypes.byref(block(**kw)), 0x70000, 0x80000, None) == -1
    assert L.hla2_last_error().decode()
    assert L.hla2_block_join_backward(ctypes.byref(block(**kw)), 0x11000, 0x12000, 0x13000, 0x14000, 0x15000, 0x16000,
                                      0x17000, 0x18000, 0x19000, 1 << 30, None) == -1


def test_block_join_refuses_outputs_that_do_not_match(L):
    a = block()
    assert L.hla2_block_join(ctypes.byref(block(D=8193)), 0x70000, 0x80000, None) == -2
    assert L.hla2_block_join(ctypes.byref(a), None, 0x80000, None) == -1
    assert L.hla2_block_join(ctypes.byref(a), 0x70000, None, None) == -1
    assert L.hla2_block_join(ctypes.byref(a), 0x70000, 0x70000, None) == -1
    assert L.hla2_block_join(ctypes.byref(block(rows=0, x=None, y=None, gate=None, scale=None, post_weight=None)), None,
                             0x80000, None) == 0
    grads = [0x13000, 0x14000, 0x15000, 0x16000, 0x17000, 0x18000]
    for i in range(6):
        g = list(grads)
        g[i] = None
        assert L.hla2_block_join_backward(ctypes.byref(a), 0x11000, 0x12000, *g, 0x19000, 1 << 30, None) == -1
    assert L.hla2_block_join_backward(ctypes.byref(a), None, None, *grads, 0x19000, 1 << 30, None) == -1
    assert L.hla2_block_join_backward(ctypes.byref(a), 0x11000, 0x12000, *grads, None, 0, None) == -3
    assert L.hla2_block_join_backward(ctypes.byref(a), 0x11000, 0x12000, *grads, 0x19000, 16, None) == -3


def join_backward(L, a, **kw):
    c = dict(dr=0x11000, dh=0x12000, dx=0x13000, dy=0x14000, dgate=0x15000, dpw=0x16000, dsc=0x17000, dnw=0x18000, ws=None,
             size=0, stream=None)
    c.update(kw)
    return L.hla2_block_join_backward(ctypes.byref(a), *c.values())


def test_block_join_refuses_overlaps_but_rows_in_place(L):
    """Without a device a call that passes the checks fails later: in the backward for want of a workspace (-3), in the
    forward at its launch (-4)."""
    a = block()
    size = 3 * 64 * 2
    call = lambda r, h, b=a: L.hla2_block_join(ctypes.byref(b), r, h, None)  # noqa: E731
    for r, h in ((0x70000, 0x70000 + size - 16), (0x10000 + 128, 0x80000), (0x70000, 0x20000 - 128), (0x30000 + 2, 0x80000),
                 (0x40000, 0x80000), (0x70000, 0x50000 + 64), (0x60000 - size + 16, 0x80000)):
        assert call(r, h) == -1, (hex(r), hex(h))
    wide = block(x_stride=128)  # rows of x between those that are written
    assert call(0x10000, 0x80000, wide) == -1
    row_gate = block(gate_cols=1, gate_stride=1)
    assert call(0x30000, 0x80000, row_gate) == -1
    if not torch.cuda.is_available():
        assert call(0x10000, 0x20000) == -4 and call(0x30000, 0x10000) == -4 and call(0x70000, 0x70000 + size) == -4
    assert join_backward(L, a) == -3
    for kw in (dict(dx=0x10000), dict(dx=0x11000, dy=0x12000), dict(dx=0x20000, dy=0x10000), dict(dgate=0x30000),
               dict(dx=0x12000, dy=0x11000, dgate=0x10000)):
        assert join_backward(L, a, **kw) == -3, kw
    assert join_backward(L, row_gate, dgate=0x30000) == -3
    for kw in (dict(dx=0x10000 + 128), dict(dx=0x11000 - 128), dict(dx=0x14000 + 16), dict(dy=0x15000), dict(dgate=0x13000 + 16),
               dict(dpw=0x17000 + 128), dict(dnw=0x16000), dict(dsc=0x13000 + size - 4), dict(dpw=0x40000), dict(dnw=0x12000),
               dict(dx=0x60000)):
        assert join_backward(L, a, **kw) == -1, kw


def test_w4_and_step_refuse_overlaps(L):
    ok = dict(x=0x10000, x_stride=256, w=0x20000, s=0x30000, z=0x34000, b=0x38000, y=0x40000, M=2, N=5, K=256, group=64,
              dtype=1, stream=None)
    call = lambda **kw: L.hla2_w4_matvec(*{**ok, **kw}.values())  # noqa: E731
    for y in (0x10000, 0x10000 + 2 * 512 - 2, 0x10000 - 18, 0x20000, 0x20000 + 5 * 128 - 2, 0x30000, 0x34000, 0x38000 + 8):
        assert call(y=y) == -1, hex(y)
        assert b"overlaps" in L.hla2_last_error()
    step = dict(state=0x10000, q=0x20000, k=0x30000, v=0x40000, out=0x50000, N=2, H=4, Hk=2, d=16, dv=32, gamma=None,
                scale=1.0, dtype=1, stream=None)
    call = lambda **kw: L.hla2_linattn_decode_step(*{**step, **kw}.values())  # noqa: E731
    for kw in (dict(out=0x20000 + 240), dict(out=0x30000 - 16), dict(out=0x40000 + 16), dict(out=0x10000 + 8176),
               dict(state=0x20000 + 240), dict(state=0x40000 - 16)):
        assert call(**kw) == -1, kw
        assert b"overlaps" in L.hla2_last_error()


def test_w4_refuses(L):
    ok = dict(x=0x10000, x_stride=256, w=0x20000, s=0x30000, z=None, b=None, y=0x40000, M=2, N=5, K=256, group=64,
              dtype=1, stream=None)

    def call(**kw):
        c = {**ok, **kw}
        return L.hla2_w4_matvec(*(c[x] for x in ok))

    for kw in (dict(x=None), dict(w=None), dict(s=None), dict(y=None), dict(x=0x10008), dict(x_stride=252),
               dict(w=0x20004), dict(s=0x30001), dict(group=16), dict(group=256), dict(K=96), dict(K=-64), dict(N=-1),
               dict(M=-1), dict(dtype=2)):
        assert call(**kw) == -1, kw
        assert L.hla2_last_error().decode()
    assert call(M=17) == -2
    assert call(M=0) == 0 and call(N=0) == 0


def test_bindings_refuse_host_tensors_and_bad_shapes():
    t = torch.zeros(1, 1, 4, 16)
    with pytest.raises(TypeError):
        hla.linattn_forward(t, t, t)
    with pytest.raises(TypeError):
        hla.block_norm(torch.zeros(2, 8), torch.zeros(8))
    with pytest.raises(ValueError):
        hla.block_join(torch.zeros(2, 8), None, torch.zeros(8))
    with pytest.raises(TypeError):
        hla.w4_matvec(torch.zeros(1, 64), torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1))
