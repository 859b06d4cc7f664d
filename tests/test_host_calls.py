"""The compiled host side of the short calls (csrc/host_calls.cpp): it declines what is not an ordinary call,
and gives what the binding's own way gives."""
import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from chunked_scan_mixer_gb300 import hla2

BF, F32 = torch.bfloat16, torch.float32
NAMES = ("linattn_forward", "linattn_backward", "linattn_decode_step", "block_join", "block_join_backward", "w4_matvec")


@pytest.fixture(scope="module")
def host():
    hla.lib()
    assert hla2._host is not None, "the module is built beside the library"
    return hla2._host


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("count", range(13))
def test_declines_other_arguments(host, name, count):
    f = getattr(host, name)
    assert f(*[None] * count) is None
    assert f(*[3] * count) is None
    assert f(*["x"] * count) is None
    assert f(*[torch.ones(2, 2)] * count) is None  # not on the GPU
    assert f(*[torch.ones(0)] * count) is None


def test_bind_checks_its_arguments(host):
    with pytest.raises(TypeError):
        host.bind(1, 2)


def test_a_module_that_does_not_load_is_gone_without(monkeypatch, tmp_path):
    bad = tmp_path / "_hla2_host.so"
    bad.write_bytes(b"not a shared object")
    for name, value in (("_lib", None), ("_host", None), ("HOST_PATH", str(bad))):
        monkeypatch.setattr(hla2, name, value)
    with pytest.warns(RuntimeWarning, match="does not load"):
        L = hla2.lib()
    assert L is hla2.lib() and hla2._host is None and L.hla2_version() > 0
    with pytest.raises(TypeError):  # the way through the binding
        hla.block_norm(torch.zeros(2, 8), torch.zeros(8))


def test_the_module_is_built_again_for_another_torch(tmp_path):
    from chunked_scan_mixer_gb300 import build

    src, so = tmp_path / "a.cpp", tmp_path / "a.so"
    src.write_text("")
    so.write_text("")
    assert build.host_stale(str(so), [str(src)], "2.9.1")  # nobody knows what it was built against
    (tmp_path / "a.so.torch").write_text("2.9.1")
    assert not build.host_stale(str(so), [str(src)], "2.9.1")
    assert build.host_stale(str(so), [str(src)], "2.11.0")
    with open(build.HOST + ".torch") as f:
        assert f.read() == torch.__version__


def both(monkeypatch, call):
    """The call by the module, which has to take it, and without it."""
    class Seen:
        def __init__(self):
            self.results = []

        def __getattr__(self, name):
            def f(*a):
                r = getattr(real, name)(*a)
                self.results.append(r)
                return r
            return f

    real = hla2._host
    call()  # sizes the cached workspace
    seen = Seen()
    monkeypatch.setattr(hla2, "_host", seen)
    quick = call()
    assert seen.results and all(r is not None for r in seen.results)
    monkeypatch.setattr(hla2, "_host", None)
    monkeypatch.setattr(hla2, "HOST_PATH", "")
    plain = call()
    monkeypatch.undo()
    return quick, plain


def same(a, b):
    if a is None or b is None:
        assert a is b
    elif isinstance(a, torch.Tensor):
        assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()
        assert torch.equal(a, b)
    else:
        assert type(a) is type(b) and len(a) == len(b)
        for x, y in zip(a, b):
            same(x, y)


def randn(*shape, dtype=F32):
    return torch.randn(shape, device="cuda", dtype=F32).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("tokens_first", [False, True])
@pytest.mark.parametrize("extras", [False, True])
def test_linear_attention(host, monkeypatch, dtype, tokens_first, extras):
    def make(heads, D):
        if tokens_first:
            return randn(2, 200, heads, D, dtype=dtype).transpose(1, 2)
        return randn(2, heads, 200, D, dtype=dtype)

    q, k, v, do = make(4, 32), make(2, 32), make(2, 64), make(4, 64)
    kw = dict(scale=0.2)
    if extras:
        kw.update(gamma=torch.tensor([0.9, 0.99], device="cuda"), init_state=randn(2, 2, 32, 64),
                  lengths=torch.tensor([200, 77], dtype=torch.int32, device="cuda"))
    same(*both(monkeypatch, lambda: hla.linattn_forward(q, k, v, **kw)))
    same(*both(monkeypatch, lambda: hla.linattn_forward(q, k, v, return_final_state=True, **kw)))
    fin = randn(2, 2, 32, 64) if extras else None
    same(*both(monkeypatch, lambda: hla.linattn_backward(q, k, v, do, dfinal_state=fin, **kw)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_step(host, monkeypatch, dtype):
    st = randn(3, 2, 32, 64)
    q, k, v, g = randn(3, 4, 32, dtype=dtype), randn(3, 2, 32, dtype=dtype), randn(3, 2, 64, dtype=dtype), 0.5 + 0.4 * torch.rand(2, device="cuda")

    def call():
        s = st.clone()
        return hla.linattn_decode_step(s, q, k, v, gamma=g, scale=0.3), s

    same(*both(monkeypatch, call))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", [(7, 96), (2, 5, 33)])
@pytest.mark.parametrize("gate", ["none", "row", "full", "strided"])
def test_block(host, monkeypatch, dtype, shape, gate):
    D = shape[-1]
    x, y, dr, dh = (randn(*shape, dtype=dtype) for _ in range(4))
    pw, sc, nw = (randn(D, dtype=dtype) for _ in range(3))
    z = {"none": None, "row": randn(*shape[:-1], 1, dtype=dtype)}.get(gate, randn(*shape, dtype=dtype))
    if gate == "strided":
        if len(shape) != 2:
            pytest.skip("rows with a stride are two-dimensional")
        z = randn(shape[0], 2 * D, dtype=dtype)[:, :D]
    same(*both(monkeypatch, lambda: hla.block_norm(x, nw)))
    same(*both(monkeypatch, lambda: hla.block_norm_backward(x, nw, dh)))
    for s, n in ((sc, nw), (None, nw), (sc, None)):
        kw = dict(gate=z, gate_act="silu", scale=s, next_weight=n)
        same(*both(monkeypatch, lambda: hla.block_join(x, y, pw, **kw)))
        same(*both(monkeypatch, lambda: hla.block_join_backward(x, y, pw, dr=dr, dh=None if n is None else dh, **kw)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", [(1, 128), (3, 2, 128)])
@pytest.mark.parametrize("extras", [False, True])
def test_w4(host, monkeypatch, dtype, shape, extras):
    x, w = randn(*shape, dtype=dtype), torch.randint(0, 256, (21, 64), device="cuda", dtype=torch.uint8)
    s = randn(21, 2, dtype=dtype)
    zeros = torch.randint(0, 16, (21, 2), device="cuda", dtype=torch.uint8) if extras else None
    bias = randn(21, dtype=dtype) if extras else None
    same(*both(monkeypatch, lambda: hla.w4_matvec(x, w, s, zeros=zeros, bias=bias)))
