"""The compiled host side of a selective state space layer's calls: it declines what is not an ordinary call, and gives what
the binding's own way gives."""
import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from chunked_scan_mixer_gb300 import hla2

from .ssm_cases import BF, F32, make_ssm
from .test_host_calls import both, host, randn, same  # noqa: F401

NAMES = ("ssm_forward", "ssm_backward", "ssm_decode_step", "short_conv_forward", "short_conv_backward",
         "short_conv_decode_step", "layer_norm", "layer_norm_backward")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("count", range(16))
def test_declines_other_arguments(host, name, count):  # noqa: F811
    f = getattr(host, name)
    for arg in (None, 3, "x", True, torch.ones(2, 2), torch.ones(0), torch.ones(2, 2, 2)):  # not on the GPU
        assert f(*[arg] * count) is None


def test_every_entry_is_bound():
    hla.lib()
    assert hla2._host is not None and all(hasattr(hla2._host, n) for n in NAMES)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("extras", [False, True])
@pytest.mark.parametrize("n, groups", [(40, 1), (900, 2)])
def test_scan(host, monkeypatch, dtype, extras, n, groups):  # noqa: F811
    c = make_ssm(2, n, 64, 16, groups, dtype=dtype, gate=extras, skip=extras, bias=extras, state=extras)
    kw = dict(lengths=torch.tensor([n, n // 3], dtype=torch.int32, device="cuda") if extras else None)
    dout, dfin = randn(2, n, 64, dtype=dtype), randn(2, 64, 16) if extras else None
    same(*both(monkeypatch, lambda: hla.ssm_forward(**c, **kw)))
    steps = {**c, "dt": 0.1 * c["dt"].abs(), "dt_bias": None}  # positive: negative ones grow to NaN, which is not its own equal
    same(*both(monkeypatch, lambda: hla.ssm_forward(**steps, return_final_state=True, dt_softplus=False, **kw)))
    same(*both(monkeypatch, lambda: hla.ssm_backward(dout=dout, dfinal_state=dfin, **c, **kw)))
    if groups == 1:  # without the groups' dimension, and as parts of a projection
        flat = {**c, "b": c["b"][:, :, 0], "c": c["c"][:, :, 0]}
        wide = torch.empty(2, n, 130, device="cuda", dtype=dtype)
        wide[..., 3:67] = c["x"]
        flat["x"] = wide[..., 3:67]
        same(*both(monkeypatch, lambda: hla.ssm_backward(dout=dout, **flat, **kw)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("groups", [1, 2])
def test_scan_step(host, monkeypatch, dtype, groups):  # noqa: F811
    c = make_ssm(3, 1, 64, 16, groups, dtype=dtype)
    one = {k: c[k][:, 0] if k in ("x", "dt", "b", "c", "gate") else c[k] for k in c if k != "init_state"}
    if groups == 1:
        one["b"], one["c"] = one["b"][:, 0], one["c"][:, 0]

    def call():
        s = c["init_state"].clone()
        return hla.ssm_decode_step(s, **one), s

    same(*both(monkeypatch, call))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("extras", [False, True])
def test_convolution(host, monkeypatch, dtype, extras):  # noqa: F811
    x, w, do = randn(2, 50, 48, dtype=dtype), randn(48, 4, dtype=dtype), randn(2, 50, 48, dtype=dtype)
    kw, state = {}, randn(2, 3, 48, dtype=dtype)
    if extras:
        kw = dict(bias=randn(48, dtype=dtype), act="none", lengths=torch.tensor([50, 7], dtype=torch.int32, device="cuda"),
                  init_state=state)
    same(*both(monkeypatch, lambda: hla.short_conv_forward(x, w, **kw)))
    same(*both(monkeypatch, lambda: hla.short_conv_forward(x, w, return_final_state=True, **kw)))
    same(*both(monkeypatch, lambda: hla.short_conv_backward(x, w, do, dfinal_state=state if extras else None, **kw)))

    def step():
        s = state.clone()
        return hla.short_conv_decode_step(s, x[:, 0], w, bias=kw.get("bias")), s

    same(*both(monkeypatch, step))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", [(7, 96), (2, 5, 33)])
def test_norm(host, monkeypatch, dtype, shape):  # noqa: F811
    x, do, w, b = randn(*shape, dtype=dtype), randn(*shape, dtype=dtype), randn(shape[-1], dtype=dtype), randn(shape[-1], dtype=dtype)
    same(*both(monkeypatch, lambda: hla.layer_norm(x, w)))
    same(*both(monkeypatch, lambda: hla.layer_norm(x, w, bias=b)))
    same(*both(monkeypatch, lambda: hla.layer_norm_backward(x, w, do)))
