"""A selective state space layer's calls from other devices and threads: they go to their tensors' device, and those on a
stream's cached scratch are made one at a time."""
import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from chunked_scan_mixer_gb300 import hla2

from .ssm_cases import make_ssm
from .test_devices import On, current, test_every_launching_function_goes_to_its_tensors_device as goes_to_its_device  # noqa: F401
from .test_threads import Busy, together

NAMES = ("_ssm_forward", "_ssm_backward", "_ssm_decode_step", "_short_conv_forward", "_short_conv_backward",
         "_short_conv_decode_step", "_layer_norm", "_layer_norm_backward")


@pytest.mark.parametrize("name", NAMES)
def test_goes_to_its_tensors_device(current, monkeypatch, name):  # noqa: F811
    goes_to_its_device(current, monkeypatch, name)


def test_the_short_calls_reach_them(current, monkeypatch):  # noqa: F811
    calls = []
    monkeypatch.setattr(hla2, "_quick", lambda *a: None)
    monkeypatch.setattr(hla2, "_cached_scratch", lambda t: None)
    for name in NAMES:
        monkeypatch.setattr(hla2, name, lambda *a, name=name: calls.append(name))
    t = On(1)
    hla.ssm_forward(t, t, t, t, t)
    hla.ssm_backward(t, t, t, t, t, t)
    hla.ssm_decode_step(t, t, t, t, t, t)
    hla.short_conv_forward(t, t)
    hla.short_conv_backward(t, t, t)
    hla.short_conv_decode_step(t, t, t)
    hla.layer_norm(t, t)
    hla.layer_norm_backward(t, t, t)
    assert calls == list(NAMES)


def test_calls_on_cached_scratch_do_not_overlap(monkeypatch):
    busy = Busy()
    buf = torch.zeros(1024, dtype=torch.uint8)
    monkeypatch.setattr(hla2, "_cached_scratch", lambda t: buf)

    class Host:
        ssm_forward = ssm_backward = short_conv_backward = staticmethod(lambda *a: (busy(*a),) * 9)
        layer_norm_backward = staticmethod(lambda *a: busy(*a))

    monkeypatch.setattr(hla2, "_host", Host)
    monkeypatch.setattr(hla2, "ShortConvGrads", lambda *a: a)
    monkeypatch.setattr(hla2, "_capturing", lambda: False)
    monkeypatch.setitem(hla2._scratch_cache, (0, None), buf)
    t = torch.zeros(1)
    together(lambda: hla2._with_scratch(busy, lambda: 512, 0, 0), lambda: hla.ssm_forward(t, t, t, t, t), lambda: hla.ssm_backward(t, t, t, t, t, t),
             lambda: hla.short_conv_backward(t, t, t), lambda: hla.layer_norm_backward(t, t, t))
    assert busy.calls == 20 and busy.most == 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_threads_on_the_default_stream(dtype):
    work = []
    for seed, n in ((1, 1500), (2, 777)):
        c = make_ssm(1, n, 64, 16, dtype=dtype, seed=seed)
        dout, w = torch.randn_like(c["x"]), torch.randn(64, 4, device="cuda").to(dtype)

        def call(c=c, dout=dout, w=w):
            return (*hla.ssm_forward(**c, return_final_state=True), *hla.ssm_backward(dout=dout, **c),
                    *hla.short_conv_backward(c["x"], w, dout)[:2], *hla.layer_norm_backward(c["x"], w[:, 0].contiguous(), dout))

        work.append((call, call()))
    torch.cuda.synchronize()
    kept = []

    def run(i):
        for _ in range(10):
            kept.append((i, work[i][0]()))

    together(lambda: run(0), lambda: run(1), each=1)
    torch.cuda.synchronize()
    assert len(kept) == 20
    for i, got in kept:
        for a, b in zip(got, work[i][1]):
            assert torch.equal(a, b)
