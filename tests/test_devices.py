"""Calls on a device that is not the current one, without such a device: the binding makes the tensors' device current
for the library call.  (No mismatched launch is made.)"""
import contextlib

import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from chunked_scan_mixer_gb300 import hla2


class On:
    """As much of a CUDA tensor as the choice of the device looks at."""
    is_cuda = True

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


@pytest.fixture
def current(monkeypatch):
    """The current device, 0 at first; torch's way of changing it, recorded."""
    now = [0]

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        try:
            yield
        finally:
            now[0] = before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    return now


def test_the_first_cuda_tensor_names_the_device(current):
    seen = hla2._on_its_device(lambda *a, **kw: current[0])
    assert seen(On(1)) == 1 and seen(On(0)) == 0 and current == [0]
    assert seen(None, 2.0, torch.zeros(1), On(3), On(1)) == 3
    assert seen(x=None, q=On(2)) == 2
    assert seen(torch.zeros(1), scale=1.0) == 0 and seen() == 0
    fails = hla2._on_its_device(lambda t: 1 / 0)
    with pytest.raises(ZeroDivisionError):
        fails(On(1))
    assert current == [0]


PUBLIC = ("forward", "backward", "decode_step", "decode_step_mq", "ahla_forward", "ahla_backward", "ahla_decode_step",
          "hla3_forward", "hla3_decode_step")
REST = ("_convert_state", "_linattn_forward", "_linattn_backward", "_linattn_decode_step", "_block_norm", "_block_join",
        "_block_backward", "_w4_matvec")


@pytest.mark.parametrize("name", PUBLIC + REST)
def test_every_launching_function_goes_to_its_tensors_device(current, monkeypatch, name):
    class Reached(Exception):
        pass

    entered = []
    real = torch.cuda.device

    @contextlib.contextmanager
    def device(index):
        with real(index):
            entered.append(index)
            raise Reached
            yield

    monkeypatch.setattr(torch.cuda, "device", device)
    f = getattr(hla2, name)
    with pytest.raises(Reached):
        f(*[On(1)] * 4)
    assert entered == [1]


def test_the_short_calls_reach_them(current, monkeypatch):
    """With the compiled module declining (as it does off the current device), each public call takes the guarded way."""
    calls = []
    monkeypatch.setattr(hla2, "_quick", lambda *a: None)
    monkeypatch.setattr(hla2, "_cached_scratch", lambda t: None)
    for name in REST[1:]:
        monkeypatch.setattr(hla2, name, lambda *a, name=name: calls.append(name) or hla.BlockJoinGrads(*[None] * 6))
    t = On(1)
    hla.linattn_forward(t, t, t)
    hla.linattn_backward(t, t, t, t)
    hla.linattn_decode_step(t, t, t, t)
    hla.block_norm(t, t)
    hla.block_join(t, t, t)
    hla.block_norm_backward(t, t, t)
    hla.block_join_backward(t, t, t)
    hla.w4_matvec(t, t, t)
    assert calls == [*REST[1:6], "_block_backward", "_block_backward", "_w4_matvec"]
