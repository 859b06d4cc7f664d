"""Calls of several threads on one stream: the scratch that they share is one call's at a time."""
import threading
import time

import pytest
import torch

import chunked_scan_mixer_gb300 as hla
from chunked_scan_mixer_gb300 import hla2


class Busy:
    """Callable that counts how many threads are inside it."""

    def __init__(self):
        self.inside = self.most = self.calls = 0
        self.lock = threading.Lock()

    def __call__(self, *args):
        with self.lock:
            self.inside += 1
            self.calls += 1
            self.most = max(self.most, self.inside)
        time.sleep(0.01)
        with self.lock:
            self.inside -= 1
        return 0


def together(*fs, each=4):
    errors = []

    def loop(f):
        try:
            for _ in range(each):
                f()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    ts = [threading.Thread(target=loop, args=(f,)) for f in fs]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors


def test_calls_on_cached_scratch_do_not_overlap(monkeypatch):
    busy, quick = Busy(), Busy()
    buf = torch.zeros(1024, dtype=torch.uint8)
    monkeypatch.setattr(hla2, "_cached_scratch", lambda t: buf)

    class Host:
        linattn_forward = staticmethod(lambda *a: busy(*a))

    monkeypatch.setattr(hla2, "_host", Host)
    monkeypatch.setattr(hla2, "_capturing", lambda: False)
    monkeypatch.setitem(hla2._scratch_cache, (0, None), buf)
    t = torch.zeros(1)
    together(lambda: hla2._with_scratch(busy, lambda: 512, 0, 0), lambda: hla.linattn_forward(t, t, t),
             lambda: hla2._alone(busy), lambda: hla2._with_scratch(busy, lambda: 512, 0, 0))
    assert busy.calls == 16 and busy.most == 1
    together(quick, quick)
    assert quick.most == 2  # the count sees an overlap


@pytest.mark.parametrize("name", ["hla2_forward", "hla2_ahla_forward", "hla2_backward", "hla2_hla3_forward", "hla2_ahla_backward"])
def test_every_call_with_a_cached_workspace_is_made_alone(name):
    import inspect

    source = inspect.getsource(hla2)
    assert f"_alone(L.{name}," in source and f"L.{name}(" not in source


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_threads_on_the_default_stream(dtype):
    """Different inputs in each thread, by the way that lets other threads run during the call and by the compiled one."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    make = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    work = []
    for n in (3000, 1777):
        q, k, v, do = make(1, 4, n, 64), make(1, 2, n, 64) / 8, make(1, 2, n, 64), make(1, 4, n, 64)
        x, w = make(3000, 256), make(256)
        kw = dict(gamma=torch.tensor([0.99, 0.999], device="cuda"), scale=0.125)

        def call(q=q, k=k, v=v, do=do, x=x, w=w, kw=kw, out=torch.empty_like(q)):
            a = hla.linattn_forward(q, k, v, out=out, return_final_state=True, **kw)
            b = hla.linattn_forward(q, k, v, return_final_state=True, **kw)
            c = hla.linattn_backward(q, k, v, do, dq=torch.empty_like(q), **kw)
            return (*(t.clone() for t in a), *b, *c, *hla.block_norm_backward(x, w, x))

        work.append((call, call()))
    torch.cuda.synchronize()
    kept = []

    def run(i):
        for _ in range(10):
            kept.append((i, work[i][0]()))

    together(lambda: run(0), lambda: run(1), each=1)
    torch.cuda.synchronize()
    hla.check_status()
    assert len(kept) == 20
    for i, got in kept:
        for a, b in zip(got, work[i][1]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_calls_of_different_sizes_do_not_lower_each_others_limit():
    """Widths that share a kernel but not its shared memory, from threads that run during each other's calls."""
    xs = [torch.randn((4000, D), device="cuda") for D in (8192, 4100, 6000)]
    ws = [torch.ones(x.shape[1], device="cuda") for x in xs]
    outs = [torch.empty_like(x) for x in xs]
    want = [hla.block_norm(x, w) for x, w in zip(xs, ws)]
    torch.cuda.synchronize()
    together(*(lambda i=i: hla.block_norm(xs[i], ws[i], out=outs[i]) for i in range(3)), each=1500)
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
