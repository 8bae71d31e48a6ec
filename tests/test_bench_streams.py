"""The benchmark's launches go to a stream that waits for no other, so what the
default stream fills for them (inputs, zeroed workspaces) is waited for first."""
import argparse
import contextlib
import types

import pytest


def test_settle_waits_before_its_first_launch():
    import bench
    seen = []

    class Event:
        def __init__(self, enable_timing):
            pass

        def record(self, stream):
            pass

        def elapsed_time(self, other):
            return bench.SETTLE_MS

    cuda = types.SimpleNamespace(Event=Event, synchronize=lambda: seen.append("wait"),
                                 stream=lambda s: contextlib.nullcontext())
    bench.settle(types.SimpleNamespace(cuda=cuda), None, lambda i: seen.append("launch"))
    assert seen[0] == "wait" and "launch" in seen


class _Reached(Exception):
    pass


@pytest.mark.gpu
@pytest.mark.parametrize("step", ["model_step", "model_step_paged"])
def test_decode_step_waits_for_its_inputs(step, monkeypatch):
    import bench
    torch = pytest.importorskip("torch")
    waits = []
    wait, side = torch.cuda.synchronize, torch.cuda.Stream

    def make(*args, **kw):
        waits.clear()                      # only a wait behind this counts
        return side(*args, **kw)

    def enter(stream):
        raise _Reached

    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: (waits.append(1), wait(*a)))
    monkeypatch.setattr(torch.cuda, "Stream", make)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    with pytest.raises(_Reached):
        getattr(bench, step)(argparse.Namespace(model_step=1, steps=1, warmup=0, batch=2, context=70, prefix=64))
    assert waits, "the first work on the side stream follows no wait"
