"""The host side of examples/decode_layer.py on the CPU: the order of its work
over streams, with torch's CUDA calls replaced by a record of them."""
import contextlib
import importlib.util
import os
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Recorder:
    """What the example uses of torch, on the CPU; `log` holds (event, stream)."""

    def __init__(self):
        import torch
        self.torch, self.log, self.now = torch, [], "main"
        rec = self

        class Stream:
            def __init__(self, name="side"):
                self.name = name

            def wait_stream(self, other):
                rec.log.append(("wait for " + other.name, self.name))

        class Event:
            def __init__(self, **kw):
                pass

            def record(self):
                pass

            synchronize = record

            def elapsed_time(self, other):
                return 1.0

        class Graph:
            def replay(self):
                rec.log.append(("replay", rec.now))

        @contextlib.contextmanager
        def stream(s):
            before, rec.now = rec.now, s.name
            yield
            rec.now = before

        self.cuda = types.SimpleNamespace(Stream=Stream, Event=Event, CUDAGraph=Graph, stream=stream,
                                          graph=lambda g: contextlib.nullcontext(), current_stream=lambda: Stream(self.now))

    def __getattr__(self, name):
        f = getattr(self.torch, name)
        if name not in ("Generator", "randn", "randint", "arange", "zeros"):
            return f

        def on_cpu(*a, **kw):
            kw.pop("device", None)
            self.log.append((name, self.now))
            return f(*a, **kw)
        return on_cpu


@pytest.fixture
def example(monkeypatch):
    spec = importlib.util.spec_from_file_location("decode_layer_host", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    rec = Recorder()

    class Layer:
        d_model = 64

        def __init__(self, kind, fmt, batch=4, max_len=1024, **sizes):
            self.batch, self.max_len = batch, max_len
            rec.log.append(("layer", rec.now))

        def prompt(self, x, lens):
            rec.log.append(("prompt", rec.now))

        def step(self, x):
            rec.log.append(("step", rec.now))
            return rec.torch.ones(4)

        def check_cache(self, x, lens, token, steps):
            pass

        def plain_step(self, x):
            return rec.torch.ones(4).double()

    monkeypatch.setattr(m, "torch", rec)
    monkeypatch.setattr(m, "AttentionLayer", Layer)
    monkeypatch.setattr(m.qmm, "check_device_error", lambda: 0)
    m.rec = rec
    return m


def test_the_first_step_waits_for_what_it_reads(example):
    example.run(steps=3)
    log = example.rec.log
    first = log.index(("step", "side"))
    made = max(i for i, e in enumerate(log[:first]) if e[1] == "main")   # prompt, token, lengths
    assert ("wait for main", "side") in log[made:first]
    assert ("wait for side", "main") in log[first:log.index(("step", "main"))]   # and the capture for the step


@pytest.mark.parametrize("steps,sizes", [(824, {}), (100, dict(max_len=128)), (1, dict(max_len=3)), (0, {}), (-1, {})])
def test_steps_past_the_cache_are_refused(example, steps, sizes):
    """Positions beyond the page table would index it out of range."""
    with pytest.raises(ValueError):
        example.run(steps=steps, **sizes)
    assert not any(e[0] in ("prompt", "step", "replay") for e in example.rec.log)


def test_steps_up_to_the_cache_run(example):
    example.run(steps=823)
    assert sum(e[0] == "replay" for e in example.rec.log) == 823
