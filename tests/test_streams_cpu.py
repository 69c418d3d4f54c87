"""What prepared objects do before a call on another stream than the one they were made on, against a fake
of torch.cuda: no GPU is needed to see which waits and records are made."""
import contextlib

import pytest
import torch

from learnable_channel_permutation_b200 import binding as b


class Stream:
    def __init__(self, raw):
        self.cuda_stream, self.waits = raw, []

    def wait_event(self, event):
        self.waits.append(event)


class Tensor:
    def __init__(self):
        self.streams = []

    def record_stream(self, s):
        self.streams.append(s)


@pytest.fixture
def cuda(monkeypatch):
    """A device whose current stream is ``now``; streams in ``capturing`` are being captured."""
    class Cuda:
        now, home, side, capturing, events = None, Stream(0), Stream(7), set(), []

    class Event:
        def record(self, stream):
            Cuda.events.append((self, stream))

    Cuda.now, Cuda.events = Cuda.home, []

    @contextlib.contextmanager
    def use(stream):
        was, Cuda.now = Cuda.now, stream
        yield
        Cuda.now = was

    Cuda.use = staticmethod(use)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: Cuda.now.cuda_stream, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: Cuda.now)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: Cuda.now in Cuda.capturing, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "Event", Event)
    return Cuda


def _held(n=2):
    ts = [Tensor() for _ in range(n)]
    return b._Held(torch.device("cuda", 0), ts), ts


def test_calls_on_the_stream_it_was_made_on_need_nothing(cuda):
    held, ts = _held()
    assert held.on(None) == 0 and held.on(cuda.home) == 0
    assert not any(t.streams for t in ts) and not cuda.home.waits


@pytest.mark.parametrize("explicit", [True, False])
def test_the_first_call_on_another_stream_waits_and_is_recorded(cuda, explicit):
    held, ts = _held()
    (event, at), = cuda.events
    assert at is cuda.home
    for _ in range(3):
        if explicit:
            assert held.on(cuda.side) == 7
        else:
            with cuda.use(cuda.side):
                assert held.on(None) == 7
    assert all(t.streams == [cuda.side] for t in ts) and cuda.side.waits == [event]
    cuda.side.waits = []


def test_a_captured_call_is_recorded_and_does_not_wait_for_work_outside_the_capture(cuda):
    held, ts = _held()
    cuda.side.waits = []
    cuda.capturing = {cuda.side}
    held.on(cuda.side)
    assert all(t.streams == [cuda.side] for t in ts) and not cuda.side.waits
    cuda.capturing = set()
    held.on(cuda.side)                      # the first call outside the capture does
    assert len(cuda.side.waits) == 1


def test_an_object_made_inside_a_capture_records_no_event(cuda):
    cuda.capturing = {cuda.home}
    held, _ = _held()
    assert held.made is None and not cuda.events
    cuda.capturing = set()


def _without_init(cls, **attrs):
    x = object.__new__(cls)
    x.__dict__.update(attrs)
    return x


def test_list_calls_go_through_it(cuda):
    held, ts = _held()
    calls = []
    fn = lambda *a: calls.append(a[-1]) or 0
    lst = _without_init(b.GradList, held=held, head=(1, 2), tail=(3, 4, 5), device=torch.device("cuda", 0), norm_out="norm")
    assert lst._call(fn, stream=cuda.side) == "norm" and calls == [7]
    assert all(t.streams == [cuda.side] for t in ts)


@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_training_goes_through_it(cuda, monkeypatch, max_norm):
    step_held, step_ts = _held()
    held, ts = _held()
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a[-1])) or 0

    monkeypatch.setattr(b, "lib", Lib)
    buf = torch.zeros(4)
    step = _without_init(b.Step, _held=step_held, hp=b.hparams(64, 2, 4, 5, 1.0, 0), n=1, arr=None, ws=buf)
    tr = _without_init(b.Trainer, _held=held, step=step, opt=b.adamw_params(), state=None, total=4, tau_start=1.0, tau_end=0.1,
                       max_norm=max_norm, grad_norm=buf, ws=buf)
    tr.run(0, 1, stream=cuda.side)
    assert calls == [("lcp_train" if max_norm is None else "lcp_train_clip", 7)]
    assert all(t.streams == [cuda.side] for t in ts + step_ts)
    calls.clear()
    step.run(stream=cuda.home)
    assert calls == [("lcp_step", 0)]
