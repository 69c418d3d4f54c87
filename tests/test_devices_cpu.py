"""Calls of prepared objects whose tensors lie on another device than the current one, against a fake of
torch.cuda: the library is called with their device current, on a stream of that device."""
import contextlib

import pytest
import torch

from learnable_channel_permutation_b200 import binding as b

HOME, OTHER = 0, 3


@pytest.fixture
def calls(monkeypatch):
    """(entry point, current device, last argument) of every library call; raw streams are named 100 + device."""
    seen, state = [], dict(device=HOME)

    @contextlib.contextmanager
    def device(index):
        was, state["device"] = state["device"], index
        yield
        state["device"] = was

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, state["device"], a[-1])) or 0

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(b, "lib", Lib)
    return seen


def _make(cls, **attrs):
    x = object.__new__(cls)
    x.__dict__.update(attrs)
    return x


def _held(index):
    return _make(b._Held, index=index, tensors=[], known={100 + index}, made=None)


@pytest.mark.parametrize("index", [HOME, OTHER])
def test_steps_and_trainers_run_on_their_own_device(calls, index):
    buf = torch.zeros(4)
    step = _make(b.Step, _held=_held(index), hp=b.hparams(64, 2, 4, 5, 1.0, 0), n=1, arr=None, ws=buf)
    step.run()
    for max_norm in (None, 1.0):
        _make(b.Trainer, _held=_held(index), step=step, opt=b.adamw_params(), state=None, total=4, tau_start=1.0, tau_end=0.1,
              max_norm=max_norm, grad_norm=buf, ws=buf).run(0, 1)
    assert calls == [(name, index, 100 + index) for name in ("lcp_step", "lcp_train", "lcp_train_clip")]


def test_a_list_asks_for_its_workspace_on_its_own_device(calls):
    b._clip_workspace(3, OTHER)
    assert [c[:2] for c in calls] == [("lcp_clip_workspace_size", OTHER)]
