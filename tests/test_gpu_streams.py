"""Prepared lists and trainers on streams other than the one they were made on, dropped while their calls are
still to run, captured, and replayed."""
import numpy as np
import pytest
import torch

from learnable_channel_permutation_b200 import binding as b
from learnable_channel_permutation_b200 import synth
from oracle import lcp_oracle as O

import gpu_helpers as H

pytestmark = pytest.mark.gpu

NORM_TOL = 2.0 ** -24 + 2.0 ** -26      # half a float32 step, and the float64 sums
BUSY = 100_000_000                      # cycles (about 50 ms) that keep a stream busy


def _grads(sizes, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(n, generator=g).cuda() for n in sizes]


def _fill_freed_memory(sizes):
    """New blocks of these byte counts on the current stream, overwritten."""
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    for x in blocks:
        x.fill_(0xff)
    return blocks


@pytest.mark.parametrize("sizes", [[3000, 7], [300001, 77, 64 * 64 * 64]])
@pytest.mark.parametrize("context", [False, True])
def test_a_list_dropped_while_its_call_is_queued(gpu_lib, sizes, context):
    """The workspace stays the call's own until it has run: nothing allocated meanwhile gets it."""
    ts = _grads(sizes, len(sizes))
    ref = [t.double().cpu().numpy() for t in ts]
    out = [torch.full_like(t, 9.0) for t in ts]
    norm = O.grad_norm(ref)
    side = torch.cuda.Stream()
    b.GradList(ts, out).clip(0.5 * norm)          # the kernels are loaded before the stream is kept busy
    for o in out:
        o.fill_(9.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    lst = b.GradList(ts, out)
    n_ws, at = lst.ws.numel(), lst.ws.data_ptr()
    if context:
        with torch.cuda.stream(side):
            got = lst.clip(0.5 * norm)
    else:
        got = lst.clip(0.5 * norm, stream=side)
    del lst
    blocks = _fill_freed_memory([n_ws, 4])
    assert not side.query(), "the stream was to be busy until here"
    assert all(x.data_ptr() != at for x in blocks)
    torch.cuda.synchronize()
    assert abs(float(got) - norm) <= NORM_TOL * norm
    f = O.clip_factor(norm, 0.5 * norm)
    for o, r in zip(out, ref):
        assert np.all(np.abs(o.double().cpu().numpy() - r * f) <= 2.0 ** -22 * np.abs(r * f))


def test_a_list_made_while_its_stream_is_busy(gpu_lib):
    """A call on an idle stream comes after what the buffers' memory was used for before."""
    ts = _grads([300001, 77], 3)
    norm = O.grad_norm([t.double().cpu().numpy() for t in ts])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n_ws = b.GradList(ts).ws.numel()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    del _fill_freed_memory([n_ws, 4])[:]          # queued behind the sleep, the blocks free for the host
    got = b.GradList(ts).norm(stream=side)
    torch.cuda.synchronize()
    assert abs(float(got) - norm) <= NORM_TOL * norm


def test_an_update_on_another_stream(gpu_lib):
    n, t = 70001, 5
    g = torch.Generator().manual_seed(1)
    state = [torch.randn(n, generator=g) * s for s in (1e-2, 1e-3, 1e-4, 1e-4)]
    state[3] = state[3].square()
    one, two = [[x.cuda() for x in state] for _ in range(2)]
    opt = b.adamw_params(lr=5e-3)
    want = b.AdamwList(*[[x] for x in one]).run(opt, t, 0.1).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = b.AdamwList(*[[x] for x in two]).run(opt, t, 0.1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(x, y) for x, y in zip(one, two))


def test_lists_captured_and_used_again(gpu_lib):
    """Captured calls of two lists, replayed on new gradients, and an eager call of the same list after that."""
    ts = [_grads([300001, 77], 4), _grads([64], 5)]
    outs = [[torch.empty_like(t) for t in x] for x in ts]
    lists = [b.GradList(t, o) for t, o in zip(ts, outs)]
    graphs, norms = [], []
    for lst in lists:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            norms.append(lst.clip(1.0))
        graphs.append(g)
    for seed in (6, 7):
        for x, y in zip(ts, (_grads([300001, 77], seed), _grads([64], seed))):
            for a, c in zip(x, y):
                a.copy_(c)
        for g, x, o, n in zip(graphs, ts, outs, norms):
            g.replay()
            torch.cuda.synchronize()
            want = O.grad_norm([t.double().cpu().numpy() for t in x])
            f = O.clip_factor(want, 1.0)
            assert abs(float(n) - want) <= NORM_TOL * want
            for a, c in zip(o, x):
                r = c.double().cpu().numpy() * f
                assert np.all(np.abs(a.double().cpu().numpy() - r) <= 2.0 ** -22 * np.abs(r))
    got = lists[0].norm()
    torch.cuda.synchronize()
    want = O.grad_norm([t.double().cpu().numpy() for t in ts[0]])
    assert abs(float(got) - want) <= NORM_TOL * want


def _trainer(max_norm):
    layers = []
    for s in (3, 4):
        wl = synth.custom(256, 512, 192, 64, 2, 4, 1.0, 5, "bf16", seed=s, outliers=True)
        W, X, L = H.to_dev(synth.make_inputs(wl)[0], "bf16")
        layers.append(b.alloc_outputs(W, X, L))
    return layers, b.Trainer(b.Step(layers, 64, 2, 4, 5, 1.0), b.adamw_params(lr=5e-3), 4, max_norm=max_norm)


@pytest.mark.parametrize("max_norm", [None, 1e-4])
def test_a_trainer_dropped_while_its_steps_are_queued(gpu_lib, max_norm):
    """Made behind queued work, run on another stream, dropped at once: the logits of a run on one stream."""
    want, tr = _trainer(max_norm)
    tr.run(0, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(BUSY)
    layers, tr = _trainer(max_norm)
    sizes = [tr.step.ws.numel(), tr.ws.numel()] + [m.numel() * 4 for pair in tr.moments for m in pair]
    tr.run(0, 4, stream=side)
    del tr
    _fill_freed_memory(sizes)
    torch.cuda.synchronize()
    assert all(torch.equal(x["L"], y["L"]) and torch.equal(x["dL"], y["dL"]) for x, y in zip(want, layers))
    assert b.device_error() == 0
