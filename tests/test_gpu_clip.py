"""The gradient norm over many tensors, clipping by it, and the AdamW update of a
list, GPU against float64.

The squares and their sum are float64 and the norm is rounded once, so it is
within half a float32 step (2^-24) of the exact norm; float64 summation of up to
2^27 values adds at most 2^27 2^-53.  The factor is rounded once and each
clipped gradient once more: 2 x 2^-24 of the value in float32, half a bf16 step
(2^-8) more in bf16.
"""
import numpy as np
import pytest
import torch

from learnable_channel_permutation_b200 import binding as b
from learnable_channel_permutation_b200 import synth
from oracle import lcp_oracle as O

import gpu_helpers as H

pytestmark = pytest.mark.gpu

NORM_TOL = 2.0 ** -24 + 2.0 ** -26


def _tensors(sizes, seed, dtypes=(torch.float32,), scale=1.0, offset=0):
    """Tensors one after another in a buffer each dtype, `offset` values from an aligned start: most are not 16-byte aligned."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for dt in dtypes:
        flat = torch.empty(offset + sum(sizes), dtype=dt, device="cuda")
        flat.copy_(torch.randn(flat.numel(), generator=g) * scale)
        out += list(flat[offset:].split(sizes))
    return out


def _f64(ts):
    return [t.double().cpu().numpy() for t in ts]


SIZES = [[1], [5], [4096], [8191, 8192, 8193], [0, 3, 0, 16384, 1], [100000, 7, 64 * 64 * 64], [1023] * 40]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtypes", [(torch.float32,), (torch.bfloat16,), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("offset", [0, 1])
def test_norm_and_clip(gpu_lib, sizes, dtypes, offset):
    ts = _tensors(sizes, len(sizes) + offset, dtypes, offset=offset)
    ref = _f64(ts)
    norm = O.grad_norm(ref)
    for max_norm in (0.5 * norm, 2.0 * norm, float("inf")):
        out = [torch.full_like(t, 9.0) for t in ts]
        lst = b.GradList(ts, out)
        n0 = float(lst.norm())
        n1 = float(lst.clip(max_norm))
        assert n0 == n1 and abs(n1 - norm) <= NORM_TOL * norm
        f = O.clip_factor(norm, max_norm)
        for t, o, r in zip(ts, out, ref):
            if f == 1.0:
                assert torch.equal(o, t)
                continue
            want = r * f
            half = 2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0
            # (2 x 2^-24 and the norm's own error are inside 2^-22)
            assert np.all(np.abs(o.double().cpu().numpy() - want) <= (half * (1 + 2.0 ** -20) + 2.0 ** -22) * np.abs(want) + 1e-40)


def test_clip_in_place_and_out_of_place_agree(gpu_lib):
    a = _tensors([5000, 33, 70000], 3, offset=3)
    c = [t.clone() for t in a]                    # another alignment
    out = [torch.empty_like(t) for t in a]
    n = b.GradList(a, out).clip(1.0).clone()
    m = b.GradList(c).clip(1.0)
    assert torch.equal(n, m) and all(torch.equal(x, y) for x, y in zip(out, c))


def test_outputs_stay_inside_their_tensors(gpu_lib):
    flat = torch.full((20011,), 3.0, device="cuda")
    b.GradList([flat[5:10002], flat[10007:20000]]).clip(1.0)
    assert torch.all(flat[:5] == 3.0) and torch.all(flat[10002:10007] == 3.0) and torch.all(flat[20000:] == 3.0)
    assert torch.all(flat[5:10002] < 1.0) and torch.all(flat[10007:20000] < 1.0)


@pytest.mark.parametrize("sizes", [[70], [65536], [65537], [64 * 64 * 64], [700001], [4096] * 16, [4097] * 16, [9] * 17,
                                   [100] * 80, [100] * 81, [30011] * 90])
def test_every_way_a_list_is_cut(gpu_lib, sizes):
    """Both sides of each border between the launches' forms, in place, with a workspace full of garbage."""
    ts = _tensors(sizes, sum(sizes))
    ref = _f64(ts)
    norm = O.grad_norm(ref)
    lst = b.GradList(ts)
    lst.ws.fill_(0xff)
    assert abs(float(lst.norm()) - norm) <= NORM_TOL * norm
    lst.ws.fill_(0xff)
    assert abs(float(lst.clip(0.5 * norm)) - norm) <= NORM_TOL * norm
    f = O.clip_factor(norm, 0.5 * norm)
    for t, r in zip(ts, ref):
        assert np.all(np.abs(t.double().cpu().numpy() - r * f) <= 2.0 ** -22 * np.abs(r * f))
    L, g, m, v = _adam_state(sizes, 2, 4)
    Lr = [O.adamw_update(*[x[i].double().cpu().numpy() for x in (L, g, m, v)], 4, lr=1e-3) for i in range(len(sizes))]
    before = [x.double().cpu().numpy() for x in L]
    b.AdamwList(L, g, m, v).run(b.adamw_params(lr=1e-3), 4)
    for i in range(len(sizes)):
        assert H.relerr(m[i].cpu().numpy(), Lr[i][1]) <= 1e-6 and H.relerr(v[i].cpu().numpy(), Lr[i][2]) <= 1e-6
        assert H.relerr(L[i].double().cpu().numpy() - before[i], Lr[i][0] - before[i]) <= 1e-4


def test_more_tensors_than_one_launch_takes(gpu_lib):
    ts = _tensors([17 + i % 9 for i in range(1500)], 8)
    norm = O.grad_norm(_f64(ts))
    lst = b.GradList(ts)
    assert abs(float(lst.clip(0.25 * norm)) - norm) <= NORM_TOL * norm
    assert abs(float(lst.norm()) - 0.25 * norm) <= 1e-5 * norm


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_is_passed_on(gpu_lib, value):
    ts = [torch.ones(1000, device="cuda"), torch.ones(3, dtype=torch.bfloat16, device="cuda")]
    ts[0][77] = value
    n = float(b.GradList(ts).clip(1.0))
    if value != value:
        assert np.isnan(n) and all(bool(t.isnan().all()) for t in ts)
    else:
        assert n == float("inf") and bool(ts[0][77].isnan()) and float(ts[0].nansum()) == 0 and float(ts[1].sum()) == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("n", [1000, 300000])
def test_no_limit_leaves_the_other_values_as_they_are(gpu_lib, value, n):
    """An infinite max_norm asks for no clipping, whatever the norm: the bad value stays the only one."""
    g = torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda()
    g[77] = value
    small = torch.ones(3, dtype=torch.bfloat16, device="cuda")
    out = [torch.zeros_like(g), torch.zeros_like(small)]
    norm = float(b.GradList([g, small], out).clip(float("inf")))
    assert not np.isfinite(norm)
    keep = torch.arange(n, device="cuda") != 77
    assert torch.equal(out[0][keep], g[keep]) and torch.equal(out[1], small) and not bool(out[0][77].isfinite())
    opt = b.adamw_params()
    one, other = [[torch.ones(n, device="cuda"), g.clone(), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")]
                  for _ in range(2)]
    b.AdamwList(*[[t] for t in one]).run(opt, 1)
    b.adamw(other[0], other[1], other[2], other[3], opt, 1)
    for x, y in zip(one, other):
        assert torch.equal(x[keep], y[keep])


@pytest.mark.parametrize("scale", [1e30, 1e-30, 1e-42])
def test_squares_neither_overflow_nor_vanish(gpu_lib, scale):
    ts = [torch.full((4099,), scale, device="cuda")]
    ref = _f64(ts)
    norm = O.grad_norm(ref)
    # below float32's normal range half a step is 2^-150 whatever the value
    assert abs(float(b.GradList(ts).norm()) - norm) <= NORM_TOL * norm + 2.0 ** -149


def test_empty_lists(gpu_lib):
    assert float(b.GradList([]).clip(1.0)) == 0.0
    assert float(b.GradList([torch.empty(0, device="cuda")]).norm()) == 0.0
    assert float(b.AdamwList([], [], [], []).run(b.adamw_params(), 1, 1.0)) == 0.0


def test_lists_refuse_overlaps_and_mismatches(gpu_lib):
    x = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError):
        b.GradList([x, x])
    with pytest.raises(ValueError):
        b.GradList([x[:40]], [x[20:60]])
    with pytest.raises(ValueError):
        b.GradList([x], [torch.zeros(63, device="cuda")])
    with pytest.raises(ValueError):
        b.GradList([x.view(8, 8).t()])
    with pytest.raises(ValueError):
        b.AdamwList([x], [x], [x.clone()], [x.clone()])
    with pytest.raises(TypeError):
        b.GradList([x.half()])
    with pytest.raises(b.LcpError):
        b.GradList([x]).clip(0.0)


def test_results_do_not_depend_on_timing(gpu_lib):
    ts = _tensors([300001, 77, 4096 * 64], 5)
    lst = b.GradList(ts, [torch.empty_like(t) for t in ts])
    first = lst.clip(1.0).clone()
    for _ in range(5):
        assert torch.equal(lst.clip(1.0), first)


# ---- AdamW of a list ------------------------------------------------------------

def _adam_state(sizes, seed, t, offset=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda s: torch.randn(offset + sum(sizes), generator=g) * s
    bufs = [rnd(1e-2), rnd(1e-3), rnd(1e-4) * (t > 1), rnd(1e-4).square() * (t > 1)]
    return [list(x.float().cuda()[offset:].split(sizes)) for x in bufs]


@pytest.mark.parametrize("t", [1, 9])
def test_adamw_list_without_clipping_is_adamw(gpu_lib, t):
    sizes = [64 * 64, 8192 * 3 + 4, 128]
    one, many = _adam_state(sizes, 1, t), _adam_state(sizes, 1, t)
    opt = b.adamw_params(lr=5e-3)
    for x in zip(*one):
        b.adamw(*x, opt, t)
    norm = O.grad_norm(_f64(many[1]))
    assert abs(float(b.AdamwList(*many).run(opt, t)) - norm) <= NORM_TOL * norm
    assert all(torch.equal(x, y) for a, c in zip(one, many) for x, y in zip(a, c))


@pytest.mark.parametrize("sizes", [[1], [64 * 64 * 64], [8191, 8193, 2], [1001] * 30])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("limit", [0.1, 10.0])
def test_adamw_list_clips(gpu_lib, sizes, offset, limit):
    t = 3
    L, g, m, v = _adam_state(sizes, 7, t, offset)
    ref = [_f64(x) for x in (L, g, m, v)]
    before = [x.clone() for x in g]
    norm = O.grad_norm(ref[1])
    opt = b.adamw_params(lr=5e-3)
    got = float(b.AdamwList(L, g, m, v).run(opt, t, limit * norm))
    assert abs(got - norm) <= NORM_TOL * norm
    assert all(torch.equal(x, y) for x, y in zip(g, before))             # the gradients stay
    f = O.clip_factor(norm, limit * norm)
    for i in range(len(sizes)):
        Lr, mr, vr = O.adamw_update(ref[0][i], ref[1][i] * f, ref[2][i], ref[3][i], t, lr=5e-3)
        # the tolerances of the one-layer update (float32 throughout)
        assert H.relerr(m[i].cpu().numpy(), mr) <= 1e-6
        assert H.relerr(v[i].cpu().numpy(), vr) <= 1e-6
        assert H.relerr(L[i].double().cpu().numpy() - ref[0][i], Lr - ref[0][i]) <= 1e-4


def test_adamw_list_mixed_alignments(gpu_lib):
    """L, dL, m and v of one tensor on different 16-byte phases: the same result as aligned ones."""
    n = 20000
    aligned = _adam_state([n], 4, 2)
    shifted = [[torch.empty(n + k, device="cuda")[k:].copy_(x[0])] for k, x in zip((0, 1, 2, 3), aligned)]
    opt = b.adamw_params()
    a, c = b.AdamwList(*aligned).run(opt, 2, 1e-3).clone(), b.AdamwList(*shifted).run(opt, 2, 1e-3)
    assert abs(float(a) - float(c)) <= 2 * NORM_TOL * float(a)
    for x, y in zip(aligned, shifted):
        assert H.relerr(y[0].cpu().numpy(), x[0].cpu().numpy()) <= 1e-6


# ---- training with clipping ------------------------------------------------------

def _trainer(total, max_norm, seeds=(3, 4)):
    layers = []
    for s in seeds:
        wl = synth.custom(256, 512, 192, 64, 2, 4, 1.0, 5, "bf16", seed=s, outliers=True)
        W, X, L = H.to_dev(synth.make_inputs(wl)[0], "bf16")
        layers.append(b.alloc_outputs(W, X, L))
    step = b.Step(layers, 64, 2, 4, 5, 1.0)
    return layers, b.Trainer(step, b.adamw_params(lr=5e-3), total, max_norm=max_norm)


def test_train_without_reaching_the_limit_is_plain_training(gpu_lib):
    plain, tp = _trainer(4, None)
    clipped, tc = _trainer(4, 1e9)
    tp.run(0, 4)
    tc.run(0, 4)
    for a, c in zip(plain, clipped):
        assert torch.equal(a["L"], c["L"]) and torch.equal(a["dL"], c["dL"])


def test_train_steps_clip_all_layers_together(gpu_lib):
    """Step by step: the norm is that of both layers' dL, and the update is AdamW of the clipped gradients."""
    layers, tr = _trainer(3, 1e-4)
    L = [d["L"].double().cpu().numpy() for d in layers]
    mom = [(np.zeros_like(x), np.zeros_like(x)) for x in L]
    for s in range(3):
        tr.run(s, 1)
        torch.cuda.synchronize()
        g = [d["dL"].double().cpu().numpy() for d in layers]
        norm = O.grad_norm(g)
        assert abs(float(tr.grad_norm) - norm) <= NORM_TOL * norm
        f = O.clip_factor(norm, 1e-4)
        assert f < 1.0
        for i, d in enumerate(layers):
            nxt, m, v = O.adamw_update(L[i], g[i] * f, *mom[i], s + 1, lr=5e-3)
            got = d["L"].double().cpu().numpy()
            assert H.relerr(got - L[i], nxt - L[i]) <= 1e-4
            L[i], mom[i] = got, (m, v)
    assert b.device_error() == 0


def test_captured_training_steps(gpu_lib):
    """A captured clipped step replayed gives what the eager call gives; a graph holds its own list."""
    eager, te = _trainer(5, 1e-4)
    cap, tc = _trainer(5, 1e-4)
    te.run(0, 1)
    tc.run(0, 1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tc.run(1, 2)
    te.run(1, 2)
    g.replay()
    torch.cuda.synchronize()
    for a, c in zip(eager, cap):
        assert torch.equal(a["L"], c["L"])
    assert torch.equal(te.grad_norm, tc.grad_norm)
