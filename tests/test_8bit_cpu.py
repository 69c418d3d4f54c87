"""Host side of the 8-bit operators and of the tensor lists: the oracle's definitions
against independent statements of them, and the refusals of every entry point
(argument checks come before anything touches a GPU)."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from learnable_channel_permutation_b200 import binding as b
from oracle import lcp_oracle as O

A = 0x10000000   # a fake, aligned device address (never dereferenced)

needs_lib = pytest.mark.skipif(not os.path.exists(b.LIB_PATH), reason="liblcp.so not built")


# ---- the oracle's definitions --------------------------------------------------

def test_e4m3_round_agrees_with_torch_on_values_ties_and_subnormals():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    every = np.unique(every[np.isfinite(every)])
    assert np.array_equal(O.e4m3_round(every), every)
    mids = (every[1:] + every[:-1]) / 2                       # every tie
    rng = np.random.default_rng(0)
    xs = np.concatenate([mids, rng.uniform(-448, 448, 4000), rng.normal(0, 0.01, 4000)]).astype(np.float32)
    want = torch.from_numpy(xs).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(O.e4m3_round(xs), want)


@pytest.mark.parametrize("amax,k", [(448.0, 0), (448.0001, 1), (224.0, -1), (1.75, -8), (1.7500001, -7), (1.0, -8),
                                    (3e38, 120), (2.0 ** -149, -127), (0.0, 0)])
def test_block_exponent(amax, k):
    assert O.block_exponent(amax) == k


def test_quantised_values_stay_within_half_a_step():
    rng = np.random.default_rng(1)
    X = rng.normal(size=(5, 320))
    perm = np.stack([rng.permutation(64) for _ in range(5)])
    q, s = O.quant8(X, perm)
    assert s.shape == (5, 3)
    back, want = O.dequant8(q, s, 1), O.gather_channels(X, perm)
    # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale below e4m3's normal range
    assert np.all(np.abs(back - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * np.repeat(s, 128, 1)[:, :320]))


def test_clip_factor():
    assert O.clip_factor(0.5, 1.0) == 1.0
    assert math.isclose(O.clip_factor(4.0, 1.0), 1.0 / 4.000001)
    assert O.clip_factor(float("inf"), 1.0) == 0.0
    assert math.isnan(O.clip_factor(float("nan"), 1.0))
    assert O.clip_factor(1e30, float("inf")) == 1.0


# ---- refusals ------------------------------------------------------------------

@needs_lib
def test_quant8_refusals():
    L = b.lib()
    call = lambda X=A, perm=None, Q=A, S=A, T=4, cin=128, B=0, dt=1: L.lcp_quant8(X, perm, Q, S, T, cin, B, dt, None)
    assert call(X=None) == 1 and call(Q=None) == 1 and call(S=None) == 1
    assert call(cin=100) == 2 and call(cin=0) == 2 and call(T=-1) == 2
    assert call(perm=A, B=48) == 2 and call(perm=A, B=64, cin=96) == 2 and call(perm=A, B=0) == 2
    assert call(dt=7) == 3
    assert call(X=A + 8) == 7 and call(Q=A + 4) == 7 and call(S=A + 1) == 7 and call(perm=A + 4, B=64) == 7
    assert call(T=0) == 0 and call(T=0, X=None, Q=None, S=None) == 0


@needs_lib
def test_quant8_weight_refusals():
    L = b.lib()
    call = lambda W=A, perm=None, mask=None, Q=A, S=A, cout=8, cin=128, B=0, dt=1: L.lcp_quant8_weight(
        W, perm, mask, Q, S, cout, cin, B, dt, None)
    assert call(W=None) == 1 and call(Q=None) == 1 and call(S=None) == 1
    assert call(cout=0) == 2 and call(cin=33) == 2 and call(perm=A, B=40) == 2 and call(perm=A, B=256) == 2
    assert call(cout=128 * 65535 + 1) == 2
    assert call(dt=9) == 3
    assert call(mask=A + 4) == 7


@needs_lib
def test_product_refusals():
    L = b.lib()
    mm = lambda Xq=A, Xs=A, Wq=A, Ws=A, Y=A, cout=8, cin=128, T=4, dt=0: L.lcp_mm8(Xq, Xs, Wq, Ws, Y, cout, cin, T, dt, None)
    assert mm(Xq=None) == 1 and mm(Ws=None) == 1 and mm(Y=None) == 1
    assert mm(cin=48) == 2 and mm(cout=0) == 2 and mm(T=-2) == 2
    assert mm(dt=2) == 3
    assert mm(Y=A + 8) == 7 and mm(Xq=A + 1) == 7
    assert mm(T=0) == 0
    n = ctypes.c_size_t(0)
    assert L.lcp_linear8_workspace_size(50, 160, ctypes.byref(n)) == 0 and n.value >= 50 * 160 + 50 * 2
    assert L.lcp_linear8_workspace_size(8, 160, ctypes.byref(n)) == 0 and n.value == 0
    assert L.lcp_linear8_workspace_size(5, 161, ctypes.byref(n)) == 2
    assert L.lcp_linear8_workspace_size(5, 160, None) == 1
    lin = lambda X=A, perm=None, Y=A, T=40, cin=128, B=0, dt=1, yt=0, ws=A, size=1 << 20: L.lcp_linear8(
        A, A, X, perm, Y, 8, cin, T, B, dt, yt, ws, size, None)
    assert lin(X=None) == 1 and lin(Y=None) == 1
    assert lin(cin=80) == 2 and lin(perm=A, B=12) == 2
    assert lin(dt=5) == 3 and lin(yt=5) == 3
    assert lin(ws=None) == 4 and lin(ws=A + 128) == 4 and lin(size=40 * 128 + 39) == 4
    assert lin(T=0, ws=None) == 0


@needs_lib
def test_list_refusals():
    L = b.lib()
    opt = b.adamw_params()
    n = ctypes.c_size_t(0)
    assert L.lcp_clip_workspace_size(3, ctypes.byref(n)) == 0 and n.value > 0
    need = n.value
    assert L.lcp_clip_workspace_size(-1, ctypes.byref(n)) == 2 and L.lcp_clip_workspace_size(3, None) == 1

    def grads(**kw):
        d = dict(g=A, out=A, n=10, dtype=0)
        d.update(kw)
        return (b.LcpGrad * 3)(b.LcpGrad(A + 4096, A + 4096, 7, 1), b.LcpGrad(d["g"], d["out"], d["n"], d["dtype"]),
                               b.LcpGrad(None, None, 0, 0))

    clip = lambda a=None, count=3, mx=1.0, norm=A, ws=A, size=need, **kw: L.lcp_grad_clip(
        a or grads(**kw), count, mx, norm, ws, size, None)
    norm = lambda **kw: L.lcp_grad_norm(grads(**kw), 3, A, A, need, None)
    assert clip(norm=None) == 1 and clip(norm=A + 2) == 7
    assert clip(g=None) == 1 and clip(out=None) == 1
    assert clip(n=-1) == 2 and clip(n=(1 << 40) + 1) == 2 and clip(count=-1) == 2
    assert clip(dtype=4) == 3
    assert clip(ws=None) == 4 and clip(size=need - 1) == 4 and clip(ws=A + 16) == 4
    assert clip(g=A + 2) == 7 and clip(g=A + 1, dtype=1) == 7 and clip(out=A + 1) == 7
    assert clip(mx=0.0) == 7 and clip(mx=-1.0) == 7 and clip(mx=float("nan")) == 7
    assert norm(g=None) == 1 and norm(dtype=4) == 3

    def tensors(**kw):
        d = dict(L=A, dL=A, m=A, v=A, n=10)
        d.update(kw)
        return (b.LcpAdamwTensor * 1)(b.LcpAdamwTensor(d["L"], d["dL"], d["m"], d["v"], d["n"]))

    upd = lambda t=1, mx=1.0, o=opt, size=need, **kw: L.lcp_adamw_list(
        tensors(**kw), 1, ctypes.byref(o), t, mx, A, A, size, None)
    assert upd(L=None) == 1 and upd(dL=None) == 1 and upd(v=None) == 1
    assert upd(n=-4) == 2
    assert upd(m=A + 2) == 7 and upd(t=0) == 7 and upd(mx=0.0) == 7 and upd(o=b.adamw_params(beta1=1.0)) == 7
    assert upd(size=8) == 4
    assert L.lcp_adamw_list(tensors(), 1, None, 1, 1.0, A, A, need, None) == 1


@needs_lib
def test_train_clip_refusals():
    L = b.lib()
    opt = b.adamw_params()
    hp = b.hparams(64, 2, 4, 5, 0.5, b.BF16)
    layer = (b.LcpLayer * 1)(b.LcpLayer(A, A, A, A, A, A, None, None, 64, 128, 32))
    st = (b.LcpAdamwState * 1)(b.LcpAdamwState(A, A))
    call = lambda mx=1.0, norm=A, ws=A, size=1 << 30, state=st, first=0: L.lcp_train_clip(
        layer, 1, ctypes.byref(hp), ctypes.byref(opt), state, first, 1, 4, 1.0, 0.1, mx, norm, ws, size, None)
    assert call(mx=0.0) == 7 and call(mx=float("nan")) == 7
    assert call(norm=None) == 1 and call(state=None) == 1
    assert call(ws=None) == 4 and call(size=16) == 4
    assert call(first=4) == 7


def test_overlapping_tensors_are_refused():
    with pytest.raises(ValueError):
        b._check_disjoint([(100, 8), (200, 4), (104, 8)])
    b._check_disjoint([(100, 4), (104, 8), (112, 0), (112, 4)])


def test_binding_refuses_what_is_not_on_a_gpu_or_has_the_wrong_shape():
    X = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        b.quant8(X)
    with pytest.raises(ValueError):
        b.quant8(X, torch.zeros(3, 64, dtype=torch.int32))
    Wq, Ws = torch.zeros(256, 128, dtype=torch.uint8).view(b.E4M3), torch.zeros(2, 1, dtype=torch.uint8).view(b.E8M0)
    Xq, Xs = torch.zeros(4, 128, dtype=torch.uint8).view(b.E4M3), torch.zeros(4, 1, dtype=torch.uint8).view(b.E8M0)
    with pytest.raises(ValueError):
        b.mm8(Xq, Xs, Wq, Ws)                       # CPU tensors
    with pytest.raises(ValueError):
        b.mm8(Xq, Xs, Wq, Ws[:1])                   # weight scales of another shape
    with pytest.raises(ValueError):
        b.mm8(Xq, Xs[:3], Wq, Ws)
    with pytest.raises(ValueError):
        b.linear8(Wq, Ws, torch.zeros(4, 96))
