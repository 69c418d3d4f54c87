"""8-bit operands and their product on the GPU against the float64 oracle.

Quantisation makes one rounding, to e4m3, of a value whose exponent alone was
moved, so values and scales are compared bit for bit.  The product adds exact
products of e4m3 values times powers of two in float32: C_in / 32 steps of the
tensor cores, each adding 32 products to the accumulator, and the partial sums of
up to eight CTAs.  With one unit in the last place (2^-23: the alignment inside a
step may truncate) of the sum of the terms' magnitudes for each of the C_in / 32 +
32 + 8 additions a term goes through, an output is within
(C_in / 32 + 40) 2^-23 sum |terms| of the exact value, and a bf16 output half a
step of bf16 (2^-8 of it) more.
"""
import numpy as np
import pytest
import torch

from learnable_channel_permutation_b200 import binding as b
from learnable_channel_permutation_b200 import synth
from oracle import lcp_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _perm(rng, cin, B):
    return np.stack([rng.permutation(B) for _ in range(cin // B)]) if B else None


def _dev_perm(perm):
    return None if perm is None else torch.from_numpy(np.ascontiguousarray(perm, np.int32)).cuda()


def _same(got, want):
    return np.array_equal(got, want, equal_nan=True)


def _rows(rng, T, cin, dtype):
    """Tokens of very different sizes, with zeros, a zero group and outlier channels."""
    X = rng.normal(size=(T, cin)) * np.exp2(rng.integers(-20, 20, size=(T, 1)))
    X[:, rng.choice(cin, max(1, cin // 50), replace=False)] *= 30
    X[rng.random((T, cin)) < 0.05] = 0
    X[0, :128] = 0
    return torch.from_numpy(X).to(DT[dtype])


# ---- quantisation -------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,cin,B", [(1, 32, 0), (1, 128, 128), (3, 160, 32), (7, 416, 0), (5, 512, 64), (33, 1120, 32),
                                     (2, 768, 256), (130, 4096, 64), (17, 11008, 64)])
def test_quant8_matches_the_oracle_bit_for_bit(gpu_lib, dtype, T, cin, B):
    rng = np.random.default_rng(T + cin + B)
    X = _rows(rng, T, cin, dtype)
    perm = _perm(rng, cin, B)
    q, s = b.quant8(X.cuda(), _dev_perm(perm))
    rq, rs = O.quant8(_np(X), perm)
    assert _same(_np(q), rq) and _same(_np(s), rs)
    assert b.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quant8_edges(gpu_lib, dtype):
    """Borders of a scale, ties, the largest and smallest magnitudes, negative zero, infinities and NaN."""
    fi = torch.finfo(DT[dtype])
    X = torch.zeros(12, 256, dtype=torch.float64)
    X[0, 3] = 448.0
    X[1, 3] = 450.0                             # just above: the next scale
    X[2, :32] = torch.arange(32) * 0.5 + 1      # many ties of e4m3 at scale 2^-4 .. 2^-5
    X[3, 7], X[3, 8] = fi.max, -fi.max
    X[4, 9] = fi.tiny
    X[4, 10] = -fi.tiny / 2 if dtype == "f32" else -fi.tiny
    X[5, 100], X[5, 130] = float("inf"), 2.0    # only the first group is lost
    X[6, 200] = float("nan")
    X[7, 5] = -0.0
    X[8] = 1e-6 * torch.arange(256)
    X[9, ::2], X[9, 1::2] = 1.0, 2.0 ** -9      # the subnormal end of a block
    X[10, 128:] = 5e-39 if dtype == "f32" else 2e-38
    X[11, 40] = -float("inf")
    X = X.to(DT[dtype])
    q, s = b.quant8(X.cuda())
    rq, rs = O.quant8(_np(X))
    assert _same(_np(q), rq) and _same(_np(s), rs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cout,cin,B,n,m", [(8, 32, 0, 0, 0), (1, 128, 32, 2, 4), (130, 160, 32, 4, 8), (200, 1120, 0, 1, 4),
                                            (129, 512, 256, 2, 4), (300, 1024, 64, 0, 0), (256, 640, 128, 8, 8)])
def test_quant8_weight_matches_the_oracle_bit_for_bit(gpu_lib, dtype, cout, cin, B, n, m):
    rng = np.random.default_rng(cout + cin + n)
    W = rng.normal(0, 0.02, (cout, cin)) * np.exp2(rng.integers(-6, 6, size=(1, cin)))
    W = torch.from_numpy(W).to(DT[dtype])
    perm = _perm(rng, cin, B)
    W64 = _np(W)
    M = O.nm_mask(W64 if perm is None else O.gather_channels(W64, perm), n, m) if m else None
    bits = None if M is None else torch.from_numpy(O.pack_mask_bits(M).view(np.int32)).cuda()
    q, s = b.quant8_weight(W.cuda(), _dev_perm(perm), bits)
    rq, rs = O.quant8_weight(W64, perm, M)
    assert _same(_np(q), rq) and _same(_np(s), rs)
    assert b.device_error() == 0


def test_quant8_weight_ignores_what_the_mask_drops(gpu_lib):
    """Infinities and NaN under the mask leave no trace; a mask that keeps nothing of a block leaves zeros."""
    rng = np.random.default_rng(4)
    W = rng.normal(size=(256, 256))
    M = rng.random((256, 256)) < 0.5
    M[:128, 128:] = False
    W[~M] = rng.choice([np.inf, -np.inf, np.nan, 1e30], size=int((~M).sum()))
    W = torch.from_numpy(W).to(torch.bfloat16)
    q, s = b.quant8_weight(W.cuda(), None, torch.from_numpy(O.pack_mask_bits(M).view(np.int32)).cuda())
    rq, rs = O.quant8_weight(_np(W), None, M)
    assert np.all(np.isfinite(rq)) and rs[0, 1] == 1.0
    assert _same(_np(q), rq) and _same(_np(s), rs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [0, 64, 256])
def test_subnormal_blocks(gpu_lib, dtype, B):
    """Blocks whose every value is subnormal in the input's type, beside blocks that hold one normal value."""
    rng = np.random.default_rng(B + 3)
    tiny = torch.finfo(DT[dtype]).tiny
    X = torch.from_numpy(rng.uniform(-1, 1, (140, 512)) * tiny * 0.99).to(DT[dtype])
    X[::3, 300] = 2.0 * tiny
    X[::5, 100] = 1.0
    perm = _perm(rng, 512, B)
    for q, s, rq, rs in ((*b.quant8(X.cuda(), _dev_perm(perm)), *O.quant8(_np(X), perm)),
                         (*b.quant8_weight(X.cuda(), _dev_perm(perm)), *O.quant8_weight(_np(X), perm))):
        assert _same(_np(q), rq) and _same(_np(s), rs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,cin,B", [(231, 11040, 32), (300, 11072, 64), (451, 11136, 128), (215, 13824, 256)])
def test_quant8_many_tokens_a_warp(gpu_lib, dtype, T, cin, B):
    """Several rounds of four tokens, the last one not whole, with infinities and NaN in some groups."""
    rng = np.random.default_rng(T + cin)
    X = _rows(rng, T, cin, dtype)
    X[5, 700], X[T - 1, cin - 1], X[T // 2, 40] = float("inf"), float("nan"), -float("inf")
    perm = _perm(rng, cin, B)
    q, s = b.quant8(X.cuda(), _dev_perm(perm))
    rq, rs = O.quant8(_np(X), perm)
    assert _same(_np(q), rq) and _same(_np(s), rs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cout,cin,B", [(255, 1184, 32), (385, 1216, 64), (129, 1408, 128), (130, 512, 256), (3, 32, 32)])
def test_quant8_weight_any_mask_under_a_permutation(gpu_lib, dtype, cout, cin, B):
    """Masks of no pattern, whole rows and blocks dropped, infinities and NaN in dropped and in kept places."""
    rng = np.random.default_rng(cout + cin)
    perm = _perm(rng, cin, B)
    A = rng.normal(size=(cout, cin)) * np.exp2(rng.integers(-6, 6, size=(1, cin)))
    M = rng.random((cout, cin)) < rng.random((cout, 1))
    M[cout // 2] = False
    M[:128, :32] = False
    A[~M] = rng.choice([np.inf, -np.inf, np.nan, 1e30, 1.0], size=int((~M).sum()))
    if cout > 128:
        A[-1, -1], M[-1, -1] = np.inf, True
    W = torch.from_numpy(O.gather_channels(A, np.argsort(perm, axis=1))).to(DT[dtype])       # A = W P_B
    q, s = b.quant8_weight(W.cuda(), _dev_perm(perm), torch.from_numpy(O.pack_mask_bits(M).view(np.int32)).cuda())
    rq, rs = O.quant8_weight(_np(W), perm, M)
    assert _same(_np(q), rq) and _same(_np(s), rs)
    assert np.isnan(rs).sum() == (1 if cout > 128 else 0)


def test_quant8_reports_an_invalid_permutation_entry(gpu_lib):
    perm = torch.arange(32, dtype=torch.int32).repeat(4, 1).cuda()
    perm[2, 5] = 32
    b.quant8(torch.zeros(3, 128, device="cuda"), perm)
    assert b.device_error() == 302
    perm[2, 5] = -1
    b.quant8_weight(torch.zeros(8, 128, device="cuda"), perm)
    assert b.device_error() == 302
    assert b.device_error() == 0


def test_outputs_stay_inside_their_buffers(gpu_lib):
    """Rows before and behind the ones of the call are left as they were."""
    rng = np.random.default_rng(5)
    T, cin, cout = 5, 160, 72
    X = torch.from_numpy(rng.normal(size=(T, cin))).float().cuda()
    q = torch.full((T + 2, cin), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.full((T + 30, 2), 0x11, dtype=torch.uint8, device="cuda")
    b.quant8(X, None, q[1:-1].view(b.E4M3), s[8:8 + T].view(b.E8M0))
    assert torch.all(q[0] == 0x11) and torch.all(q[-1] == 0x11)
    assert torch.all(s[:8] == 0x11) and torch.all(s[8 + T:] == 0x11)
    Wq, Ws = b.quant8_weight(torch.from_numpy(rng.normal(size=(cout, cin))).float().cuda())
    for tokens in (T, 150):
        Xq, Xs = b.quant8(torch.randn(tokens, cin, device="cuda"))
        for dt in (torch.float32, torch.bfloat16):
            Y = torch.full((tokens + 2, cout), 7.0, dtype=dt, device="cuda")
            b.mm8(Xq, Xs, Wq, Ws, Y[1:-1])
            assert torch.all(Y[0] == 7.0) and torch.all(Y[-1] == 7.0)


# ---- the product --------------------------------------------------------------

def _operand(rng, rows, cin, scale_rows):
    q = torch.from_numpy(rng.normal(0, 110, (rows, cin))).clamp(-448, 448).to(b.E4M3)
    s = torch.from_numpy(rng.integers(115, 128, (scale_rows, -(-cin // 128))).astype(np.uint8)).view(b.E8M0)
    return q, s


def _check(Y, xq, xs, wq, ws, tag=""):
    cin = xq.shape[1]
    x, w = O.dequant8(_np(xq), _np(xs), 1), O.dequant8(_np(wq), _np(ws), 128)
    ref, terms = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = (cin / 32 + 40) * 2.0 ** -23 * terms
    if Y.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(_np(Y) - ref)
    assert np.all(err <= tol + 1e-300), (tag, float(np.max(err / (tol + 1e-300))))


def _product(rng, T, cin, cout, dt=torch.float32):
    xq, xs = _operand(rng, T, cin, T)
    wq, ws = _operand(rng, cout, cin, -(-cout // 128))
    Y = b.mm8(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), out_dtype=dt)
    torch.cuda.synchronize()
    assert b.device_error() == 0, "a bounded wait inside the product expired"
    return Y, xq, xs, wq, ws


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 100, 127, 128, 129, 200, 256, 333, 512])
@pytest.mark.parametrize("cin,cout", [(256, 136), (1120, 264)])
def test_mm8_token_counts(gpu_lib, T, cin, cout):
    _check(*_product(np.random.default_rng(T + cin), T, cin, cout))


@pytest.mark.parametrize("cin", [32, 64, 96, 128, 160, 480, 544, 640, 1000 // 32 * 32, 4096, 5152, 11008, 13824])
@pytest.mark.parametrize("T,cout", [(1, 40), (20, 129), (300, 384)])
def test_mm8_channel_counts(gpu_lib, cin, T, cout):
    _check(*_product(np.random.default_rng(T + cin), T, cin, cout))


@pytest.mark.parametrize("cout", [1, 7, 8, 127, 128, 130, 511, 4097])
@pytest.mark.parametrize("T", [3, 260])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_mm8_output_widths_and_types(gpu_lib, cout, T, dt):
    _check(*_product(np.random.default_rng(cout + T), T, 672, cout, dt))


@pytest.mark.parametrize("T", [1, 40, 1000])
def test_mm8_many_tiles(gpu_lib, T):
    """More tiles than the GPU has SMs, several rounds of each CTA."""
    _check(*_product(np.random.default_rng(T), T, 1024, 11008, torch.bfloat16))


@pytest.mark.parametrize("T,cin,cout", [(150, 33024, 136), (20, 40000, 72), (5000, 96, 8), (3, 32, 19000), (1, 32768 * 4, 130)])
def test_mm8_long_and_narrow(gpu_lib, T, cin, cout):
    """More channels than a tile's scales are staged for, many tokens of few channels, many outputs of one group."""
    _check(*_product(np.random.default_rng(T + cin), T, cin, cout))


def test_mm8_scales_of_every_row_and_group(gpu_lib):
    """One nonzero value a row at a time, with scales that name the row and the group."""
    T, cin, cout = 300, 1408, 400
    G = cin // 128
    q = torch.zeros(T, cin)
    q[torch.arange(T), (torch.arange(T) * 37) % cin] = 1.0
    xs = ((torch.arange(T)[:, None] * 5 + torch.arange(G)[None] * 3) % 40 + 100).to(torch.uint8)
    w = torch.ones(cout, cin)
    ws = ((torch.arange(4)[:, None] * 11 + torch.arange(G)[None] * 7) % 30 + 110).to(torch.uint8)
    args = (q.to(b.E4M3), xs.view(b.E8M0), w.to(b.E4M3), ws.view(b.E8M0))
    for rows in (slice(0, T), slice(0, 5), slice(40, 130)):
        sub = (args[0][rows].contiguous(), args[1][rows].contiguous(), args[2], args[3])
        Y = b.mm8(*[t.cuda() for t in sub])
        want = O.mm8(*[_np(t) for t in sub])
        assert np.array_equal(_np(Y), want)            # one power of two an output: exact


@pytest.mark.parametrize("T", [4, 200])
def test_mm8_nan_and_extreme_scales(gpu_lib, T):
    """A NaN scale or value makes its token's (its 128 channels') outputs NaN and no other; the ends of the scales' range
    cancel."""
    rng = np.random.default_rng(T)
    xq, xs = _operand(rng, T, 384, T)
    wq, ws = _operand(rng, 300, 384, 3)
    xs = xs.view(torch.uint8).clone()
    ws = ws.view(torch.uint8).clone()
    xs[0], ws[0] = 254, 1
    xs[1], ws[1] = 3, 250
    xs[2, 1] = 255
    qb = xq.view(torch.uint8).clone()
    qb[3, 17] = 0x7f
    wb = wq.view(torch.uint8).clone()
    wb[290, 383] = 0xff
    Y = _np(b.mm8(qb.view(b.E4M3).cuda(), xs.view(b.E8M0).cuda(), wb.view(b.E4M3).cuda(), ws.view(b.E8M0).cuda()))
    nan = np.isnan(Y)
    assert nan[2].all() and nan[3].all() and nan[:, 290].all()
    rest = np.ones_like(nan)
    rest[[2, 3]] = False
    rest[:, 290] = False
    assert not nan[rest].any()
    x, w = O.dequant8(_np(qb.view(b.E4M3)), _np(xs.view(b.E8M0)), 1), O.dequant8(_np(wb.view(b.E4M3)), _np(ws.view(b.E8M0)), 128)
    with np.errstate(invalid="ignore", over="ignore"):
        ref, terms = x @ w.T, np.abs(x) @ np.abs(w).T
    fit = rest & (terms < 1e38)                       # what float32 can hold
    assert fit.sum() > 0.3 * rest.sum()
    assert np.all(np.abs(Y - ref)[fit] <= ((12 + 40) * 2.0 ** -23 * terms + 1e-44)[fit])


# ---- the layer ----------------------------------------------------------------

@pytest.mark.parametrize("xdt", ["bf16", "f32"])
@pytest.mark.parametrize("T,cin,cout,B", [(1, 4096, 512, 64), (5, 160, 40, 32), (33, 1024, 200, 256), (300, 2048, 264, 128),
                                          (64, 480, 1000, 0)])
def test_linear8_is_the_quantiser_and_the_product(gpu_lib, xdt, T, cin, cout, B):
    rng = np.random.default_rng(T + cin)
    X = _rows(rng, T, cin, xdt).cuda()
    perm = _dev_perm(_perm(rng, cin, B))
    wq, ws = (t.cuda() for t in _operand(rng, cout, cin, -(-cout // 128)))
    for dt in (torch.float32, torch.bfloat16):
        Y = b.linear8(wq, ws, X, perm, out_dtype=dt)
        q, s = b.quant8(X, perm)
        assert torch.equal(Y, b.mm8(q, s, wq, ws, out_dtype=dt))
        _check(Y, q, s, wq, ws)
    assert b.device_error() == 0


@pytest.mark.parametrize("T", [1, 2, 3, 6, 9, 16, 19, 33, 64])
@pytest.mark.parametrize("cin,cout,B", [(4096, 11008, 64), (2272, 19200, 32), (13824, 640, 256)])
def test_linear8_few_tokens_over_many_groups(gpu_lib, T, cin, cout, B):
    """Ranges of channels several times the ring's length in one CTA, for every number of token pairs."""
    rng = np.random.default_rng(T + cout)
    X = _rows(rng, T, cin, "bf16").cuda()
    perm = _dev_perm(_perm(rng, cin, B))
    wq, ws = (t.cuda() for t in _operand(rng, cout, cin, -(-cout // 128)))
    Y = b.linear8(wq, ws, X, perm)
    q, s = b.quant8(X, perm)
    assert torch.equal(Y, b.mm8(q, s, wq, ws))
    assert b.device_error() == 0
    rows = np.unique(np.concatenate([np.arange(0, cout, 37), [cout - 1]]))
    sel = torch.from_numpy(rows).cuda()
    w = _np(wq.view(torch.uint8)[sel].view(b.E4M3)) * np.repeat(_np(ws), 128, 1)[rows // 128][:, :cin]
    x = O.dequant8(_np(q), _np(s), 1)
    assert np.all(np.abs(_np(Y)[:, rows] - x @ w.T) <= (cin / 32 + 40) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T))


def test_no_tokens(gpu_lib):
    wq, ws = (t.cuda() for t in _operand(np.random.default_rng(0), 40, 128, 1))
    X = torch.empty(0, 128, device="cuda")
    q, s = b.quant8(X)
    assert q.shape == (0, 128) and s.shape == (0, 1)
    assert b.mm8(q, s, wq, ws).shape == (0, 40)
    assert b.linear8(wq, ws, X).shape == (0, 40)


def test_streams_and_captured_calls(gpu_lib):
    """A call on a side stream; two captured graphs that share a workspace, replayed in turn on new inputs; results the
    same bits every time."""
    rng = np.random.default_rng(11)
    cin, cout = 1024, 384
    wq, ws = (t.cuda() for t in _operand(rng, cout, cin, 3))
    perm = _dev_perm(_perm(rng, cin, 64))
    Xs = [torch.from_numpy(rng.normal(size=(T, cin))).to(torch.bfloat16).cuda() for T in (3, 150)]
    want = [b.linear8(wq, ws, X, perm) for X in Xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [b.linear8(wq, ws, X, perm) for X in Xs]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    wsp = torch.empty(b.linear8_workspace(150, cin), dtype=torch.uint8, device="cuda")
    ins = [torch.zeros_like(X) for X in Xs]
    outs = [torch.empty_like(y) for y in want]
    graphs = []
    for X, Y in zip(ins, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.linear8(wq, ws, X, perm, Y, workspace=wsp)
        graphs.append(g)
    for _ in range(3):
        for X, src, Y, g, y in zip(ins, Xs, outs, graphs, want):
            X.copy_(src)
            Y.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(Y, y)


def test_trained_layer_deployed_in_8_bits(gpu_lib):
    """The whole way: clipped training steps of two layers, hardening, the 8-bit weight, the 8-bit product on the
    calibration tokens; the output against the oracle's and against the unquantised hardened layer's."""
    wl = synth.custom(200, 512, 96, 64, 4, 8, 0.5, 5, "bf16", seed=21, outliers=True)
    layers = []
    for seed in (21, 22):
        li = synth.make_inputs(synth.custom(200, 512, 96, 64, 4, 8, 0.5, 5, "bf16", seed=seed, outliers=True))[0]
        W, X, L = (torch.from_numpy(li.W).cuda().to(torch.bfloat16), torch.from_numpy(li.X).cuda().to(torch.bfloat16),
                   torch.from_numpy(li.L).cuda())
        d = b.alloc_outputs(W, X, L)
        d["perm"] = torch.empty(8, 64, dtype=torch.int32, device="cuda")
        layers.append(d)
    tr = b.Trainer(b.Step(layers, 64, wl.n, wl.m, wl.iters, 1.0, flags=b.FLAG_HARD), b.adamw_params(lr=5e-3), 4, max_norm=1e-3)
    tr.run(0, 4)
    b.Step(layers, 64, wl.n, wl.m, wl.iters, 0.1, flags=b.FLAG_HARD).run()
    for d in layers:
        wq, ws = b.quant8_weight(d["W"], d["perm"], d["mask"])
        Y = b.linear8(wq, ws, d["X"], d["perm"])
        perm = d["perm"].cpu().numpy().astype(np.int64)
        M = O.unpack_mask_bits(d["mask"].cpu().numpy().view(np.uint32), 512)
        W64, X64 = _np(d["W"]), _np(d["X"])
        rq, rs = O.quant8_weight(W64, perm, M)
        assert _same(_np(wq), rq) and _same(_np(ws), rs)
        xq, xs = O.quant8(X64, perm)
        x, w = O.dequant8(xq, xs, 1), O.dequant8(rq, rs, 128)
        assert np.all(np.abs(_np(Y) - x @ w.T) <= (512 / 32 + 40) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T))
        # against the layer that was trained: each operand is off by half a step of e4m3, 2^-4 of the value,
        # or 2^-10 of its scale near zero
        A, xp = np.where(M, O.gather_channels(W64, perm), 0.0), O.gather_channels(X64, perm)
        da = np.maximum(2.0 ** -4 * np.abs(A), 2.0 ** -10 * np.repeat(np.repeat(rs, 128, 0)[:200], 128, 1))
        dx = np.maximum(2.0 ** -4 * np.abs(xp), 2.0 ** -10 * np.repeat(xs, 128, 1))
        bound = np.abs(xp) @ da.T + dx @ np.abs(A).T + dx @ da.T
        assert np.all(np.abs(_np(Y) - xp @ A.T) <= bound * (1 + 1e-4))
    assert b.device_error() == 0
