"""linear8 on up to 8 tokens, the launch that quantises as it multiplies: the forms that the 8-bit tests' sizes
leave out.  The same tolerances: an output is the product of the quantised operands bit for bit, and
within (C_in / 32 + 40) 2^-23 sum |terms| of its exact value."""
import numpy as np
import pytest
import torch

from learnable_channel_permutation_b200 import binding as b
from oracle import lcp_oracle as O

pytestmark = pytest.mark.gpu


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _inputs(seed, T, cin, cout, B, dtype):
    """Tokens of very different sizes with outlier channels, a permutation, an 8-bit weight."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    ints = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device="cuda")
    X = normal(T, cin) * torch.exp2(ints(-20, 20, T, 1).float()) * torch.where(ints(0, 50, cin) == 0, 30.0, 1.0)
    perm = torch.rand(cin // B, B, generator=g, device="cuda").argsort(1).int() if B else None
    wq = (normal(cout, cin) * 110).clamp(-448, 448).to(b.E4M3)
    ws = ints(115, 128, -(-cout // 128), -(-cin // 128)).to(torch.uint8).view(b.E8M0)
    return X.to(dtype), perm, wq, ws


def _check(Y, q, s, wq, ws):
    cin, cout = wq.shape[1], wq.shape[0]
    rows = np.unique(np.concatenate([np.arange(0, cout, 37), [cout - 1]]))
    w = _np(wq.view(torch.uint8)[torch.from_numpy(rows).cuda()].view(b.E4M3)) * np.repeat(_np(ws), 128, 1)[rows // 128][:, :cin]
    x = O.dequant8(_np(q), _np(s), 1)
    ref, tol = x @ w.T, (cin / 32 + 40) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    if Y.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(_np(Y)[:, rows] - ref) <= tol)


# C_out / C_in pairs: a ring of its own for each CTA or two CTAs an SM, with and without a split, groups
# of a CTA in every remainder of four, C_in that ends inside a group
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("cin,cout", [(4096, 11008), (2272, 19200), (13824, 640), (5248, 24), (1120, 1000), (32, 130)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("order", ["plain", "permuted"])
def test_every_token_count_type_and_order(gpu_lib, T, cin, cout, dtype, order):
    B = 0 if order == "plain" else 64 if cin % 64 == 0 else 32
    X, perm, wq, ws = _inputs(T + cin + cout, T, cin, cout, B, dtype)
    q, s = b.quant8(X, perm)
    for out in (torch.float32, torch.bfloat16):
        Y = b.linear8(wq, ws, X, perm, out_dtype=out)
        assert torch.equal(Y, b.mm8(q, s, wq, ws, out_dtype=out))
        _check(Y, q, s, wq, ws)
    assert b.device_error() == 0


@pytest.mark.parametrize("groups", range(9, 44))
def test_every_length_of_the_last_chunk(gpu_lib, groups):
    """Long ranges of groups in one CTA (so many outputs that C_in is not split), every remainder of the ring and of a chunk."""
    for T in (2, 8):
        X, perm, wq, ws = _inputs(groups + T, T, 128 * groups - 32 * (groups % 4), 19200, 32, torch.float32)
        q, s = b.quant8(X, perm)
        assert torch.equal(b.linear8(wq, ws, X, perm), b.mm8(q, s, wq, ws))
    assert b.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinities_and_nan_stay_with_their_token(gpu_lib, dtype):
    X, _, wq, ws = _inputs(1, 7, 1120, 264, 0, dtype)
    X[2, 700], X[6, 1119] = float("inf"), float("nan")
    Y = b.linear8(wq, ws, X)
    bad = Y.isnan().all(1).cpu().tolist()
    assert bad == [False, False, True, False, False, False, True] and int(Y.isnan().any(1).sum()) == 2
