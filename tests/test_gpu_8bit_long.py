"""Products of many tokens over as many channels as the pair kernel stages a tile's scales for (256 groups), with
scale rows of every alignment, against float64 at the tolerance of the 8-bit product."""
import numpy as np
import pytest
import torch

from learnable_channel_permutation_b200 import binding as b

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,last", [(129, 128), (170, 32), (171, 96), (213, 128), (254, 64), (255, 128), (256, 32), (256, 128),
                                         (257, 32)])
@pytest.mark.parametrize("T,cout", [(67, 130), (300, 264), (1000, 40)])
def test_long_rows_of_scales(gpu_lib, groups, last, T, cout):
    cin = 128 * (groups - 1) + last
    g = torch.Generator(device="cuda").manual_seed(groups + T)
    operand = lambda rows, srows: ((torch.randn(rows, cin, generator=g, device="cuda") * 110).clamp(-448, 448).to(b.E4M3),
                                   torch.randint(115, 128, (srows, groups), generator=g, device="cuda").to(torch.uint8).view(b.E8M0))
    (xq, xs), (wq, ws) = operand(T, T), operand(cout, -(-cout // 128))
    Y = b.mm8(xq, xs, wq, ws)
    value = lambda q, s, rows: q.double() * s.double().repeat_interleave(rows, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :cin]
    x, w = value(xq, xs, 1), value(wq, ws, 128)
    tol = (cin / 32 + 40) * 2.0 ** -23 * (x.abs() @ w.abs().T)
    assert bool(((Y.double() - x @ w.T).abs() <= tol).all())
    assert b.device_error() == 0
