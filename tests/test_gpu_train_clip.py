"""lcp_train_clip through the C ABI where the Python trainer does not reach."""
import ctypes

import pytest
import torch

from learnable_channel_permutation_b200 import binding as b

pytestmark = pytest.mark.gpu


def test_training_no_layers_gives_the_norm_of_an_empty_list(gpu_lib):
    n = ctypes.c_size_t(0)
    b.check(b.lib().lcp_clip_workspace_size(0, ctypes.byref(n)))
    ws = torch.empty(max(n.value, 256), dtype=torch.uint8, device="cuda")
    norm = torch.full((3,), 7.0, device="cuda")
    hp, opt = b.hparams(64, 2, 4, 5, 0.5, b.BF16), b.adamw_params()
    run = lambda count: b.check(b.lib().lcp_train_clip(None, 0, ctypes.byref(hp), ctypes.byref(opt), None, 0, count, 2, 1.0, 0.1,
                                                       1.0, norm[1:].data_ptr(), ws.data_ptr(), ws.numel(),
                                                       torch.cuda.current_stream().cuda_stream))
    run(0)                                  # no step: there is no norm to give
    assert norm.tolist() == [7.0, 7.0, 7.0]
    run(2)
    assert norm.tolist() == [7.0, 0.0, 7.0]
