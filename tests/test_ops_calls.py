"""Calls of the operators next to the layer that are easily left out: another device's sizes, errors of
an earlier call, forward-mode derivatives, captured steps, version counters, arguments of other types."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
pytestmark = gpu

from scale_gated_linear_b200 import (MSGLAError, _lib, gated_scan, gated_scan_backward, gated_scan_forward,  # noqa: E402
                                     gated_scan_step, group_norm, group_norm_backward, group_norm_forward)

BF16, F32 = torch.bfloat16, torch.float32


def randn(*shape, dtype=F32, seed=0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def test_workspace_sizes_are_of_the_named_device():
    """A size for a device that does not exist is refused: it would be that of the current one."""
    lib, n = _lib.load(), ctypes.c_size_t()
    for gradients in (0, 1):
        for S in (1, 4, 5000):
            good = _lib.NormConfig(0, 0, 64, 4, 0, 1, 1e-5)
            assert lib.msgla_group_norm_workspace_size(good, 8, S, gradients, ctypes.byref(n)) == 0
            bad = _lib.NormConfig(torch.cuda.device_count(), 0, 64, 4, 0, 1, 1e-5)
            assert lib.msgla_group_norm_workspace_size(bad, 8, S, gradients, ctypes.byref(n)) < 0
