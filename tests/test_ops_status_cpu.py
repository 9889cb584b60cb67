"""Arguments of the operators' failure reporting and test hook."""
import ctypes

import pytest
import torch

from bit_diffusion_transformer_w4a4_b200 import svdq


def test_error_site_arguments():
    L = svdq.lib()
    assert L.svdq_ops_device_error_site(None, None) == 1
    if not torch.cuda.is_available():
        v = ctypes.c_int(-1)
        assert L.svdq_ops_device_error_site(None, ctypes.byref(v)) == 4 and v.value == -1
        with pytest.raises(svdq.SvdqError):
            svdq.ops_error_site()


def test_hook_arguments():
    L = svdq.lib()
    assert L.svdq_ops_debug_set_fault(4, 0) == 1 and L.svdq_ops_debug_set_fault(1 << 31, 0) == 1
    assert L.svdq_ops_debug_set_fault(3, 5000) == 0 and L.svdq_ops_debug_set_fault(0, 0) == 0
