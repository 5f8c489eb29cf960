"""Refusals of the distillation calls that need no GPU."""
import ctypes

import pytest
import torch

from fp8_state_qat_amd import _lib, api

P, FAKE = ctypes.c_void_p, 1 << 20


@pytest.mark.parametrize("temperature", [1e-38, 1e-31, 1e-45, 1e30, -1.0])
def test_temperatures_whose_inverse_leaves_fp32_are_refused(temperature):
    s = _lib.GdnDistill(rows=3, vocab=20, topk=2, dtype=0, temperature=temperature, kd_weight=1.0, ce_weight=0.0,
                        ignore_index=-100, row_stride=20, d_row_stride=20)
    L = _lib.lib()
    at = [P(FAKE * i) for i in range(1, 9)]
    assert L.gdn_distill_fwd_bwd(ctypes.byref(s), *at, None) == 1 and "temperature" in _lib.last_error()
    assert L.gdn_distill_bwd(ctypes.byref(s), *at, None) == 1 and "temperature" in _lib.last_error()
    assert L.gdn_distill_fwd(ctypes.byref(s), *at[:7], None) == 1 and "temperature" in _lib.last_error()


@pytest.mark.parametrize("out", [True, False, 3, "x", [[0.0]]])
def test_an_out_that_is_no_tensor_is_refused(out):
    a = torch.zeros(3, 20), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    with pytest.raises(ValueError, match="out must be a torch tensor"):
        api.distill_fwd_bwd(*a, out=out)
    with pytest.raises(ValueError, match="out must be a torch tensor"):
        api.distill_bwd(*a, torch.zeros(3, 4), out=out)
