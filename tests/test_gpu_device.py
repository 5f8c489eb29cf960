"""Tensors on another device than the current one are refused before anything is launched (the current device's index is
taken from torch; with one GPU a test can only move that)."""
import pytest
import torch

from fp8_state_qat_amd import api

pytestmark = pytest.mark.gpu


def calls():
    T, H, d = 8, 1, 64
    x = [torch.zeros(T, H, d, device="cuda") for _ in range(4)]
    b, g = torch.zeros(T, H, device="cuda"), torch.zeros(T, H, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    S = torch.zeros(T, H, d, d, device="cuda")
    z, ids, top = torch.zeros(3, 20), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    z, ids, top = z.cuda(), ids.cuda(), top.cuda()
    stats = torch.zeros(3, 4, device="cuda")
    return {
        "chunk_grad": lambda: api.chunk_grad(*x[:3], b, g, cu, x[3]),
        "distill_fwd": lambda: api.distill_fwd(z, ids, top),
        "distill_bwd": lambda: api.distill_bwd(z, ids, top, stats),
        "distill_fwd_bwd": lambda: api.distill_fwd_bwd(z, ids, top),
        "chunk_fwd": lambda: api.chunk_fwd(*x[:3], b, g, cu),
        "decode_step": lambda: api.decode_step(*x[:3], b, g, S),
        "state_qdq": lambda: api.state_qdq(S[0]),
        "lin_attn_fwd": lambda: api.lin_attn_fwd(*x[:3], g, cu),
        "lin_attn_step": lambda: api.lin_attn_step(*x[:3], g, S),
        "act_pack": lambda: api.act_pack(z),
    }


@pytest.mark.parametrize("name", ["chunk_grad", "distill_fwd", "distill_bwd", "distill_fwd_bwd", "chunk_fwd",
                                  "decode_step", "state_qdq", "lin_attn_fwd", "lin_attn_step", "act_pack"])
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    call = calls()[name]
    call()
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        with pytest.raises(ValueError, match="current device"):
            call()
