"""The binding's lists of gradients: whose memory they name is checked before any address of theirs reaches a
kernel (no GPU; `meta` and made-up GPUs stand for other devices)."""
import pytest
import torch

import sparse_mixture_experts_30_amd as moe


def _both(l, norm, ws):
    for call in (lambda: moe.moe_grad_norm(l, norm, ws, stream=0), lambda: moe.moe_clip_grads(l, 1.0, norm, ws, stream=0),
                 lambda: moe.moe_clip_grads(l, 1.0, norm, None, norm_given=True, stream=0)):
        yield call


def test_gradients_in_host_memory_are_refused():
    l = moe.gradients([torch.zeros(8), torch.zeros(8, dtype=torch.bfloat16)])
    ws = torch.empty(moe.moe_grad_norm_workspace_bytes(l), dtype=torch.uint8)
    for call in _both(l, torch.zeros(1), ws):
        with pytest.raises(ValueError, match="gradients on cpu"):
            call()


def test_a_list_over_several_devices_is_refused():
    t, m = torch.zeros(8), torch.zeros(8, device="meta")
    with pytest.raises(ValueError, match="several devices: cpu, meta"):
        moe.gradients([t, m])
    with pytest.raises(ValueError, match="several devices"):
        moe.gradients([t], [m])


def test_another_than_the_current_gpu_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    l = moe.gradients([torch.zeros(8)])
    l.device = torch.device("cuda", 1)
    for call in _both(l, torch.zeros(1), torch.empty(2048 * 8, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="current GPU is 0"):
            call()
    l.device = torch.device("cuda", 0)
    for call in _both(l, torch.zeros(1), torch.empty(2048 * 8, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="norm on cpu"):
            call()
    for call in (lambda: moe.moe_grad_norm(l, 0x1000, torch.empty(2048 * 8, dtype=torch.uint8), stream=0),
                 lambda: moe.moe_clip_grads(l, 1.0, 0x1000, torch.empty(2048 * 8, dtype=torch.uint8), stream=0)):
        with pytest.raises(ValueError, match="ws on cpu"):
            call()


def test_norm_of_whole_numbers_is_refused():
    l = moe.gradients([])
    for dtype in (torch.int32, torch.float64, torch.bfloat16):
        with pytest.raises(ValueError, match="not float32"):
            moe.moe_grad_norm(l, torch.zeros(1, dtype=dtype), None, stream=0)
