"""Dense layers on 4-bit weights at prompt lengths, where they take the kernels with tall row tiles: which
kernel runs, and its rows against 64-bit products of the values that codes and scales stand for, within the
tolerance of the 4-bit experts (two roundings to bf16, twice their size)."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_30_amd as moe
from oracle import block

from gpu_util import DEV, log, sync
from test_gpu_int4 import GROUP, TOL, _matrix, _pack

pytestmark = pytest.mark.gpu


def _kernels(call):
    """Names of the kernels that a call launches."""
    moe.moe_kernel_timer_read()
    moe.moe_kernel_timer_enable(True)
    try:
        call()
        sync()
    finally:
        moe.moe_kernel_timer_enable(False)
    return {name.split("<")[0] for name in moe.moe_kernel_timer_read()}


# By ceil(T / 64) x I / 128 tall workgroups: the 16-row kernel below 512, tiles of 32 rows below 1000, then of 64.
@pytest.mark.parametrize("T,H,I,kernel", [
    (16, 256, 1024, "few"), (17, 256, 1024, "few"), (333, 384, 1152, "few"),
    (1001, 384, 4096, "many"), (257, 256, 13184, "many"), (1500, 512, 2816, "many"),
    (2049, 384, 4096, "many"), (4096, 256, 2048, "many"), (800, 640, 10112, "many")])
@pytest.mark.parametrize("wd", ["int4g128", "int4g32"])
def test_prompts(wd, T, H, I, kernel):
    rng, group = np.random.default_rng(T + H + I), GROUP[wd]
    C = moe.config(H, 2, 1, 1, 1, 128, I, 1.0, "bf16", wd)
    m = {"ws13": _matrix(rng, 1, 2 * I, H, group), "ws2": _matrix(rng, 1, H, I, group)}
    packed = {k: _pack(C, which, *m[k]) for k, which in (("ws13", moe.MOE_WS13), ("ws2", moe.MOE_WS2))}
    w13, w2 = (torch.from_numpy(block.dequantize_int4(*m[k], group)[0]).to(DEV, torch.float64) for k in ("ws13", "ws2"))
    x = torch.randn(T, H, generator=torch.Generator(device=DEV).manual_seed(T), device=DEV).bfloat16()
    y = torch.full((T + 3, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.full((moe.moe_dense_ffn_workspace_bytes(C, T),), 0xFF, dtype=torch.uint8, device=DEV)
    W = moe.weights(packed=True, **packed)
    assert _kernels(lambda: moe.moe_dense_ffn(C, T, x, W, y, ws)) == {f"grouped_gemm_int4_{kernel}"}
    assert torch.isnan(y[T:]).all()
    g, u = (x.double() @ w13.T).chunk(2, dim=1)
    ref = (g * torch.sigmoid(g) * u) @ w2.T
    bad = ((y[:T].double() - ref).norm(dim=1) / ref.norm(dim=1)).max().item()
    log(f"dense {wd} T={T} H={H} I={I}: worst row {bad:.2e}")
    assert bad <= TOL
    first = y[:T].clone()
    moe.moe_dense_ffn(C, T, x, W, y, ws)
    sync()
    assert torch.equal(first, y[:T])
