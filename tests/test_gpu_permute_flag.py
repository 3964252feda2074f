"""The error flag of the permutation is written by every call, whatever the workspace held: with 512
experts (as many as the scan has threads) and more ids than one block takes, too."""
import numpy as np
import pytest
import torch

import synth
import sparse_mixture_experts_30_amd as moe
from synth import device as sd

from gpu_util import DEV, random_routing, run_permute

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fill", [0x00, 0xFF])
@pytest.mark.parametrize("E", [2, 511, 512])
@pytest.mark.parametrize("T", [16, 3000])
def test_flag_is_written(T, E, fill):
    cfg = synth.C1.replace(name="flag", T=T, E=E, G=1, TG=1, K=1)
    idx = random_routing(T, 1, E, seed=T + E)
    for bad in (None, E, -1, 2 ** 31 - 1):
        i = idx.copy()
        if bad is not None:
            i[T // 2, 0] = bad
        ws = torch.full((moe.moe_workspace_bytes(sd.moe_config(cfg), T),), fill, dtype=torch.uint8, device=DEV)
        counts, offsets, perm, pos, status = run_permute(cfg, i, ws=ws)
        assert status == (moe.MOE_OK if bad is None else moe.MOE_ERR_DEVICE_CHECK), bad
        valid = i[(i >= 0) & (i < E)]
        assert np.array_equal(counts, np.bincount(valid, minlength=E)) and offsets[E] == valid.size
