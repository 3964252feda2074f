"""Norm and clipping of gradients of more than 2^30 and 2^31 values: offsets past
32 bits, runs that end at 2^30 values, inside a chunk of a flat buffer."""
import pytest
import torch

import sparse_mixture_experts_30_amd as moe

from gpu_util import DEV

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def _norm2(t):
    return sum(float((c.double() ** 2).sum()) for c in t.split(1 << 27))


def _fill(n, dtype, seed):
    """Values that differ along the whole length, larger where 2^30 and 2^31 are crossed."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.empty(n, dtype=dtype, device=DEV)
    for c in t.split(1 << 27):
        c.copy_(torch.randn(c.numel(), generator=g, device=DEV))
    for at in (0, 1 << 30, 1 << 31, n - 3):
        t[max(0, at - 5):at + 7] = 1000.0
    return t


@pytest.mark.parametrize("pieces", [[((1 << 31) + 11, torch.bfloat16, 3)],
                                    [(1001, torch.float32, 1), ((1 << 30) + 5, torch.float32, 0), (77, torch.bfloat16, 1)]])
def test_more_values_than_a_run(pieces):
    grads = [_fill(n + skip, dt, i)[skip:] for i, (n, dt, skip) in enumerate(pieces)]
    want = sum(_norm2(g) for g in grads) ** 0.5
    limit = 0.25 * want
    before = [[c.clone() for c in (g[:4096], g[(1 << 30) - 4096:(1 << 30) + 4096], g[(1 << 31) - 4096:], g[-4096:])]
              for g in grads]
    l = moe.gradients(grads)
    norm, ws = torch.zeros(1, device=DEV), torch.empty(moe.moe_grad_norm_workspace_bytes(l), dtype=torch.uint8, device=DEV)
    moe.moe_clip_grads(l, limit, norm, ws)
    torch.cuda.synchronize()
    assert abs(float(norm) - want) <= 2 * E * want
    f = limit / (want + 1e-6)
    for g, b in zip(grads, before):
        u = 5 * E + (2.0 ** -8 if g.dtype == torch.bfloat16 else 0)
        for c, o in zip((g[:4096], g[(1 << 30) - 4096:(1 << 30) + 4096], g[(1 << 31) - 4096:], g[-4096:]), b):
            assert torch.all((c.double() - f * o.double()).abs() <= u * f * o.double().abs())
    # every value was scaled once: the norm is the limit, to the roundings of the values
    after = sum(_norm2(g) for g in grads) ** 0.5
    assert abs(after - f * want) <= 2.0 ** -8 * f * want


def test_neighbours_in_a_flat_buffer_across_a_full_run():
    """Pieces without gaps: the first run is full inside the second piece."""
    flat = _fill((1 << 30) + 5000, torch.bfloat16, 9)
    cut = (1 << 29) + 3
    want, tail = _norm2(flat) ** 0.5, flat[-5100:].clone()
    l = moe.gradients([flat[:cut], flat[cut:]])
    norm, ws = torch.zeros(1, device=DEV), torch.empty(moe.moe_grad_norm_workspace_bytes(l), dtype=torch.uint8, device=DEV)
    moe.moe_clip_grads(l, want / 8, norm, ws)
    torch.cuda.synchronize()
    assert abs(float(norm) - want) <= 2 * E * want
    f = want / 8 / (want + 1e-6)
    assert torch.all((flat[-5100:].double() - f * tail.double()).abs() <= (2.0 ** -8 + 5 * E) * f * tail.double().abs())
    assert abs(_norm2(flat) ** 0.5 - f * want) <= 2.0 ** -8 * f * want
