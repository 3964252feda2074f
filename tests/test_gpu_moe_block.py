"""The example block end to end: its three paths against plain torch in 64 bits on the host, with the
routing held at the library's choice.

Tolerances (relative L2).  Every intermediate is rounded to bf16 once (2^-8 of a value at most, 1.7e-3 in
the root mean square) and up to nine of them lie between an input and a gradient: 1.7e-3 sqrt(9) = 5e-3,
doubled for correlated roundings: 1e-2.  On e4m3 weights and rows the layer's own bound, 6e-2 against the
values that the weights' codes and scales stand for."""
import importlib.util
import os

import pytest
import torch

from gpu_util import log

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
block = importlib.util.module_from_spec(spec)
spec.loader.exec_module(block)

H, E, G, TG, K, I, Is, RHO = SHAPE = (256, 8, 2, 2, 2, 128, 128, 2.5)


def _rows(T, seed):
    return torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def _rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return float((a - b).norm() / b.norm())


def _ffn(x, w13, w2):
    g, u = (x @ w13.t()).chunk(2, dim=1)
    return (torch.nn.functional.silu(g) * u) @ w2.t()


def _plain(p, x, res, idx):
    """(out, sum) in 64 bits for chosen experts idx; p: weights, with or without an adapter."""
    s = x + res
    n = s / torch.sqrt((s * s).mean(1, keepdim=True) + block.EPS) * p["norm"]
    sc = torch.sigmoid(n @ p["gate_w"].t()).gather(1, idx)
    tw = RHO * sc / (sc.sum(1, keepdim=True) + 1e-20)
    out = _ffn(n, p["ws13"], p["ws2"])
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        y = _ffn(n[t], p["w13"][e], p["w2"][e])
        if "adapter" in p:
            y = y + p["adapter"][e] * n[t]
        out = out.index_add(0, t, tw[t, k][:, None] * y)
    return out, s


def test_training_step():
    T = 70
    w = block.make_weights(H, E, I, Is)
    adapter = 0.1 * _rows(E, 1)
    tr = block.Training(w, adapter, *SHAPE, T=T)
    x, res, dout, dsum = (_rows(T, i) for i in (2, 3, 4, 5))
    out, s = tr.forward(x, res)
    d = tr.backward(dout, dsum)
    torch.cuda.synchronize()
    p = {k: v.double().cpu().requires_grad_() for k, v in {**w, "adapter": adapter}.items()}
    xd = x.double().cpu().requires_grad_()
    ref, refs = _plain(p, xd, res.double().cpu(), tr.idx.long().cpu())
    assert _rel(out, ref.detach()) <= 1e-2 and _rel(s, refs.detach()) <= 1e-2
    torch.autograd.backward([ref, refs], [dout.double().cpu(), dsum.double().cpu()])
    got = {"x": xd.grad, **{k: p[k].grad for k in p if k != "bias"}}
    for k, v in got.items():
        r = _rel(d[k], v)
        log(f"block gradient {k}: {r:.2e}")
        assert r <= 1e-2, (k, r)


@pytest.mark.parametrize("group", [128, 32])
@pytest.mark.parametrize("T", [1, 20, 50])
def test_serving_step(T, group):
    """Against the same block on the values that the 4-bit codes stand for."""
    import sparse_mixture_experts_30_amd as moe
    w = block.make_weights(H, E, I, Is)
    s4 = block.Serving(w, *SHAPE, max_tokens=T, group=group)
    x, res, out = _rows(T, 6), _rows(T, 7), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    r0 = res.clone()
    idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
    s4.step(x, res, out)
    moe.moe_forward(s4.cfg, T, s4.n[:T], s4.weights, torch.empty_like(out), s4.ws, topk_idx=idx)
    torch.cuda.synchronize()
    assert torch.equal(res, (x.float() + r0.float()).bfloat16())
    p = {k: v.double().cpu() for k, v in w.items()}
    for k in ("w13", "w2", "ws13", "ws2"):
        g = p[k].reshape(*p[k].shape[:-1], -1, group)
        sc = (w[k].float().cpu().reshape(g.shape).abs().amax(-1, keepdim=True) / 7).bfloat16().double()
        p[k] = ((g / sc).round().clamp(-8, 7) * sc).reshape(p[k].shape)
    ref, _ = _plain(p, x.double().cpu(), r0.double().cpu(), idx.long().cpu())
    r = _rel(out, ref)
    log(f"4-bit block T={T} group {group}: {r:.2e}")
    assert r <= 1e-2


def test_serving_step_fp8():
    import sparse_mixture_experts_30_amd as moe
    T = 40
    w = block.make_weights(H, E, I, Is)
    packed, scales = block.fp8_weights(w, moe.config(*SHAPE, "bf16", "fp8"))
    s8 = block.ServingFp8(packed, scales, w, *SHAPE, max_tokens=T)
    x, res, out = _rows(T, 8), _rows(T, 9), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    r0 = res.clone()
    s8.step(x, res, out)
    torch.cuda.synchronize()
    p = {k: v.double().cpu() for k, v in w.items()}
    for k in scales:
        s = scales[k].double().cpu().repeat_interleave(128, -2).repeat_interleave(128, -1)
        p[k] = (w[k].float().cpu() / s.float()).to(torch.float8_e4m3fn).double() * s
    ref, _ = _plain(p, x.double().cpu(), r0.double().cpu(), s8.idx.long().cpu())
    r = _rel(out, ref)
    log(f"e4m3 block: {r:.2e}")
    assert r <= 6e-2
