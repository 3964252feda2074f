"""The example's dense training step with clipping, and its serving step on 8-bit integer experts, end to end
against plain torch and the 64-bit definitions on the host.

Tolerances (relative L2).  Every intermediate is rounded to bf16 once (2^-8 of a value at most, 1.7e-3 in the
root mean square) and up to six of them lie between an input and a gradient: 4.2e-3, doubled for correlated
roundings: 1e-2.  On 8-bit experts the reference starts from the normed rows that the library holds and follows
the definition; h's codes, the experts' outputs and the layer's are left: three, 1e-2 again."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import sparse_mixture_experts_30_amd as moe
from oracle import block as oracle_block

from gpu_util import log

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
block = importlib.util.module_from_spec(spec)
spec.loader.exec_module(block)

H, E, G, TG, K, I, Is, RHO = SHAPE = (256, 8, 2, 2, 2, 128, 384, 2.5)
TOL = 1e-2


def _rows(T, seed):
    return torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def _rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("T", [1, 70, 300])
@pytest.mark.parametrize("share", [0.3, 4.0])
def test_dense_training_step(T, share):
    w = block.make_weights(H, E, I, Is)
    tr = block.DenseTraining(w, H, Is, T)
    x, res, dout, dsum = (_rows(T, i) for i in (2, 3, 4, 5))
    p = {k: w[k].double().cpu().requires_grad_() for k in ("norm", "ws13", "ws2")}
    xd = x.double().cpu().requires_grad_()
    s = xd + res.double().cpu()
    n = s / torch.sqrt((s * s).mean(1, keepdim=True) + block.EPS) * p["norm"]
    g, u = (n @ p["ws13"].t()).chunk(2, dim=1)
    ref = (torch.nn.functional.silu(g) * u) @ p["ws2"].t()
    torch.autograd.backward([ref, s], [dout.double().cpu(), dsum.double().cpu()])
    norm = float(torch.sqrt(sum((v.grad ** 2).sum() for v in p.values())))
    max_norm = share * norm
    out, sums = tr.forward(x, res)
    dx, grads, got = tr.backward(dout, dsum, max_norm)
    torch.cuda.synchronize()
    assert _rel(out, ref.detach()) <= TOL and _rel(sums, s.detach()) <= TOL and _rel(dx, xd.grad) <= TOL
    assert abs(float(got) - norm) <= TOL * norm
    f = min(1.0, max_norm / (norm + 1e-6))
    for k, v in p.items():
        r = _rel(grads[k], v.grad * f)
        log(f"dense block T={T} {k}: {r:.2e}")
        assert r <= TOL, k
    # a second step on the same buffers: the gradients are written anew, not added to
    before = {k: v.clone() for k, v in grads.items()}
    tr.forward(x, res)
    tr.backward(dout, dsum, max_norm)
    torch.cuda.synchronize()
    assert all(torch.equal(before[k], grads[k]) for k in grads)


def test_dense_training_step_captured():
    """Norm, dense block, both backwards and clipping as one graph, replayed."""
    T = 130
    w = block.make_weights(H, E, I, Is)
    tr = block.DenseTraining(w, H, Is, T)
    x, res, dout, dsum = (_rows(T, i) for i in (2, 3, 4, 5))

    def step():
        tr.forward(x, res)
        return tr.backward(dout, dsum, 0.5)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (tr.out, tr.dx, tr.grad_norm, *tr.grads.values())]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = block.DenseTraining(w, H, Is, T)
    for _ in range(3):
        for t in (tr.out, tr.dx, tr.grad_norm, tr.gu, *tr.grads.values()):
            t.fill_(9.0)
        tr.ws.fill_(0xFF)
        graph.replay()
        other.forward(x, res)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((tr.out, tr.dx, tr.grad_norm, *tr.grads.values()), want))


@pytest.mark.parametrize("T", [1, 20, 150])
def test_serving_step_on_8_bit_experts(T):
    w = block.make_weights(H, E, I, Is)
    s8 = block.Serving(w, *SHAPE, max_tokens=T, bits=8)
    x, res, out = _rows(T, 6), _rows(T, 7), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    r0 = res.clone()
    idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
    tw = torch.empty(T, K, dtype=torch.float32, device="cuda")
    s8.step(x, res, out)
    moe.moe_forward(s8.cfg, T, s8.n[:T], s8.weights, torch.empty_like(out), s8.ws, topk_idx=idx, topk_w=tw)
    torch.cuda.synchronize()
    assert torch.equal(res, (x.float() + r0.float()).bfloat16())
    n, i, t = s8.n[:T].double().cpu().numpy(), idx.cpu().numpy(), tw.double().cpu().numpy()
    q = {k: oracle_block.quantize_int8(w[k].double().cpu().numpy()) for k in ("w13", "w2", "ws13", "ws2")}
    ref = oracle_block.swiglu_int8(n, q["ws13"], q["ws2"])
    for e in range(E):
        r, k = np.nonzero(i == e)
        if len(r):
            ref[r] += t[r, k][:, None] * oracle_block.swiglu_int8(n[r], tuple(v[e] for v in q["w13"]), tuple(v[e] for v in q["w2"]))
    r = _rel(out, torch.from_numpy(ref))
    log(f"8-bit block T={T}: {r:.2e}")
    assert r <= TOL
