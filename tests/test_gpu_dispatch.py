"""Sorted token rows, their gradient and the combine's gradient on the GPU.
Copies and single products are compared bit for bit; a sum of n fp32 terms is
within n 2^-24 of the sum of magnitudes, a dot product over H values within
(H / 64 + 16) 2^-24, and a rounding to bf16 within 2^-8 of the value."""
import numpy as np
import pytest
import torch

import synth
import sparse_mixture_experts_30_amd as moe
from oracle import block

from gpu_util import DEV, host, random_routing, run_permute, sync

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = [(1, 64, 1), (1, 7168, 8), (5, 192, 3), (33, 1024, 4), (261, 512, 8), (70, 7168, 9), (7, 8256, 16),
         (3, 256, 64), (1025, 128, 2)]
LARGE = (1200, 7168, 8)   # past the size from which rows are read and written non-temporally


def _cfg(H, K, act):
    return moe.config(H, 64, 1, 1, K, 128, 0, 1.0, act, act)


def _pos(T, K, drop=False):
    """Positions as the permutation makes them; drop: some slots without a row."""
    c = synth.C1.replace(name="pos", T=T, E=64, G=1, TG=1, K=K)
    _, _, _, pos, status = run_permute(c, random_routing(T, K, 64, seed=T + K, skew=True))
    assert status == moe.MOE_OK
    if drop:
        rng = np.random.default_rng(T)
        gone = rng.random(T * K) < 0.3
        pos = np.where(gone, rng.choice([-1, -2 ** 31, T * K, 2 ** 31 - 1], T * K), pos).astype(np.int32)
    return pos


def _rows(seed, T, H, act):
    return torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).to(DT[act]).to(DEV)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,K", SIZES + [LARGE])
def test_dispatch(T, H, K, act, drop):
    pos, x = _pos(T, K, drop), _rows(1, T, H, act)
    rows = torch.full((T * K, H), 7.0, dtype=DT[act], device=DEV)
    moe.moe_dispatch(_cfg(H, K, act), T, x, _dev(pos), rows)
    sync()
    want = np.full((T * K, H), 7.0, np.float32)
    ok = (pos >= 0) & (pos < T * K)
    want[pos[ok]] = np.repeat(host(x), K, axis=0)[ok]
    assert np.array_equal(host(rows), want)


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("T,H,K", [s for s in SIZES if s[1] % 128 == 0] + [(9, 640, 5), (2400, 7168, 8)])
def test_dispatch_quantized(T, H, K, drop):
    rng = np.random.default_rng(T + H)
    pos, q = _pos(T, K, drop), rng.integers(0, 256, (T, H), dtype=np.uint8)
    s = rng.random((T, H // 128), dtype=np.float32)
    rq = torch.full((T * K, H), 9, dtype=torch.uint8, device=DEV)
    rs = torch.full((T * K, H // 128), 9.0, device=DEV)
    moe.moe_dispatch_quantized(_cfg(H, K, "bf16"), T, _dev(q), _dev(s), _dev(pos), rq, rs)
    sync()
    ok = (pos >= 0) & (pos < T * K)
    wq, wsc = np.full((T * K, H), 9, np.uint8), np.full((T * K, H // 128), 9.0, np.float32)
    wq[pos[ok]], wsc[pos[ok]] = np.repeat(q, K, axis=0)[ok], np.repeat(s, K, axis=0)[ok]
    assert np.array_equal(host(rq), wq) and np.array_equal(host(rs), wsc)


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,K", SIZES + [LARGE])
def test_dispatch_backward(T, H, K, act, drop):
    pos, d, add = _pos(T, K, drop), _rows(2, T * K, H, act), _rows(3, T, H, act)
    cfg, N = _cfg(H, K, act), T * K
    ones = np.ones((T, K))
    u = 2.0 ** -8 if act == "bf16" else 2.0 ** -24
    for a in (add, None):
        dx = torch.full((T, H), float("nan"), dtype=DT[act], device=DEV)
        moe.moe_dispatch_backward(cfg, T, d, _dev(pos), dx, dx_add=a)
        sync()
        ref, mag = block.combine(host(d), pos, ones, N), block.combine(np.abs(host(d)), pos, ones, N)
        if a is not None:
            ref, mag = ref + host(a), mag + np.abs(host(a))
        assert np.all(np.abs(host(dx) - ref) <= (K + 1) * 2.0 ** -24 * mag + u * np.abs(ref))
        if a is not None:
            b = a.clone()
            moe.moe_dispatch_backward(cfg, T, d, _dev(pos), b, dx_add=b)
            sync()
            assert torch.equal(b, dx)


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,K", SIZES + [LARGE])
def test_combine_backward(T, H, K, act, drop):
    pos, dout, y = _pos(T, K, drop), _rows(4, T, H, act), _rows(5, T * K, H, act)
    w = np.random.default_rng(6).random((T, K), dtype=np.float32)
    cfg = _cfg(H, K, act)
    dy = torch.full((T * K, H), 7.0, dtype=DT[act], device=DEV)
    dw = torch.full((T, K), float("nan"), device=DEV)
    moe.moe_combine_backward(cfg, T, dout, y, _dev(pos), _dev(w), dy, dw)
    sync()
    ok = (pos >= 0) & (pos < T * K)
    want = np.full((T * K, H), 7.0, np.float32)
    want[pos[ok]] = block.stored(w[:, :, None] * host(dout)[:, None, :], act).reshape(T * K, H)[ok]
    assert np.array_equal(host(dy), want)
    ref = block.combine_backward_w(host(dout), host(y), pos, K)
    mag = block.combine_backward_w(np.abs(host(dout)), np.abs(host(y)), pos, K)
    assert np.all(np.abs(host(dw) - ref) <= (H / 64 + 16) * 2.0 ** -24 * mag)
    assert np.all(host(dw).reshape(-1)[~ok] == 0)
    b, dw2 = y.clone(), torch.empty_like(dw)
    moe.moe_combine_backward(cfg, T, dout, b, _dev(pos), _dev(w), b, dw2)   # dy over y
    sync()
    assert torch.equal(dw2, dw) and np.array_equal(host(b)[pos[ok]], want[pos[ok]])


def test_the_two_ends_are_the_layers_backward():
    """combine backward -> expert backward -> dispatch backward against the whole layer's backward:
    the same input gradient up to the gate's part, which a zero gate weight removes."""
    from synth import device as sd
    cfg = synth.C3.replace(name="ends", T=70, H=256, E=8, G=2, TG=2, K=2, I=128, Is=128, rho=1.0)
    inp = synth.gen_inputs(cfg)
    inp["gate_w"] = np.zeros_like(inp["gate_w"])
    dev = sd.to_device(inp)
    C, T, W = sd.moe_config(cfg), cfg.T, sd.weights_struct(dev)
    N = T * cfg.K
    f32, i32 = dict(dtype=torch.float32, device=DEV), dict(dtype=torch.int32, device=DEV)
    lg, idx, w = torch.empty((T, cfg.E), **f32), torch.empty((T, cfg.K), **i32), torch.empty((T, cfg.K), **f32)
    ws = sd.workspace(cfg, T)
    moe.moe_gate(C, T, dev["x"], dev["gate_w"], dev["bias"], lg, idx, w, ws)
    counts, off = torch.empty(cfg.E, **i32), torch.empty(cfg.E + 1, **i32)
    perm, pos = torch.empty(N, **i32), torch.empty(N, **i32)
    moe.moe_permute(C, T, idx, counts, off, perm, pos, ws)
    y, ys = _rows(7, N, cfg.H, "bf16"), _rows(8, T, cfg.H, "bf16")
    moe.moe_expert_ffn(C, T, dev["x"], perm, off, W, y, ys, ws)
    dout = _rows(9, T, cfg.H, "bf16")
    g = {k: torch.empty_like(dev[k]) for k in ("w13", "w2", "ws13", "ws2")}
    g2 = {k: torch.empty_like(dev[k]) for k in g}
    dx, dgw = torch.empty_like(dout), torch.empty_like(dev["gate_w"])
    wb = torch.empty(moe.moe_backward_workspace_bytes(C, T), dtype=torch.uint8, device=DEV)
    moe.moe_backward(C, T, dev["x"], W, lg, idx, w, perm, off, pos, y, dout, dx, dgw, g["w13"], g["w2"], g["ws13"],
                     g["ws2"], wb)
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    moe.moe_combine_backward(C, T, dout, y, pos, w, dy, dw)
    drows, dxs, out = torch.empty_like(y), torch.empty_like(dout), torch.empty_like(dout)
    moe.moe_expert_ffn_backward(C, T, dev["x"], perm, off, W, dy, dout, drows, dxs, g2["w13"], g2["w2"], g2["ws13"],
                                g2["ws2"], wb)
    moe.moe_dispatch_backward(C, T, drows, pos, out, dx_add=dxs)
    sync()
    assert torch.equal(out, dx)
    for k in g:
        assert torch.equal(g[k], g2[k]), k
