"""Experts in 8-bit integers on the GPU against the 64-bit definition.

Tolerances.  Codes are exact whole numbers for bf16 rows; scales are one fp32
quotient.  A product is exact in integers and then scaled twice in fp32, so g
and u are off by 4 x 2^-24 of themselves, h by 2^-18 (the exponential and its
quotient included); a code of h can then differ, by one, only where 127 h / max
lies within 127 x 2^-17 of a half.  Each output is bounded by the codes that
may differ, 2^-17 of its terms for h's scale and products, and 2^-8 of itself
for the rounding to bf16."""
import numpy as np
import pytest
import torch

import synth
import sparse_mixture_experts_30_amd as moe
from oracle import block

from gpu_util import DEV, host, log, random_routing, rel_l2, run_permute, sync

pytestmark = pytest.mark.gpu

WHICH = {"w13": moe.MOE_W13, "w2": moe.MOE_W2, "ws13": moe.MOE_WS13, "ws2": moe.MOE_WS2}


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _bf16_dev(a):
    return _dev(np.asarray(a, np.float32)).to(torch.bfloat16)


def _cfg(H=256, E=4, K=2, I=128, Is=128):
    return moe.config(H, E, 1, 1, K, I, Is, 1.0, "bf16", "int8")


def _swiglu_bounds(x, w13, w2):
    """y and its bound."""
    q, s = block.quantize_int8(x)
    g, u = np.split(block.int8_product(q, s, *w13), 2, axis=1)
    h = g / (1 + np.exp(-g)) * u
    a = np.abs(h).max(axis=1, keepdims=True)
    t = np.where(a > 0, 127 * h / np.where(a > 0, a, 1), 0.0)
    q, s = block.quantize_int8(h)
    near = np.abs(t - np.floor(t) - 0.5) <= 127 * 2.0 ** -17
    c, cs = (np.asarray(v, np.float64) for v in w2)
    y = block.int8_product(q, s, c, cs)
    terms = (np.abs(q) @ np.abs(c).T) * s[:, None] * cs
    flips = (near.astype(np.float64) @ np.abs(c).T) * s[:, None] * cs
    e = flips + 2.0 ** -17 * (terms + flips)
    return y, e + 2.0 ** -8 * (np.abs(y) + e)


class Layer:
    def __init__(self, H, E, K, I, Is, seed=0):
        rng = np.random.default_rng(seed)
        self.C, self.H, self.E, self.K, self.I, self.Is = _cfg(H, E, K, I, Is), H, E, K, I, Is
        shapes = {"w13": (E, 2 * I, H), "w2": (E, H, I)}
        if Is:
            shapes.update(ws13=(1, 2 * Is, H), ws2=(1, H, Is))
        self.w, self.kw = {}, {}
        for name, sh in shapes.items():
            q = rng.integers(-127, 128, sh).astype(np.int8)
            s = ((0.3 + rng.random(sh[:-1])) / (73 * np.sqrt(sh[-1]))).astype(np.float32)
            self.w[name] = (q, s)
            buf = torch.full((moe.moe_packed_bytes(self.C, WHICH[name]),), 0xEE, dtype=torch.uint8, device=DEV)
            moe.moe_pack_weight(self.C, WHICH[name], _dev(q), buf)
            self.kw[name], self.kw[name + "_scale"] = buf, _dev(s)
        self.W = moe.weights(packed=True, **self.kw)

    def rows(self, T, seed=1):
        rng = np.random.default_rng(seed)
        return block.bf16((rng.standard_normal((T, self.H)) * np.exp(rng.standard_normal((T, 1)))).astype(np.float32))

    def run(self, T, x, idx, quantized=False):
        c = synth.C1.replace(name="int8", T=T, E=self.E, G=1, TG=1, K=self.K)
        _, off, perm, _, _ = run_permute(c, idx)
        N = T * self.K
        y = torch.full((N + 2, self.H), float("nan"), dtype=torch.bfloat16, device=DEV)
        ys = torch.full((T + 2, self.H), float("nan"), dtype=torch.bfloat16, device=DEV) if self.Is else None
        ws = torch.full((moe.moe_workspace_bytes(self.C, T),), 0xFF, dtype=torch.uint8, device=DEV)
        if quantized:
            xq = torch.empty(T, self.H, dtype=torch.uint8, device=DEV)
            xs = torch.empty(T, dtype=torch.float32, device=DEV)
            moe.moe_quantize_act(self.C, T, _bf16_dev(x), xq, xs)
            moe.moe_expert_ffn_quantized(self.C, T, xq, xs, _dev(perm), _dev(off), self.W, y, ys, ws)
        else:
            moe.moe_expert_ffn(self.C, T, _bf16_dev(x), _dev(perm), _dev(off), self.W, y, ys, ws)
        sync()
        return y, ys, off, perm

    def check(self, T, idx, seed=1):
        x, N = self.rows(T, seed), T * self.K
        y, ys, off, perm = self.run(T, x, idx)
        g = host(y)
        assert np.isnan(g[N:]).all()
        ref, tol = np.zeros((N, self.H)), np.zeros((N, self.H))
        for e in range(self.E):
            r = slice(off[e], off[e + 1])
            if off[e + 1] > off[e]:
                ref[r], tol[r] = _swiglu_bounds(x[perm[r] // self.K], tuple(v[e] for v in self.w["w13"]),
                                                tuple(v[e] for v in self.w["w2"]))
        d = np.abs(g[:N] - ref)
        log(f"int8 T={T} rel {rel_l2(g[:N], ref):.2e} worst share of the bound {np.max(d / (tol + 1e-30)):.2f}")
        assert np.all(d <= tol)
        if self.Is:
            ref, tol = _swiglu_bounds(x, tuple(v[0] for v in self.w["ws13"]), tuple(v[0] for v in self.w["ws2"]))
            g = host(ys)
            assert np.all(np.abs(g[:T] - ref) <= tol) and np.isnan(g[T:]).all()
        y2, ys2, _, _ = self.run(T, x, idx, quantized=True)
        assert torch.equal(y[:N], y2[:N]) and (not self.Is or torch.equal(ys[:T], ys2[:T]))


@pytest.mark.parametrize("T,H,E,K,I,Is", [
    (1, 256, 4, 2, 128, 128), (1, 640, 8, 8, 384, 0), (2, 128, 4, 1, 128, 256), (5, 384, 70, 3, 256, 128),
    (16, 256, 2, 1, 256, 384), (17, 256, 4, 2, 128, 128), (33, 512, 4, 3, 128, 0), (64, 128, 2, 2, 640, 128),
    (65, 896, 8, 2, 128, 128), (100, 256, 3, 3, 256, 1024), (200, 384, 4, 2, 384, 128), (515, 256, 2, 1, 128, 128),
    (700, 128, 4, 4, 128, 256), (1100, 256, 2, 2, 256, 0)])
def test_against_the_definition(T, H, E, K, I, Is):
    Layer(H, E, K, I, Is, seed=T).check(T, random_routing(T, K, E, T))


@pytest.mark.parametrize("T", [1, 20, 150, 600])
def test_one_expert_has_every_row(T):
    idx = np.full((T, 1), 3, np.int32)
    Layer(256, 6, 1, 128, 0).check(T, idx)


def test_wide_shared_expert_and_many_experts():
    Layer(256, 512, 4, 128, 640, seed=9).check(48, random_routing(48, 4, 512, 4))


@pytest.mark.parametrize("rows,H", [(1, 128), (3, 256), (64, 7168), (7, 8192), (5, 8320), (2, 20480), (300, 1024)])
def test_quantiser(rows, H):
    rng = np.random.default_rng(rows + H)
    x = block.bf16((rng.standard_normal((rows, H)) * np.exp(3 * rng.standard_normal((rows, 1)))).astype(np.float32))
    x[0, : H // 2] = x[0].max() / 2          # exact halves of the largest: ties
    if rows > 2:
        x[1] = 0.0
        x[2] = block.bf16(x[2] * np.float32(2.0 ** 118) / np.abs(x[2]).max())
    C = _cfg(H=H)
    xq = torch.full((rows + 1, H), 77, dtype=torch.uint8, device=DEV)
    xs = torch.full((rows + 1,), 77.0, device=DEV)
    moe.moe_quantize_act(C, rows, _bf16_dev(x), xq, xs)
    sync()
    q, s = block.quantize_int8(x)
    assert np.array_equal(xq[:rows].view(torch.int8).cpu().numpy(), q)
    assert np.array_equal(host(xs)[:rows], np.where(s == 1.0, 1.0, (np.abs(x).max(1).astype(np.float32) / np.float32(127))))
    assert (xq[rows] == 77).all() and float(xs[rows]) == 77.0


def test_quantiser_at_the_ends_of_the_range():
    x = np.zeros((5, 128), np.float32)
    x[0, :3] = block.bf16(np.array([3.3e38, 1.65e38, -3.3e38], np.float32))   # 127 x overflows
    x[1, :2] = np.float32(2.0 ** -126), np.float32(2.0 ** -127)
    x[2, 5] = np.nan
    x[3, 6] = -np.inf
    x[4, 7] = 1.0
    xq, xs = torch.empty(5, 128, dtype=torch.uint8, device=DEV), torch.empty(5, device=DEV)
    moe.moe_quantize_act(_cfg(H=128), 5, _bf16_dev(x), xq, xs)
    sync()
    q, s = xq.view(torch.int8).cpu().numpy(), host(xs)
    assert q[0, :3].tolist() == [127, 64, -127] and q[1, :2].tolist() == [127, 64]
    assert np.isnan(s[2]) and np.isnan(s[3]) and (q[2:4] == 0).all()
    assert q[4, 7] == 127 and s[4] == np.float32(1 / 127)


def test_a_token_that_is_not_finite_stays_in_its_rows():
    L, T = Layer(256, 4, 2, 128, 128), 40
    idx, x = random_routing(T, 2, 4, 0), L.rows(T)
    y, ys, _, perm = L.run(T, x, idx)
    x2 = x.copy()
    x2[7, 3], x2[11, 200] = np.nan, np.inf
    z, zs, _, _ = L.run(T, x2, idx)
    hit = np.isin(perm // 2, (7, 11))
    assert np.isnan(host(z)[:80][hit]).all() and torch.equal(z[:80][_dev(~hit)], y[:80][_dev(~hit)])
    assert np.isnan(host(zs)[[7, 11]]).all() and torch.equal(zs[:7], ys[:7])


@pytest.mark.parametrize("name,shape", [("w13", (4, 256, 256)), ("w2", (4, 256, 128)), ("ws13", (256, 256)),
                                        ("ws2", (256, 128))])
def test_quantise_weight(name, shape):
    w = block.bf16(np.random.default_rng(1).standard_normal(shape).astype(np.float32))
    w[..., 3, :] = 0.0
    codes = torch.empty(shape, dtype=torch.int8, device=DEV)
    scales = torch.empty(shape[:-1], dtype=torch.float32, device=DEV)
    moe.moe_quantize_weight(_cfg(), WHICH[name], _bf16_dev(w), codes, scales)
    sync()
    q, s = block.quantize_int8(w)
    assert np.array_equal(codes.cpu().numpy(), q)
    assert np.all(np.abs(host(scales) - s) <= 2.0 ** -24 * s)


@pytest.mark.parametrize("T", [1, 8, 32, 33, 200])
def test_layer_and_its_variants(T):
    """moe_forward on 8-bit experts is its parts; the overlapped, no-allocation and captured forms give its bits."""
    H, E, K, I, Is = 256, 8, 2, 128, 256
    L = Layer(H, E, K, I, Is, seed=3)
    rng = np.random.default_rng(T)
    gw, bias = _dev((rng.standard_normal((E, H)) / 16).astype(np.float32)), _dev((0.01 * rng.standard_normal(E)).astype(np.float32))
    W = moe.weights(gate_w=gw, bias=bias, packed=True, **L.kw)
    x = _bf16_dev(L.rows(T))
    ws = torch.full((moe.moe_workspace_bytes(L.C, T),), 0xFF, dtype=torch.uint8, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    idx, cnt, perm = torch.empty(T, K, **i32), torch.empty(E, **i32), torch.empty(T * K, **i32)
    tw, out = torch.empty(T, K, device=DEV), torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    moe.moe_forward(L.C, T, x, W, out, ws, topk_idx=idx, topk_w=tw, counts=cnt, perm=perm)
    off, pos, pm, cn = torch.empty(E + 1, **i32), torch.empty(T * K, **i32), torch.empty_like(perm), torch.empty_like(cnt)
    moe.moe_permute(L.C, T, idx, cn, off, pm, pos, ws)
    y, ys, ref = (torch.empty(n, H, dtype=torch.bfloat16, device=DEV) for n in (T * K, T, T))
    moe.moe_expert_ffn(L.C, T, x, pm, off, W, y, ys, ws)
    moe.moe_combine(L.C, T, y, ys, pos, tw, ref)
    sync()
    assert torch.equal(perm, pm) and torch.equal(out, ref) and out.float().abs().max() > 0
    side = torch.cuda.Stream()
    for f in ("overlap", "noalloc"):
        o = torch.full_like(out, float("nan"))
        if f == "overlap":
            moe.moe_forward_overlap(L.C, T, x, W, o, ws, side)
        else:
            moe.moe_forward_noalloc(L.C, T, x, W, o)
        sync()
        assert torch.equal(o, out), f
    g, o = torch.cuda.CUDAGraph(), torch.full_like(out, float("nan"))
    with torch.cuda.graph(g):
        moe.moe_forward(L.C, T, x, W, o, ws)
    for _ in range(3):
        o.fill_(float("nan"))
        ws.fill_(0xFF)
        g.replay()
        moe.moe_forward_noalloc(L.C, T, x, W, ref)
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(ref, out)
