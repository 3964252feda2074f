"""The feed-forward block of dense layers and its backward on the GPU against
the 64-bit formulas, value by value.

Tolerances.  Every rounding to bf16 is off by at most u = 2^-8 of the value, a
sum of n fp32 products by at most n 2^-24 of the sum of their magnitudes (and
the exponential with its quotient by far less than 2^-18).  Carried through
the formulas with |silu'| <= 1.1 and |silu''| <= 0.5 this gives a bound for
each output value; no rounding is counted that the kernels do not make."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_30_amd as moe
from oracle import block

from gpu_util import DEV, host, log, rel_l2, sync

pytestmark = pytest.mark.gpu

U, F = 2.0 ** -8, 2.0 ** -18
GUARD = 3


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(torch.bfloat16)


def _sum(n):
    return n * 2.0 ** -24


class Block:
    def __init__(self, T, H, I, seed=0, scale=1.0):
        rng = np.random.default_rng(seed + 1000 * T + H + I)
        self.T, self.H, self.I = T, H, I
        self.x = block.bf16(scale * rng.standard_normal((T, H)).astype(np.float32))
        self.w13 = block.bf16((rng.standard_normal((2 * I, H)) / np.sqrt(H)).astype(np.float32))
        self.w2 = block.bf16((rng.standard_normal((H, I)) / np.sqrt(I)).astype(np.float32))
        self.dy = block.bf16(rng.standard_normal((T, H)).astype(np.float32))
        self.C = moe.config(H, 2, 1, 1, 1, 64, I, 1.0, "bf16", "bf16")
        self.dev = {k: _bf16(getattr(self, k)) for k in ("x", "w13", "w2", "dy")}
        self.W = moe.weights(ws13=self.dev["w13"], ws2=self.dev["w2"])

    def ws(self, backward=False):
        f = moe.moe_dense_ffn_backward_workspace_bytes if backward else moe.moe_dense_ffn_workspace_bytes
        return torch.full((f(self.C, self.T),), 0xFF, dtype=torch.uint8, device=DEV)

    def rows(self, n, cols, dtype=torch.bfloat16):
        """n rows and some behind them that no call may touch."""
        return torch.full((n + GUARD, cols), float("nan"), dtype=dtype, device=DEV)

    def forward(self, keep=True):
        y, gu = self.rows(self.T, self.H), self.rows(self.T, 2 * self.I, torch.float32) if keep else None
        moe.moe_dense_ffn(self.C, self.T, self.dev["x"], self.W, y, self.ws(), gu=gu)
        return y, gu

    def backward(self, gu, dx=True):
        out = {"dx": self.rows(self.T, self.H) if dx else None, "dw13": self.rows(2 * self.I, self.H),
               "dw2": self.rows(self.H, self.I)}
        moe.moe_dense_ffn_backward(self.C, self.T, self.dev["x"], self.W, self.dev["dy"], out["dx"], out["dw13"],
                                   out["dw2"], self.ws(True), gu=gu)
        return out

    def bounds(self):
        """Values and bounds of everything, in 64 bits."""
        x, w13, w2, dy = (np.asarray(a, np.float64) for a in (self.x, self.w13, self.w2, self.dy))
        a = np.abs
        g, u = np.split(x @ w13.T, 2, axis=1)
        dg_, du_ = (_sum(self.H) * t for t in np.split(a(x) @ a(w13).T, 2, axis=1))   # of the fp32 sums
        s = 1 / (1 + np.exp(-g))
        silu = g * s
        h = silu * u
        eh = 1.1 * dg_ * a(u) + a(silu) * du_ + F * a(h)
        eh16 = eh + U * (a(h) + eh)
        y = h @ w2.T
        ey = eh16 @ a(w2).T + _sum(self.I) * ((a(h) + eh16) @ a(w2).T)
        r = {"y": (y, ey + U * (a(y) + ey)), "gu": (np.concatenate([g, u], 1),
             np.concatenate([dg_, du_], 1))}
        # backward from the kept g, u
        eg, eu = np.split(r["gu"][1], 2, axis=1)
        dh = dy @ w2
        edh = _sum(self.H) * (a(dy) @ a(w2))
        d1 = s + g * s * (1 - s)
        dg, du = dh * u * d1, dh * silu
        m = a(dh) + edh   # second-order products of errors are inside the larger factor
        edg = edh * (a(u) + eu) * (a(d1) + 0.5 * eg) + m * eu * (a(d1) + 0.5 * eg) + m * a(u) * 0.5 * eg + F * a(dg)
        edu = edh * (a(silu) + 1.1 * eg) + m * 1.1 * eg + F * a(du)
        hb = 1.1 * eg * (a(u) + eu) + (a(silu)) * eu + F * a(h)
        hb = hb + U * (a(h) + hb)
        da = np.concatenate([dg, du], 1)
        eda = np.concatenate([edg, edu], 1)
        eda = eda + U * (a(da) + eda)
        for name, v, e, n in (("dx", da @ w13, (eda, a(da), a(w13)), 2 * self.I),):
            err = e[0] @ e[2] + _sum(n) * ((e[1] + e[0]) @ e[2])
            r[name] = (v, err + U * (a(v) + err))
        v = da.T @ x
        err = eda.T @ a(x) + _sum(self.T) * ((a(da) + eda).T @ a(x))
        r["dw13"] = (v, err + U * (a(v) + err))
        v = dy.T @ h
        err = a(dy).T @ hb + _sum(self.T) * (a(dy).T @ (a(h) + hb))
        r["dw2"] = (v, err + U * (a(v) + err))
        return r


def _check(name, got, ref):
    n = ref[0].shape[0]
    g = host(got)
    d = np.abs(g[:n] - ref[0])
    log(f"{name}: rel L2 {rel_l2(g[:n], ref[0]) if ref[0].any() else 0:.2e}, worst share of the bound {np.max(d / (ref[1] + 1e-300)):.2f}")
    assert np.all(d <= ref[1]), name
    assert np.isnan(g[n:]).all(), f"{name}: rows behind the last were written"


SHAPES = [(1, 64, 64), (2, 320, 192), (16, 256, 512), (17, 192, 128), (31, 512, 64), (63, 64, 320), (64, 320, 320), (65, 128, 576),
          (129, 576, 192), (255, 256, 256), (257, 320, 128), (300, 128, 1088), (513, 64, 64), (33, 1088, 128)]


@pytest.mark.parametrize("T,H,I", SHAPES)
def test_forward_and_backward(T, H, I):
    b = Block(T, H, I)
    ref = b.bounds()
    y, gu = b.forward()
    sync()
    _check("y", y, ref["y"])
    _check("gu", gu, ref["gu"])
    y2, _ = b.forward(keep=False)
    out = b.backward(gu[:T])
    again = b.backward(None)   # g and u computed again
    only = b.backward(gu[:T], dx=False)
    sync()
    assert torch.equal(y[:T], y2[:T])
    for k in ("dx", "dw13", "dw2"):
        _check(k, out[k], ref[k])
        n = ref[k][0].shape[0]
        assert torch.equal(out[k][:n], again[k][:n]), k
        if k != "dx":
            assert torch.equal(out[k][:n], only[k][:n]), k


def test_formula_is_the_oracle():
    b = Block(9, 128, 64)
    r = b.bounds()
    dx, dw13, dw2 = block.swiglu_backward(b.x, b.w13, b.w2, b.dy)
    for k, v in (("y", block.swiglu(b.x, b.w13, b.w2)), ("dx", dx), ("dw13", dw13), ("dw2", dw2)):
        assert np.allclose(r[k][0], v, rtol=1e-12, atol=1e-12)


def test_large_gates_saturate():
    """silu far out on both sides: no NaN from the exponential."""
    b = Block(40, 128, 128, scale=60.0)
    y, gu = b.forward()
    out = b.backward(gu[:40])
    sync()
    ref = b.bounds()
    assert np.abs(ref["gu"][0]).max() > 150
    for k, t in (("y", y), ("dx", out["dx"]), ("dw13", out["dw13"]), ("dw2", out["dw2"])):
        g = host(t)[:ref[k][0].shape[0]]
        assert np.isfinite(g).all() and np.all(np.abs(g - ref[k][0]) <= ref[k][1]), k


def test_a_row_of_nan_stays_in_its_row():
    b = Block(70, 192, 192)
    b.dev["x"][33] = float("nan")
    y, _ = b.forward()
    sync()
    bad = np.isnan(host(y)[:70]).any(axis=1)
    assert bad[33] and bad.sum() == 1
    assert np.isnan(host(y)[33]).all()


def test_no_tokens():
    b = Block(1, 128, 192)
    out = {k: torch.full(s, 7.0, dtype=torch.bfloat16, device=DEV) for k, s in (("dw13", (384, 128)), ("dw2", (128, 192)))}
    moe.moe_dense_ffn(b.C, 0, None, b.W, None, None)
    moe.moe_dense_ffn_backward(b.C, 0, None, b.W, None, None, out["dw13"], out["dw2"], None)
    sync()
    assert all((t == 0).all() for t in out.values())


def test_dx_over_dy():
    b = Block(100, 128, 192)
    _, gu = b.forward()
    out = b.backward(gu[:100])
    dy = b.dev["dy"].clone()
    dw13, dw2 = torch.empty_like(b.dev["w13"]), torch.empty_like(b.dev["w2"])
    moe.moe_dense_ffn_backward(b.C, 100, b.dev["x"], b.W, dy, dy, dw13, dw2, b.ws(True), gu=gu[:100])
    sync()
    assert torch.equal(dy, out["dx"][:100]) and torch.equal(dw2, out["dw2"][:128])


@pytest.mark.parametrize("T", [3, 150])
def test_captured_and_on_another_stream(T):
    b = Block(T, 256, 320)
    y, gu = b.forward()
    out = b.backward(gu[:T])
    sync()
    want = [t.clone() for t in (y, gu, *out.values())]
    ws, wsb = b.ws(), b.ws(True)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.moe_dense_ffn(b.C, T, b.dev["x"], b.W, y, ws, gu=gu)
        moe.moe_dense_ffn_backward(b.C, T, b.dev["x"], b.W, b.dev["dy"], out["dx"], out["dw13"], out["dw2"], wsb,
                                   gu=gu[:T])
    for _ in range(3):
        for t in (y, gu, *out.values()):
            t.fill_(float("nan"))
        ws.fill_(0xFF)
        wsb.fill_(0xFF)
        g.replay()
        b.forward()   # the program's own work in between
        torch.cuda.synchronize()
        for t, w in zip((y, gu, *out.values()), want):
            assert torch.equal(t[:-GUARD], w[:-GUARD])
    with torch.cuda.stream(s):
        y2, _ = b.forward()
    s.synchronize()
    assert torch.equal(y2[:T], want[0][:T])


@pytest.mark.parametrize("wd,packed", [("bf16", True), ("fp8", False), ("fp8", True), ("fp8e8m0", True), ("int4g128", True),
                                       ("int4g32", True), ("f32", False), ("int8", True)])
@pytest.mark.parametrize("T", [1, 40, 200])
def test_other_weights_are_the_shared_expert(wd, packed, T):
    """Every other weight type: the bits that the shared expert of a routed layer gives."""
    H, I, E, K = 256, 384, 4, 2
    rng = np.random.default_rng(T)
    act = "f32" if wd == "f32" else "bf16"
    dt = torch.float32 if wd == "f32" else torch.bfloat16
    C = moe.config(H, E, 1, 1, K, 128, I, 1.0, act, wd)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(DEV).to(dt)
    w, keep = {}, []
    for name, which, shape in (("w13", moe.MOE_W13, (E, 256, H)), ("w2", moe.MOE_W2, (E, H, 128)),
                               ("ws13", moe.MOE_WS13, (2 * I, H)), ("ws2", moe.MOE_WS2, (H, I))):
        m = torch.from_numpy((rng.standard_normal(shape) / np.sqrt(shape[-1])).astype(np.float32)).to(DEV)
        if wd.startswith("int4"):
            g = 32 if wd == "int4g32" else 128
            q = torch.empty(*shape[:-1], shape[-1] // 2, dtype=torch.uint8, device=DEV)
            s = torch.empty(*shape[:-1], shape[-1] // g, dtype=torch.bfloat16, device=DEV)
            moe.moe_quantize_weight(C, which, m.bfloat16(), q, s)
            w[name] = torch.empty(moe.moe_packed_bytes(C, which), dtype=torch.uint8, device=DEV)
            moe.moe_pack_quantized(C, which, q, s, w[name])
        elif wd == "int8":
            q = torch.empty(shape, dtype=torch.int8, device=DEV)
            w[name + "_scale"] = torch.empty(shape[:-1], dtype=torch.float32, device=DEV)
            moe.moe_quantize_weight(C, which, m.bfloat16(), q, w[name + "_scale"])
            w[name] = torch.empty(moe.moe_packed_bytes(C, which), dtype=torch.uint8, device=DEV)
            moe.moe_pack_weight(C, which, q, w[name])
        else:
            if wd.startswith("fp8"):
                w[name + "_scale"] = torch.full((*shape[:-2], shape[-2] // 128, shape[-1] // 128), 0.125, device=DEV)
                m = (m / 0.125).to(torch.float8_e4m3fn).view(torch.uint8)
            elif wd == "bf16":
                m = m.bfloat16()
            w[name] = m
            if packed:
                w[name] = torch.empty(moe.moe_packed_bytes(C, which), dtype=torch.uint8, device=DEV)
                moe.moe_pack_weight(C, which, m, w[name])
        keep.append(m)
    W = moe.weights(packed=packed, **w)
    idx = torch.arange(T * K, dtype=torch.int32, device=DEV).reshape(T, K) % E
    cnt, off = torch.empty(E, dtype=torch.int32, device=DEV), torch.empty(E + 1, dtype=torch.int32, device=DEV)
    perm, pos = (torch.empty(T * K, dtype=torch.int32, device=DEV) for _ in range(2))
    ws = torch.empty(moe.moe_workspace_bytes(C, T), dtype=torch.uint8, device=DEV)
    moe.moe_permute(C, T, idx, cnt, off, perm, pos, ws)
    y, ys, yd = (torch.full((n, H), float("nan"), dtype=dt, device=DEV) for n in (T * K, T, T + GUARD))
    moe.moe_expert_ffn(C, T, x, perm, off, W, y, ys, ws)
    D = moe.weights(packed=packed, **{k: v for k, v in w.items() if k.startswith("ws")})
    wd_ws = torch.full((moe.moe_dense_ffn_workspace_bytes(C, T),), 0xFF, dtype=torch.uint8, device=DEV)
    moe.moe_dense_ffn(C, T, x, D, yd, wd_ws)
    sync()
    assert torch.equal(yd[:T], ys) and torch.isnan(yd[T:]).all()
    assert torch.isfinite(ys.float()).all() and ys.float().abs().max() > 0
