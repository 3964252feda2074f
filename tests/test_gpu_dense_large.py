"""Dense layers at sizes that take every kind of tile and many ranges of k,
against the formulas in 64 bits on the GPU, value by value.

The bounds are those of small layers: every rounding to bf16 is off by at most
2^-8 of the value, a sum of n fp32 products by n 2^-24 of the sum of their
magnitudes, the exponential with its quotient by far less than 2^-18, carried
through the formulas with |silu'| <= 1.1 and |silu''| <= 0.5.  Over thousands of
terms that bound is far above what roundings add up to, so the 2-norm of the
differences is held too: the output's rounding is at most 2^-8 of it, and that of
h or [dg du], different in every term, adds at most as much on average (a k step
of 64 left out of 8192 would be 9%)."""
import pytest
import torch

import sparse_mixture_experts_30_amd as moe

from gpu_util import DEV, log

pytestmark = pytest.mark.gpu

U, F, E = 2.0 ** -8, 2.0 ** -18, 2.0 ** -24
GUARD = 2


def _rand(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def _room(n, cols, dtype=torch.bfloat16):
    return torch.full((n + GUARD, cols), float("nan"), dtype=dtype, device=DEV)


def _check(name, got, value, bound):
    n = value.shape[0]
    d = (got[:n].double() - value).abs()
    assert torch.isfinite(got[:n]).all(), name
    rel = float(d.norm() / value.norm())
    log(f"{name}: rel L2 {rel:.2e}, worst share of the bound {float((d / bound).max()):.2f}")
    assert torch.all(d <= bound) and rel <= 2 * U, name
    assert torch.isnan(got[n:]).all(), f"{name}: rows behind the last were written"


def _out(v, e):
    """Bound of a value that is rounded to bf16 at the end."""
    return e + U * (v.abs() + e) + 1e-300


@pytest.mark.parametrize("T,H,I", [
    (4001, 4032, 4032),    # tiles of 256 in every product, ragged all round
    (2100, 2112, 2752),    # tiles of 256 and of 128, ranges of k
    (1031, 4096, 1088),
    (300, 1024, 2752),     # tiles of 64 rows for dh, nine and ten ranges of k
    (40, 1088, 8128),      # sixteen ranges
    (3001, 64, 64),        # sixteen ranges of the tokens
    (70001, 64, 128),      # very many rows
    (1, 8192, 64),
])
def test_forward_and_backward(T, H, I):
    g = torch.Generator(device=DEV).manual_seed(T + H + I)
    x, dy = _rand(g, T, H), _rand(g, T, H)
    w13, w2 = _rand(g, 2 * I, H, scale=H ** -0.5), _rand(g, H, I, scale=I ** -0.5)
    C, W = moe.config(H, 2, 1, 1, 1, 64, I, 1.0, "bf16", "bf16"), moe.weights(ws13=w13, ws2=w2)
    ws = torch.full((max(moe.moe_dense_ffn_workspace_bytes(C, T), moe.moe_dense_ffn_backward_workspace_bytes(C, T)),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    y, gu, dx = _room(T, H), _room(T, 2 * I, torch.float32), _room(T, H)
    dw13, dw2 = _room(2 * I, H), _room(H, I)
    moe.moe_dense_ffn(C, T, x, W, y, ws, gu=gu)
    ws.fill_(0xFF)
    moe.moe_dense_ffn_backward(C, T, x, W, dy, dx, dw13, dw2, ws, gu=gu)
    torch.cuda.synchronize()

    x, dy, w13, w2 = (t.double() for t in (x, dy, w13, w2))
    proj = x @ w13.T
    eproj = H * E * (x.abs() @ w13.abs().T)
    _check("gu", gu, proj, eproj + 1e-300)
    (gt, u), (eg, eu) = proj.chunk(2, 1), eproj.chunk(2, 1)
    s = torch.sigmoid(gt)
    silu, d1 = gt * s, s + gt * s * (1 - s)
    h = silu * u
    eh = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + F * h.abs()
    eh = eh + U * (h.abs() + eh)
    v = h @ w2.T
    _check("y", y, v, _out(v, eh @ w2.abs().T + I * E * ((h.abs() + eh) @ w2.abs().T)))
    dh, edh = dy @ w2, H * E * (dy.abs() @ w2.abs())
    dg, du = dh * u * d1, dh * silu
    m = dh.abs() + edh
    edg = edh * (u.abs() + eu) * (d1.abs() + 0.5 * eg) + m * eu * (d1.abs() + 0.5 * eg) + m * u.abs() * 0.5 * eg + F * dg.abs()
    edu = edh * (silu.abs() + 1.1 * eg) + m * 1.1 * eg + F * du.abs()
    da, eda = torch.cat([dg, du], 1), torch.cat([edg, edu], 1)
    eda = eda + U * (da.abs() + eda)
    v = da @ w13
    _check("dx", dx, v, _out(v, eda @ w13.abs() + 2 * I * E * ((da.abs() + eda) @ w13.abs())))
    v = da.T @ x
    _check("dw13", dw13, v, _out(v, eda.T @ x.abs() + T * E * ((da.abs() + eda).T @ x.abs())))
    v = dy.T @ h
    _check("dw2", dw2, v, _out(v, dy.abs().T @ eh + T * E * (dy.abs().T @ (h.abs() + eh))))


def test_in_place_and_without_dx_are_the_same_bits():
    """dx over dy, and no dx at all, where the three gradients otherwise share a launch and where they do not."""
    for T, H, I in ((300, 1024, 2752), (4001, 2048, 2816)):
        g = torch.Generator(device=DEV).manual_seed(T)
        x, dy = _rand(g, T, H), _rand(g, T, H)
        w13, w2 = _rand(g, 2 * I, H, scale=H ** -0.5), _rand(g, H, I, scale=I ** -0.5)
        C, W = moe.config(H, 2, 1, 1, 1, 64, I, 1.0, "bf16", "bf16"), moe.weights(ws13=w13, ws2=w2)
        ws = torch.empty(moe.moe_dense_ffn_backward_workspace_bytes(C, T), dtype=torch.uint8, device=DEV)
        outs = []
        for dx in (torch.empty_like(x), dy.clone(), None):
            dw13, dw2 = torch.empty_like(w13), torch.empty_like(w2)
            d = dx if dx is not None and not outs == [] else dy
            moe.moe_dense_ffn_backward(C, T, x, W, d, dx, dw13, dw2, ws)
            outs.append((dx, dw13, dw2))
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], outs[1][0])
        assert all(torch.equal(outs[0][i], o[i]) for o in outs[1:] for i in (1, 2))


def test_more_than_two_billion_values():
    """Offsets past 31 and 32 bits: rows from the start, around the middle and at the end, and the weights' gradients."""
    T, H, I = (1 << 20) + 77, 2112, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    for c in x.split(1 << 16):
        c.copy_(torch.randn(c.shape, generator=g, device=DEV))
    dy = x.roll(1, 0)
    w13, w2 = _rand(g, 2 * I, H, scale=H ** -0.5), _rand(g, H, I, scale=I ** -0.5)
    C, W = moe.config(H, 2, 1, 1, 1, 64, I, 1.0, "bf16", "bf16"), moe.weights(ws13=w13, ws2=w2)
    ws = torch.empty(max(moe.moe_dense_ffn_workspace_bytes(C, T), moe.moe_dense_ffn_backward_workspace_bytes(C, T)),
                     dtype=torch.uint8, device=DEV)
    y, gu, dx = _room(T, H), _room(T, 2 * I, torch.float32), _room(T, H)
    dw13, dw2 = torch.empty_like(w13), torch.empty_like(w2)
    moe.moe_dense_ffn(C, T, x, W, y, ws, gu=gu)
    moe.moe_dense_ffn_backward(C, T, x, W, dy, dx, dw13, dw2, ws, gu=gu)
    torch.cuda.synchronize()
    a, b = w13.double(), w2.double()
    rdw13, rdw2 = torch.zeros_like(a), torch.zeros_like(b)

    def ref(r):
        xr, dyr = x[r].double(), dy[r].double()
        gt, u = (xr @ a.T).chunk(2, 1)
        s = torch.sigmoid(gt)
        dh = dyr @ b
        da = torch.cat([dh * u * (s + gt * s * (1 - s)), dh * gt * s], 1)
        return xr, dyr, gt * s * u, da

    for at in range(0, T, 1 << 16):
        r = slice(at, min(T, at + (1 << 16)))
        xr, dyr, h, da = ref(r)
        rdw13 += da.T @ xr
        rdw2 += dyr.T @ h
        # the 2-norm of two roundings each
        for got, want in ((y[r], h @ b.T), (dx[r], da @ a)):
            assert float((got.double() - want).norm() / want.norm()) <= 2 * U, at
    for got, want in ((dw13, rdw13), (dw2, rdw2)):
        # beside the two roundings those of an fp32 sum of T terms, each at most 2^-24 of the sum so far and as often up
        # as down: sqrt(T) 2^-24 of the result on average, with room of 16
        assert float((got.double() - want).norm() / want.norm()) <= 2 * U + T ** 0.5 * E * 16
    assert torch.isnan(y[T:]).all() and torch.isnan(dx[T:]).all() and torch.isnan(gu[T:]).all()
