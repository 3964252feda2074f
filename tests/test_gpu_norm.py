"""Residual add + RMS norm and its backward on the GPU against the 64-bit
reference.

Tolerances.  A row's fp32 sums add at most H / 64 terms in sequence and 16
more in trees, so their relative error is below c = (H / 64 + 16) 2^-24 of the
sum of magnitudes.  One rounding to bf16 is at most 2^-8 of the value, to e4m3
2^-4 of it or 2^-10 of the scale."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_30_amd as moe
from oracle import block

from gpu_util import DEV, host, sync

pytestmark = pytest.mark.gpu

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _cfg(H, act, q=""):
    return moe.config(H, 2, 1, 1, 1, 128, 0, 1.0, act, q or act)


def _rows(seed, T, H, act, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, generator=g) * std).to(DT[act]).to(DEV)


def _weight(seed, H):
    return (1 + 0.2 * torch.randn(H, generator=torch.Generator().manual_seed(seed))).to(DEV)


def _c(H):
    return (H / 64 + 16) * 2.0 ** -24


def _u(act):
    return 2.0 ** -8 if act == "bf16" else 2.0 ** -24


def _forward(cfg, x, res, w, outs=("sum", "y"), act="bf16", stream=None):
    T, H = x.shape
    o = {}
    if "sum" in outs:
        o["sum"] = torch.full_like(x, float("nan"))
    if "y" in outs:
        o["y"] = torch.full_like(x, float("nan"))
    if "q" in outs:
        o["yq"] = torch.full((T, H), 0x55, dtype=torch.uint8, device=DEV)
        o["ys"] = torch.full((T, H // 128), float("nan"), device=DEV)
    moe.moe_add_rmsnorm(cfg, T, x, res, w, EPS, stream=stream, **o)
    sync()
    return o


def _check_y(y, ref, H, act):
    assert np.all(np.abs(host(y) - ref) <= (_u(act) + 8 * _c(H)) * np.abs(ref))


# Every register-held width and the widths past them; rows around a workgroup.
SIZES = [(1, 64), (1, 7168), (2, 128), (3, 192), (33, 1024), (5, 2048), (4, 2112), (7, 4160), (130, 7168), (3, 8192),
         (2, 8256), (2, 16384), (2, 16448), (2, 32768), (2, 32832), (1031, 256),
         (1700, 7168)]   # past the size from which rows are read non-temporally


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SIZES)
def test_forward(T, H, act):
    x, res, w = _rows(1, T, H, act), _rows(2, T, H, act, 3.0), _weight(3, H)
    for r in (res, None):
        o = _forward(_cfg(H, act), x, r, w)
        s = block.stored(host(x) + host(r), act) if r is not None else host(x)
        assert np.array_equal(host(o["sum"]), s)
        _check_y(o["y"], block.rmsnorm(s, host(w), EPS), H, act)


@pytest.mark.parametrize("q", ["fp8", "fp8e8m0"])
@pytest.mark.parametrize("T,H", [(1, 128), (3, 7168), (37, 1024), (2, 2176), (2, 8320), (2, 32896), (515, 384)])
def test_forward_e4m3(T, H, q):
    x, res, w = _rows(4, T, H, "bf16"), _rows(5, T, H, "bf16"), _weight(6, H)
    if T > 2:
        x[1].zero_()
        res[1].zero_()                                        # a row of zeros
    o = _forward(_cfg(H, "bf16", q), x, res, w, ("sum", "y", "q"))
    ref = block.rmsnorm(block.bf16(host(x) + host(res)), host(w), EPS)
    _check_y(o["y"], ref, H, "bf16")
    t = ref.reshape(T, -1, 128)
    a, s = np.abs(t).max(axis=2), host(o["ys"]).astype(np.float64)
    tol = 8 * _c(H) + 2.0 ** -23
    some = a > 0
    assert np.all(s[~some] == 1.0)
    if q == "fp8":
        assert np.all(np.abs(s - a / 448)[some] <= tol * (a / 448)[some])
    else:
        assert np.all(np.frexp(s)[0] == 0.5)                  # powers of two
        assert np.all((a / 448 <= s * (1 + tol))[some]) and np.all((s / 2 < a / 448 * (1 + tol))[some])
    v = host(o["yq"].view(torch.float8_e4m3fn).float()).reshape(t.shape) * s[:, :, None]
    assert np.all(np.abs(v - t) <= (2.0 ** -4 * np.abs(t) + 2.0 ** -10 * s[:, :, None]) * (1 + 1e-4))
    # without y and without sum: the same codes
    p = _forward(_cfg(H, "bf16", q), x, res, w, ("q",))
    assert torch.equal(p["yq"], o["yq"]) and torch.equal(p["ys"], o["ys"])


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1024, 7168, 40960])
def test_sum_in_place(H, act):
    x, res, w = _rows(7, 9, H, act), _rows(8, 9, H, act), _weight(9, H)
    o = _forward(_cfg(H, act), x, res, w)
    for target in ("residual", "x"):
        a, b = x.clone(), res.clone()
        y = torch.empty_like(x)
        moe.moe_add_rmsnorm(_cfg(H, act), 9, a, b, w, EPS, sum=b if target == "residual" else a, y=y)
        sync()
        assert torch.equal(b if target == "residual" else a, o["sum"]) and torch.equal(y, o["y"])


def test_non_finite_rows_stay_in_their_rows():
    H = 1024
    x, w = _rows(10, 6, H, "bf16"), _weight(11, H)
    clean = _forward(_cfg(H, "bf16", "fp8"), x, None, w, ("y", "q"))
    x[1, 5], x[3, 700], x[4, 0] = float("nan"), float("inf"), -float("inf")
    o = _forward(_cfg(H, "bf16", "fp8"), x, None, w, ("y", "q"))
    y, v = host(o["y"]), host(o["yq"].view(torch.float8_e4m3fn).float())
    assert np.all(np.isnan(y[1])) and np.all(np.isnan(v[1]))
    for t, c in ((3, 700), (4, 0)):        # rstd = 0: zeros, and inf * 0
        assert np.isnan(y[t, c]) and np.isnan(v[t, c]) and np.all(np.delete(y[t], c) == 0)
    for t in (0, 2, 5):
        assert np.array_equal(y[t], host(clean["y"])[t])
        assert torch.equal(o["yq"][t], clean["yq"][t]) and torch.equal(o["ys"][t], clean["ys"][t])


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SIZES + [(2051, 512), (1, 40960)])
def test_backward(T, H, act):
    r, dy, ds, w = _rows(12, T, H, act, 2.0), _rows(13, T, H, act), _rows(14, T, H, act), _weight(15, H)
    if T > 2:
        r[2].zero_()
    cfg = _cfg(H, act)
    ws = torch.full((moe.moe_add_rmsnorm_backward_workspace_bytes(cfg, T),), 0xFF, dtype=torch.uint8, device=DEV)
    R, G, W = (host(a).astype(np.float64) for a in (r, dy, w))
    rstd = 1 / np.sqrt((R * R).mean(axis=1, keepdims=True) + EPS)
    n, g = R * rstd, G * W
    for d in (ds, None):
        dx, dw = torch.full_like(r, float("nan")), torch.full((H,), float("nan"), device=DEV)
        moe.moe_add_rmsnorm_backward(cfg, T, r, w, EPS, dy, dx, dw, ws, dsum=d)
        sync()
        ref, refw = block.rmsnorm_backward(R, W, EPS, G, None if d is None else host(d))
        mag = rstd * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True))
        mag += 0 if d is None else np.abs(host(d))
        assert np.all(np.abs(host(dx) - ref) <= 8 * _c(H) * mag + _u(act) * np.abs(ref))
        c = (T + 64) * 2.0 ** -24 + 4 * _c(H)
        assert np.all(np.abs(host(dw) - refw) <= c * np.abs(G * n).sum(axis=0))
        # the same bits again, and in place
        for alias in (dy, d):
            if alias is None:
                continue
            a, b = dy.clone(), None if d is None else d.clone()
            out = a if alias is dy else b
            dw2 = torch.empty_like(dw)
            moe.moe_add_rmsnorm_backward(cfg, T, r, w, EPS, a, out, dw2, ws, dsum=b)
            sync()
            assert torch.equal(out, dx) and torch.equal(dw2, dw)


def test_backward_of_no_rows_is_a_zero_weight_gradient():
    cfg, dw = _cfg(512, "bf16"), torch.full((512,), 7.0, device=DEV)
    moe.moe_add_rmsnorm_backward(cfg, 0, None, None, EPS, None, None, dw, None)
    sync()
    assert torch.count_nonzero(dw) == 0


def test_on_another_stream():
    T, H = 300, 7168
    x, w = _rows(16, T, H, "bf16"), _weight(17, H)
    want = _forward(_cfg(H, "bf16"), x, None, w)["y"]
    s = torch.cuda.Stream()
    y = torch.empty_like(x)
    sync()
    with torch.cuda.stream(s):
        moe.moe_add_rmsnorm(_cfg(H, "bf16"), T, x, None, w, EPS, y=y)
    s.synchronize()
    assert torch.equal(y, want)


# Largest values of a tile around and below those where 448 / a leaves fp32 (1.3e-36), down to its smallest
# number.  Beside the rounding to e4m3, a scale below 2^-126 is rounded by up to 2^-150 and multiplies codes
# up to 448, and y itself is rounded by up to 2^-150 for each of two products: 512 x 2^-150 in all.
@pytest.mark.parametrize("q", ["fp8", "fp8e8m0"])
@pytest.mark.parametrize("H", [1792, 17920])
def test_tiles_of_tiny_values(H, q):
    T, sizes = 3, [1e-34, 1.4e-36, 1.2e-36, 1e-37, 1e-38, 1e-40, 1e-42, 4e-43, 2e-43, 1e-44, 1e-45, 0.0, 1.0, 1e-37]
    x, g = _rows(18, T, H, "bf16").view(T, -1, 128), np.random.default_rng(19)
    x[:, :, 1::2] = 0                                          # zeros beside the tiny values
    x[1, :, 1:] = 0                                            # one value a tile
    x = x.reshape(T, H)
    w = (np.repeat(np.resize(np.array(sizes, np.float32), H // 128), 128) * (0.5 + g.random(H))).astype(np.float32)
    o = _forward(_cfg(H, "bf16", q), x, None, torch.from_numpy(w).to(DEV), ("y", "q"))
    t = block.rmsnorm(host(x), w, EPS).reshape(T, -1, 128)
    a, s = np.abs(t).max(axis=2), host(o["ys"]).astype(np.float64)
    assert np.all(np.isfinite(s)) and np.all(s > 0)
    v = host(o["yq"].view(torch.float8_e4m3fn).float()).astype(np.float64)
    assert np.all(np.isfinite(v)) and np.all(v[host(x) == 0] == 0)
    v = v.reshape(t.shape) * s[:, :, None]
    scale = a / 448 if q == "fp8" else s
    assert np.all(np.abs(v - t) <= (2.0 ** -4 * np.abs(t) + 2.0 ** -10 * scale[:, :, None]) * (1 + 1e-4) + 512 * 2.0 ** -150)


@pytest.mark.parametrize("act,H", [("bf16", 16448), ("f32", 8256)])
def test_wide_backward_of_many_rows(act, H):
    """Rows too wide for registers, three to a workgroup: its share of dweight is read back and added to."""
    T = 1100
    r, dy, w = _rows(20, T, H, act, 2.0), _rows(21, T, H, act), _weight(22, H)
    cfg = _cfg(H, act)
    ws = torch.full((moe.moe_add_rmsnorm_backward_workspace_bytes(cfg, T),), 0xFF, dtype=torch.uint8, device=DEV)
    dx, dw = torch.full_like(r, float("nan")), torch.full((H,), float("nan"), device=DEV)
    moe.moe_add_rmsnorm_backward(cfg, T, r, w, EPS, dy, dx, dw, ws)
    sync()
    R, G, W = (host(a).astype(np.float64) for a in (r, dy, w))
    ref, refw = block.rmsnorm_backward(R, W, EPS, G)
    rstd = 1 / np.sqrt((R * R).mean(axis=1, keepdims=True) + EPS)
    n, g = R * rstd, G * W
    mag = rstd * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True))
    assert np.all(np.abs(host(dx) - ref) <= 8 * _c(H) * mag + _u(act) * np.abs(ref))
    assert np.all(np.abs(host(dw) - refw) <= ((T + 64) * 2.0 ** -24 + 4 * _c(H)) * np.abs(G * n).sum(axis=0))
