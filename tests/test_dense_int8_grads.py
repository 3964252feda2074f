"""The 64-bit references of dense layers, 8-bit experts and gradient clipping
against central differences and hand-worked values, and the refusals of their
entry points (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_mixture_experts_30_amd as moe
from oracle import block

FAKE = 0x1000  # never dereferenced: every call below fails validation first
INV, UNS, WS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE, moe.MOE_OK


def _cfg(H=256, E=8, K=2, I=128, Is=128, act="bf16", wd="bf16"):
    return moe.config(H, E, 1, 1, K, I, Is, 1.0, act, wd)


def _call(name, cfg, *args):
    return getattr(moe.lib(), name)(ctypes.byref(cfg), *args, None)


def _differences(f, a, h=1e-6):
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        p, m = a.copy(), a.copy()
        p[i] += h
        m[i] -= h
        g[i] = (f(p) - f(m)) / (2 * h)
    return g


def test_swiglu_gradient_is_the_forwards_difference():
    rng = np.random.default_rng(0)
    x, w13, w2, dy = (rng.standard_normal(s) for s in ((3, 4), (10, 4), (4, 5), (3, 4)))
    dx, dw13, dw2 = block.swiglu_backward(x, w13, w2, dy)
    # difference of step h: truncation h^2 ~ 1e-12, rounding 1e-16 / h ~ 1e-10
    for got, f, at in ((dx, lambda a: (dy * block.swiglu(a, w13, w2)).sum(), x),
                       (dw13, lambda a: (dy * block.swiglu(x, a, w2)).sum(), w13),
                       (dw2, lambda a: (dy * block.swiglu(x, w13, a)).sum(), w2)):
        assert np.allclose(got, _differences(f, at), rtol=0, atol=1e-8)


def test_int8_rule_by_hand():
    q, s = block.quantize_int8([[254.0, -254.0, 127.0, 1.0, 3.0, -2.9], [0.0] * 6])
    assert s.tolist() == [2.0, 1.0]
    assert q.tolist() == [[127, -127, 64, 0, 2, -1], [0] * 6]   # 63.5, 0.5 and 1.5 to even
    y = block.int8_product(q[:1], s[:1], [[1, 0, 0, 0, 0, 0], [0, 0, 1, 0, 2, 0]], [0.5, 4.0])
    assert y.tolist() == [[127.0, 2 * 4.0 * (64 + 4)]]


def test_clip_by_hand():
    n, (a, b) = block.clip([np.array([3.0]), np.array([4.0, 0.0])], 1.0)
    assert n == 5.0 and np.allclose([a[0], b[0]], [0.6, 0.8], rtol=1e-6)
    n, (a, b) = block.clip([np.array([3.0]), np.array([4.0])], 6.0)
    assert a[0] == 3.0 and b[0] == 4.0
    n, (a,) = block.clip([np.array([np.inf, 2.0])], 1.0)
    assert n == np.inf and a.tolist() == [np.inf, 2.0]


# ------------------------------------------------------------------- dense

def _dense(cfg, T=4, x=FAKE, w=None, gu=FAKE, y=FAKE, ws=FAKE * 256, n=1 << 50):
    w = w or moe.weights(ws13=FAKE, ws2=FAKE)
    return moe.lib().moe_dense_ffn(ctypes.byref(cfg), T, x, ctypes.byref(w), gu, y, ws, n, None)


def test_dense_refusals():
    c = _cfg()
    for kw in (dict(x=None), dict(y=None), dict(T=-1), dict(w=moe.weights(ws13=FAKE)), dict(w=moe.weights(ws2=FAKE)),
               dict(x=FAKE + 8), dict(y=FAKE + 8), dict(gu=FAKE + 8), dict(w=moe.weights(ws13=FAKE + 8, ws2=FAKE)),
               dict(w=moe.weights(ws13=FAKE, ws2=FAKE + 8))):
        assert _dense(c, **kw) == INV, kw
    for kw in (dict(ws=None), dict(n=100), dict(ws=FAKE * 256 + 4)):
        assert _dense(c, **kw) == WS, kw
    assert _dense(_cfg(Is=0)) == INV and "shared_intermediate_size" in moe.moe_last_error()
    assert _dense(c, w=moe.weights(ws13=FAKE, ws2=FAKE, packed=True)) == UNS and "gu" in moe.moe_last_error()
    for wd in ("fp8", "int4g128", "int8"):
        assert _dense(_cfg(wd=wd), w=moe.weights(ws13=FAKE, ws2=FAKE, packed=True)) == UNS
        assert _dense(_cfg(wd=wd), gu=None, w=moe.weights(ws2=FAKE, packed=True)) == INV
    assert _dense(_cfg(act="f32", wd="f32")) == UNS
    assert _dense(c, T=0, x=None, y=None, ws=None, n=0) == OK
    assert _dense(c, T=1 << 31) == UNS
    assert _dense(_cfg(H=64, Is=1 << 21)) == UNS and "too large" in moe.moe_last_error()
    for wd in ("fp8", "int8"):   # scales
        assert _dense(_cfg(wd=wd), gu=None, w=moe.weights(ws13=FAKE, ws2=FAKE, ws13_scale=FAKE, packed=True)) == INV
        assert _dense(_cfg(wd=wd), gu=None, n=64,
                      w=moe.weights(ws13=FAKE, ws2=FAKE, ws13_scale=FAKE, ws2_scale=FAKE, packed=True)) == WS
    assert moe.moe_dense_ffn_workspace_bytes(_cfg(Is=0), 4) == 0
    assert moe.moe_dense_ffn_workspace_bytes(c, -1) == 0
    for wd in ("bf16", "fp8", "fp8e8m0", "int4g32", "int8"):
        assert moe.moe_dense_ffn_workspace_bytes(_cfg(wd=wd), 4) >= 4 * 128


def test_binding_refuses_kept_projections_of_two_bytes():
    w, gu = moe.weights(ws13=FAKE, ws2=FAKE), torch.empty(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="float32"):
        moe.moe_dense_ffn(_cfg(), 4, FAKE, w, FAKE, None, gu=gu, stream=0)
    with pytest.raises(ValueError, match="float32"):
        moe.moe_dense_ffn_backward(_cfg(), 4, FAKE, w, FAKE, FAKE, FAKE, FAKE, None, gu=gu, stream=0)


def test_dense_backward_refusals():
    def f(c=_cfg(), T=4, x=FAKE, w=moe.weights(ws13=FAKE, ws2=FAKE), gu=FAKE, dy=FAKE, dx=FAKE, dw13=FAKE, dw2=FAKE,
          ws=FAKE * 256, n=1 << 50):
        return moe.lib().moe_dense_ffn_backward(ctypes.byref(c), T, x, ctypes.byref(w), gu, dy, dx, dw13, dw2, ws, n, None)
    for kw in (dict(x=None), dict(dy=None), dict(dw13=None), dict(dw2=None), dict(T=0, dw2=None), dict(T=-1),
               dict(c=_cfg(Is=0)), dict(w=moe.weights(ws13=FAKE)), dict(w=moe.weights(ws2=FAKE))):
        assert f(**kw) == INV, kw
    for k in ("x", "gu", "dy", "dx", "dw13", "dw2"):
        assert f(**{k: FAKE + 8}) == INV and "aligned" in moe.moe_last_error(), k
    for kw in (dict(ws=None), dict(n=100), dict(ws=FAKE * 256 + 4)):
        assert f(**kw) == WS, kw
    assert f(w=moe.weights(ws13=FAKE, ws2=FAKE, packed=True)) == UNS
    for wd in ("fp8", "fp8e8m0", "int4g128", "int8"):
        assert f(c=_cfg(wd=wd)) == UNS
        assert moe.moe_dense_ffn_backward_workspace_bytes(_cfg(wd=wd), 4) == 0
    assert f(c=_cfg(act="f32", wd="f32")) == UNS
    assert moe.moe_dense_ffn_backward_workspace_bytes(_cfg(), 4) >= 7 * 4 * 128 * 2


# -------------------------------------------------------------------- int8

def test_int8_refusals():
    c, L = _cfg(wd="int8"), moe.lib()
    for kw in (dict(H=192), dict(I=192), dict(Is=64), dict(H=131072 + 128), dict(I=131072 + 128), dict(Is=131072 + 128)):
        assert moe.moe_workspace_bytes(_cfg(wd="int8", **kw), 4) == 0
        assert "128" in moe.moe_last_error() or "131072" in moe.moe_last_error()
    assert moe.moe_workspace_bytes(_cfg(wd="int8", H=131072), 1) > 0
    assert moe.moe_workspace_bytes(_cfg(wd="int8", act="f32"), 4) == 0
    for which, weights in ((moe.MOE_W13, 8 * 256 * 256), (moe.MOE_W2, 8 * 256 * 128), (moe.MOE_WS13, 256 * 256),
                           (moe.MOE_WS2, 256 * 128)):
        assert moe.moe_packed_bytes(c, which) == weights
    for i in range(3):
        args = [FAKE] * 3
        args[i] = None
        assert _call("moe_quantize_weight", c, moe.MOE_W13, *args) == INV
    assert _call("moe_pack_quantized", c, moe.MOE_W13, FAKE, FAKE, FAKE) == UNS
    assert _call("moe_pack_weight", c, moe.MOE_W13, None, FAKE) == INV
    assert _call("moe_pack_weight", c, moe.MOE_W13, FAKE + 8, FAKE) == INV
    assert _call("moe_pack_weight", c, moe.MOE_W13, FAKE, FAKE + 8) == INV
    names = [m + s for m in ("w13", "w2", "ws13", "ws2") for s in ("", "_scale")]

    def ffn(packed=True, x=FAKE, y=FAKE, n=64, **kw):
        w = moe.weights(packed=packed, **{**dict.fromkeys(names, FAKE), **kw})
        return L.moe_expert_ffn(ctypes.byref(c), 4, x, FAKE, FAKE, ctypes.byref(w), y, FAKE, FAKE * 256, n, None)
    assert ffn(packed=False) == UNS and "packed" in moe.moe_last_error()
    assert ffn() == WS
    for k in names:
        assert ffn(**{k: None}) == INV and ffn(**{k: FAKE + 8}) == INV, k
    assert ffn(x=FAKE + 8) == INV and ffn(y=FAKE + 8) == INV
    w = moe.weights(packed=True, gate_w=FAKE, bias=FAKE, **dict.fromkeys(names, FAKE))
    assert L.moe_forward(ctypes.byref(c), 4, FAKE + 8, ctypes.byref(w), FAKE, None, None, None, None, None, FAKE * 256,
                         1 << 40, None) == INV
    # forward only
    assert moe.moe_backward_workspace_bytes(c, 4) == moe.moe_expert_ffn_backward_workspace_bytes(c, 4) == 0
    assert L.moe_forward_decode_fused(ctypes.byref(c), 4, FAKE, ctypes.byref(w), FAKE, None, None, None, None, None,
                                      FAKE * 256, 1 << 40, None) == UNS
    # its rows are not those of the e4m3 calls
    assert _call("moe_dispatch_quantized", c, 4, *[FAKE] * 5) == UNS
    assert _call("moe_add_rmsnorm", c, 4, FAKE, None, FAKE, 1e-6, None, FAKE, FAKE, FAKE) == UNS
    assert _call("moe_add_rmsnorm", c, 4, FAKE, None, None, 1e-6, None, FAKE, None, None) == INV   # bf16 rows: as ever
    # a workgroup of 256 threads a row, fewer than 2^32 threads a launch
    most = (2 ** 32 - 1) // 256
    assert _call("moe_quantize_act", c, most + 1, FAKE, FAKE, FAKE) == UNS
    assert _call("moe_quantize_act", c, most, None, FAKE, FAKE) == INV
    assert moe.moe_workspace_bytes(c, most // 3 + 1) == 0 and moe.moe_workspace_bytes(c, most // 3) > 0
    assert _call("moe_quantize_weight", _cfg(wd="int8", E=512, I=16384), moe.MOE_W13, FAKE, FAKE, FAKE) == UNS


# --------------------------------------------------------------- gradients

def _list(grads, out=None, counts=None, types=None):
    n = len(grads)
    arrays = ((ctypes.c_void_p * n)(*grads), (ctypes.c_void_p * n)(*(out or grads)),
              (ctypes.c_int64 * n)(*(counts or [100] * n)), (ctypes.c_int32 * n)(*(types or [moe.MOE_F32] * n)))
    m = moe.MoeGradients(n, *[ctypes.addressof(a) for a in arrays])
    m.keep = arrays
    return m


def _clip(l, max_norm=1.0, norm=FAKE, given=0, ws=FAKE * 256, n=0):
    """The workspace is refused last: WS means that everything else passed."""
    return moe.lib().moe_clip_grads(ctypes.byref(l), max_norm, norm, given, ws, n, None)


def test_gradient_refusals():
    a, b = 0x10000, 0x20000
    assert _clip(_list([a, b])) == WS
    assert _clip(_list([a, b]), ws=None, n=1 << 30) == WS and _clip(_list([a, b]), ws=FAKE * 256 + 8, n=1 << 30) == WS
    assert _clip(_list([a, b]), norm=None) == INV
    for m in (-1.0, float("nan"), -float("inf")):
        assert _clip(_list([a]), max_norm=m) == INV
    assert _clip(_list([a]), max_norm=float("inf")) == WS
    assert _clip(_list([a, b], counts=[100, -1])) == INV
    assert _clip(_list([a, None])) == INV and _clip(_list([a, None], counts=[100, 0])) == WS
    assert _clip(_list([a, b + 2])) == INV and _clip(_list([a, b + 2], types=[0, 1])) == WS
    assert _clip(_list([a, b], types=[0, moe.MOE_FP8_E4M3])) == UNS
    assert _clip(_list([a, 1 << 50], counts=[100, 1 << 41])) == UNS
    for field in ("grad", "out", "count", "dtype"):
        l = _list([a, b])
        setattr(l, field, None)
        assert _clip(l) == INV
    l = _list([a, b])
    l.n = -1
    assert _clip(l) == INV and moe.moe_grad_norm_workspace_bytes(l) == 0
    L = moe.lib()
    l = _list([a, b])
    l.out = None   # not needed for the norm
    assert L.moe_grad_norm(ctypes.byref(l), FAKE, FAKE * 256, 0, None) == WS
    assert L.moe_grad_norm(ctypes.byref(l), None, FAKE * 256, 1 << 30, None) == INV
    assert L.moe_grad_norm(None, FAKE, FAKE * 256, 1 << 30, None) == INV
    assert moe.moe_grad_norm_workspace_bytes(_list([a])) == 2048 * 8
    # 168 runs a launch, of 2^30 values at most each
    assert moe.moe_grad_norm_workspace_bytes(_list([a] * 168)) == 2 * 2048 * 8
    assert moe.moe_grad_norm_workspace_bytes(_list([a], counts=[168 << 30])) == 2 * 2048 * 8
    assert moe.moe_grad_norm_workspace_bytes(_list([a], types=[9])) == 0


@pytest.mark.parametrize("grads,out,counts,ok", [
    ([0, 400], [0, 400], [100, 100], True),                 # in place, one after another
    ([400, 0], [400, 0], [100, 100], True),                 # the same, unordered
    ([0, 396], [0, 396], [100, 100], False),                # in place, overlapping
    ([0, 0], [0, 0], [100, 100], False),                    # the same gradient twice
    ([0, 0], [4000, 4400], [100, 100], True),               # twice, into two places
    ([0, 400], [4000, 4396], [100, 100], False),            # outputs overlap
    ([0, 400], [400, 0], [100, 100], False),                # swapped: an output is another's gradient
    ([0], [4], [100], False),                               # its own gradient in part
    ([0, 1000, 2000], [5000, 400, 6000], [100] * 3, True),  # an output between gradients
    ([0, 1000, 2000], [5000, 604, 6000], [100] * 3, False),
    ([0, 1000], [0, 5000], [1000, 100], False),             # in place, over another's gradient
    ([0, 1000, 500], [5000, 1000, 7000], [1000, 100, 10], False),
    ([0, 0], [0, 0], [100, 0], True),                       # an empty one overlaps nothing
])
def test_overlapping_outputs_are_refused(grads, out, counts, ok):
    base = 0x100000
    l = _list([base + g for g in grads], [base + o for o in out], counts)
    assert _clip(l) == (WS if ok else INV), moe.moe_last_error()
    if not ok:
        assert "overlaps" in moe.moe_last_error()


def test_overlap_check_against_all_pairs():
    rng = np.random.default_rng(0)
    seen = set()
    for _ in range(400):
        n = int(rng.integers(1, 6))
        grads = [int(v) * 4 for v in rng.integers(0, 60, n)]
        out = [g if rng.random() < 0.5 else int(rng.integers(0, 120)) * 4 for g in grads]
        counts = [int(v) for v in rng.integers(0, 12, n)]
        bad = False
        for i in range(n):
            for j in range(n):
                for other, kind in ((grads[j], "g"), (out[j], "o")):
                    if (i == j and kind == "o") or (i == j and out[i] == grads[i]):
                        continue
                    bad |= counts[i] > 0 and counts[j] > 0 and out[i] < other + 4 * counts[j] and other < out[i] + 4 * counts[i]
        base = 0x100000
        l = _list([base + g for g in grads], [base + o for o in out], counts)
        assert _clip(l) == (INV if bad else WS), (grads, out, counts)
        seen.add(bad)
    assert seen == {True, False}


def test_binding_checks_gradients():
    t = torch.zeros(8, 8)
    with pytest.raises(ValueError, match="contiguous"):
        moe.gradients([t[:, :4]])
    with pytest.raises(ValueError, match="float16"):
        moe.gradients([t.half()])
    with pytest.raises(ValueError, match="outputs"):
        moe.gradients([t], [])
    with pytest.raises(ValueError, match="output of"):
        moe.gradients([t], [t.bfloat16()])
    with pytest.raises(ValueError, match="output of"):
        moe.gradients([t], [t[:4]])
    l = moe.gradients([t, t.bfloat16()])
    assert l.n == 2


@pytest.mark.parametrize("H,I", [(7168, 18432), (2048, 5632), (512, 1024), (7168, 2048), (128, 128)])
def test_a_workspace_for_a_batch_does_for_smaller_ones(H, I):
    for f in (moe.moe_dense_ffn_workspace_bytes, moe.moe_dense_ffn_backward_workspace_bytes):
        for wd in ("bf16", "int8"):
            sizes = [f(_cfg(H=H, Is=I, wd=wd), T) for T in range(0, 5000)]
            assert sizes == sorted(sizes)
