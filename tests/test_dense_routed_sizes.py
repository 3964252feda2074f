"""Dense layers do not depend on the routed sizes of their configuration: neither what is refused nor the
workspace (no GPU)."""
import ctypes

import pytest

import sparse_mixture_experts_30_amd as moe

FAKE = 0x1000  # never dereferenced: every call below fails validation first
INV, UNS, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "fp8"), ("bf16", "fp8e8m0"), ("bf16", "int4g128"), ("bf16", "int4g32"),
         ("bf16", "int8")]
# (E, G, TG, K, I, scaling) of routed layers, some of which no routed call takes
ROUTED = [(8, 1, 1, 2, 128, 1.0), (256, 8, 4, 8, 2048, 2.5), (128, 1, 1, 64, 128, 1.0), (512, 1, 1, 8, 1 << 18, 1.0),
          (1024, 1, 1, 8, 128, 1.0), (8, 1, 1, 100, 72, 1.0), (0, 0, 0, 0, 0, 0.0)]
EXACT = (2, 1, 1, 1, 128, 1.0)


def _cfg(routed, act, wd, H=256, Is=384):
    E, G, TG, K, I, rho = routed
    return moe.config(H, E, G, TG, K, I, Is, rho, act, wd)


def _forward(c, T, n=1):
    """The workspace is refused last: WS means that everything else passed."""
    w = moe.weights(packed=c.weight_dtype not in (moe.MOE_F32, moe.MOE_BF16),
                    **{k: FAKE for k in ("ws13", "ws2", "ws13_scale", "ws2_scale")})
    return moe.lib().moe_dense_ffn(ctypes.byref(c), T, FAKE, ctypes.byref(w), None, FAKE, FAKE * 256, n, None)


def _backward(c, T, n=1):
    w = moe.weights(ws13=FAKE, ws2=FAKE)
    return moe.lib().moe_dense_ffn_backward(ctypes.byref(c), T, FAKE, ctypes.byref(w), None, FAKE, FAKE, FAKE, FAKE,
                                            FAKE * 256, n, None)


@pytest.mark.parametrize("act,wd", TYPES)
@pytest.mark.parametrize("routed", ROUTED)
def test_routed_sizes_take_no_part(act, wd, routed):
    c, d = _cfg(routed, act, wd), _cfg(EXACT, act, wd)
    for T in (1, 40, 5000):
        assert moe.moe_dense_ffn_workspace_bytes(c, T) == moe.moe_dense_ffn_workspace_bytes(d, T) > 0
        assert _forward(c, T) == WS, moe.moe_last_error()
        if wd == "bf16":
            assert moe.moe_dense_ffn_backward_workspace_bytes(c, T) == moe.moe_dense_ffn_backward_workspace_bytes(d, T) > 0
            assert _backward(c, T) == WS, moe.moe_last_error()


@pytest.mark.parametrize("routed", [(256, 8, 4, 8, 2048, 2.5), (128, 1, 1, 64, 128, 1.0)])
def test_most_tokens(routed):
    """8-bit layers quantise T rows in one launch of 256 threads a row; the others count tokens in 31 bits."""
    most = (2 ** 32 - 1) // 256
    c = _cfg(routed, "bf16", "int8")
    assert _forward(c, most) == WS and _forward(c, most + 1) == UNS
    assert moe.moe_dense_ffn_workspace_bytes(c, most) > 0 and moe.moe_dense_ffn_workspace_bytes(c, most + 1) == 0
    c = _cfg(routed, "bf16", "fp8")
    assert _forward(c, 2 ** 31 - 1) == WS and _forward(c, 2 ** 31) == UNS and _forward(c, -1) == INV


def test_its_own_sizes_are_still_checked():
    for wd, kw, status in (("bf16", dict(H=100), UNS), ("int8", dict(Is=64), UNS), ("int8", dict(Is=131072 + 128), UNS),
                           ("bf16", dict(Is=0), INV), ("bf16", dict(H=0), INV), ("bf16", dict(Is=-64), INV)):
        assert _forward(_cfg(ROUTED[0], "bf16", wd, **kw), 4) == status, kw
    assert moe.lib().moe_dense_ffn(None, 4, FAKE, ctypes.byref(moe.weights()), None, FAKE, FAKE * 256, 1, None) == INV
    assert moe.lib().moe_dense_ffn_workspace_bytes(None, 4) == 0
    assert moe.lib().moe_dense_ffn_backward_workspace_bytes(None, 4) == 0
