"""The many-row kernel of the 8-bit experts, value by value against the 64-bit definition with the bounds of the
few-row tests (codes next to a half may differ by one, sums are exact).  Every case asserts through the kernel timer
that this kernel ran, so that none can drift to the other one.

A layer's 8-bit products take it with more than 16 tokens, more than 14 rows an expert and 256 workgroups or more:
(row tiles of 128, of the routed rows, the experts and the tokens) x max(I, Is) / 128."""
import contextlib

import numpy as np
import pytest
import torch

import sparse_mixture_experts_30_amd as moe

from gpu_util import DEV, host, log, random_routing, rel_l2, sync
from test_gpu_int8 import WHICH, Layer, _bf16_dev, _dev, _swiglu_bounds

pytestmark = pytest.mark.gpu

# Rows of the experts: tiles of one to four blocks of 32 rows, whole and one row around, one tile alone or several
# that share a weight tile, none at all; 1534 rows.
ROWS = [1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 257, 0, 316]


@contextlib.contextmanager
def only_many():
    """The 8-bit products inside all run in the many-row kernel."""
    moe.moe_kernel_timer_read()
    moe.moe_kernel_timer_enable(True)
    try:
        yield
        sync()
    finally:
        moe.moe_kernel_timer_enable(False)
    names = {n for n in moe.moe_kernel_timer_read() if n.startswith("grouped_gemm")}
    assert names == {"grouped_gemm_int8_many<true>", "grouped_gemm_int8_many<false>"}


def _rows_routing(rows, seed):
    idx = np.repeat(np.arange(len(rows), dtype=np.int32), rows)
    np.random.default_rng(seed).shuffle(idx)
    return idx[:, None]


# k steps of gate and up (H / 128) 1 to 7 and 13, of down (I / 128, Is / 128) 1 to 13; H / 128 odd leaves half of
# the down projection's last pair of tiles to no one; the shared expert wider, narrower or absent.
@pytest.mark.parametrize("H,I,Is", [(128, 1024, 128), (256, 128, 1024), (384, 256, 1152), (512, 384, 1024), (640, 1280, 0),
                                    (768, 512, 1024), (896, 640, 1280), (1664, 896, 1664), (384, 1408, 0)])
def test_rows_of_every_tile_height(H, I, Is):
    L = Layer(H, len(ROWS), 1, I, Is, seed=H + I)
    with only_many():
        L.check(sum(ROWS), _rows_routing(ROWS, H), seed=2)


@pytest.mark.parametrize("T,E,K,H,I,Is", [(700, 8, 3, 384, 256, 1152), (257, 4, 4, 256, 2048, 2176), (130, 2, 2, 640, 6528, 6528),
                                          (1000, 32, 2, 256, 512, 640), (97, 4, 2, 128, 8320, 128)])
def test_several_experts_a_token(T, E, K, H, I, Is):
    """Skewed loads: expert 0 has every token.  I = 8320: rows of h that the quantiser does not hold in registers."""
    L = Layer(H, E, K, I, Is, seed=T)
    with only_many():
        L.check(T, random_routing(T, K, E, seed=T, skew=True))


@pytest.mark.parametrize("T,H,Is", [(600, 256, 8320), (1001, 384, 4096), (257, 896, 11008), (4097, 128, 1024)])
def test_dense_layer(T, H, Is):
    L = Layer(H, 2, 1, 128, Is, seed=Is)
    C = moe.config(H, 2, 1, 1, 1, 128, Is, 1.0, "bf16", "int8")
    W = moe.weights(packed=True, **{k: v for k, v in L.kw.items() if k.startswith("ws")})
    x = L.rows(T)
    y = torch.full((T + 3, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.full((moe.moe_dense_ffn_workspace_bytes(C, T),), 0xFF, dtype=torch.uint8, device=DEV)
    with only_many():
        moe.moe_dense_ffn(C, T, _bf16_dev(x), W, y, ws)
    ref, tol = _swiglu_bounds(x, tuple(v[0] for v in L.w["ws13"]), tuple(v[0] for v in L.w["ws2"]))
    g = host(y)
    log(f"dense int8 T={T} H={H} Is={Is}: rel {rel_l2(g[:T], ref):.2e}")
    assert np.all(np.abs(g[:T] - ref) <= tol) and np.isnan(g[T:]).all()


def test_a_token_that_is_not_finite_stays_in_its_rows():
    L, T = Layer(384, 4, 2, 2048, 2176), 500
    idx, x = random_routing(T, 2, 4, 0), L.rows(T)
    x2 = x.copy()
    x2[7, 3], x2[250, 200] = np.nan, np.inf
    with only_many():
        y, ys, _, perm = L.run(T, x, idx)
        z, zs, _, _ = L.run(T, x2, idx)
    hit = np.isin(perm // 2, (7, 250))
    assert np.isnan(host(z)[:2 * T][hit]).all() and torch.equal(z[:2 * T][_dev(~hit)], y[:2 * T][_dev(~hit)])
    rest = _dev(~np.isin(np.arange(T), (7, 250)))
    assert np.isnan(host(zs)[[7, 250]]).all() and torch.equal(zs[:T][rest], ys[:T][rest])


def test_longest_products():
    """Every code 127 along 131072 inputs, in the four waves of a tile at once: g = u = 1 by the choice of scales."""
    H, I, T = 131072, 1024, 4100   # 33 row tiles and 2 experts x 8 column tiles
    C = moe.config(H, 2, 1, 1, 1, I, 0, 1.0, "bf16", "int8")
    kw = {}
    for name, rows, cols, scale in (("w13", 2 * I, H, 1.0 / (127.0 * H)), ("w2", H, I, 2.0 ** -10)):
        q = torch.full((2, rows, cols), 127, dtype=torch.int8, device=DEV)
        kw[name] = torch.empty(moe.moe_packed_bytes(C, WHICH[name]), dtype=torch.uint8, device=DEV)
        moe.moe_pack_weight(C, WHICH[name], q, kw[name])
        kw[name + "_scale"] = torch.full((2, rows), scale, dtype=torch.float32, device=DEV)
    W = moe.weights(packed=True, **kw)
    x = torch.ones(T, H, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    perm = torch.arange(T, dtype=torch.int32, device=DEV)
    y = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(moe.moe_workspace_bytes(C, T), dtype=torch.uint8, device=DEV)
    with only_many():
        moe.moe_expert_ffn(C, T, x, perm, off, W, y, None, ws)
    # silu(1) 127 1024 2^-10, off by half a step of bf16 and a few of fp32 (all rows and columns are alike)
    want = 127.0 / (1.0 + np.exp(-1.0))
    assert (y.float() - want).abs().max().item() <= want * (2.0 ** -8 + 2.0 ** -17)


@pytest.mark.parametrize("T", [300, 777])
def test_layer_and_its_variants(T):
    """moe_forward is its parts; the overlapped, captured and quantised forms give its bits."""
    H, E, K, I, Is = 384, 8, 2, 2048, 2176
    L = Layer(H, E, K, I, Is, seed=3)
    rng = np.random.default_rng(T)
    gw, bias = _dev((rng.standard_normal((E, H)) / 20).astype(np.float32)), _dev((0.01 * rng.standard_normal(E)).astype(np.float32))
    W = moe.weights(gate_w=gw, bias=bias, packed=True, **L.kw)
    x = _bf16_dev(L.rows(T))
    ws = torch.full((moe.moe_workspace_bytes(L.C, T),), 0xFF, dtype=torch.uint8, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    idx, cnt, perm = torch.empty(T, K, **i32), torch.empty(E, **i32), torch.empty(T * K, **i32)
    tw, out = torch.empty(T, K, device=DEV), torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    with only_many():
        moe.moe_forward(L.C, T, x, W, out, ws, topk_idx=idx, topk_w=tw, counts=cnt, perm=perm)
    off, pos, pm, cn = torch.empty(E + 1, **i32), torch.empty(T * K, **i32), torch.empty_like(perm), torch.empty_like(cnt)
    moe.moe_permute(L.C, T, idx, cn, off, pm, pos, ws)
    y, ys, ref = (torch.empty(n, H, dtype=torch.bfloat16, device=DEV) for n in (T * K, T, T))
    xq, xs = torch.empty(T, H, dtype=torch.uint8, device=DEV), torch.empty(T, dtype=torch.float32, device=DEV)
    moe.moe_quantize_act(L.C, T, x, xq, xs)
    with only_many():
        moe.moe_expert_ffn_quantized(L.C, T, xq, xs, pm, off, W, y, ys, ws)
    moe.moe_combine(L.C, T, y, ys, pos, tw, ref)
    sync()
    assert torch.equal(perm, pm) and torch.equal(out, ref) and out.float().abs().max() > 0
    side, o = torch.cuda.Stream(), torch.full_like(out, float("nan"))
    moe.moe_forward_overlap(L.C, T, x, W, o, ws, side)
    sync()
    assert torch.equal(o, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_forward(L.C, T, x, W, o, ws)
    other = torch.empty_like(ws)
    for _ in range(3):
        o.fill_(float("nan"))
        ws.fill_(0xFF)
        g.replay()
        moe.moe_forward(L.C, T, x, W, ref, other)
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(ref, out)


def test_two_streams_at_once():
    """Two layers, each with its own workspace, on streams of their own: the bits of one after the other."""
    layers = [(Layer(384, 4, 2, 2048, 2816, seed=s), 300 + 41 * s) for s in range(2)]
    todo = []
    for L, T in layers:
        x, idx = L.rows(T, seed=T), random_routing(T, 2, 4, T)
        y, ys, off, perm = L.run(T, x, idx)
        ws = torch.full((moe.moe_workspace_bytes(L.C, T),), 0xFF, dtype=torch.uint8, device=DEV)
        todo.append((L, T, _bf16_dev(x), _dev(perm), _dev(off), y, ys, torch.empty_like(y), torch.empty_like(ys), ws))
    sync()
    streams = [torch.cuda.Stream() for _ in todo]
    for _ in range(5):
        for L, T, *_, z, zs, _ in todo:
            z.fill_(float("nan"))
            zs.fill_(float("nan"))
        sync()
        for s, (L, T, x, perm, off, _, _, z, zs, ws) in zip(streams, todo):
            moe.moe_expert_ffn(L.C, T, x, perm, off, L.W, z, zs, ws, stream=s)
        sync()
        for L, T, _, _, _, y, ys, z, zs, _ in todo:
            assert torch.equal(z[:2 * T], y[:2 * T]) and torch.equal(zs[:T], ys[:T])
