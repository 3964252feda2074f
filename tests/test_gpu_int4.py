"""4-bit expert weights on the GPU against 64-bit products of the values that
the codes and scales stand for.

Tolerance of a row (relative L2).  h and y are rounded to bf16 once each, 2^-8
of a value at most and about 1.7e-3 in the root mean square; the two add to
2.4e-3, fp32 sums are far below, and a factor of two is left for short rows:
5e-3.  One weight column left out or taken twice moves a row by 1 / sqrt(7168)
= 1.2e-2 or more."""
import numpy as np
import pytest
import torch

import synth
import sparse_mixture_experts_30_amd as moe
from oracle import block
from synth import device as sd

from gpu_util import DEV, host, log, random_routing, run_permute, sync, worst_row_rel

pytestmark = pytest.mark.gpu

TOL = 5e-3
GROUP = {"int4g128": 128, "int4g32": 32}


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _bf16_dev(a):
    return _dev(np.asarray(a, np.float32)).to(torch.bfloat16)


def _matrix(rng, experts, rows, cols, group):
    """Codes over the whole range (all of 0..15), uneven scales, one group of scale 0."""
    q = rng.integers(0, 16, (experts, rows, cols), dtype=np.uint8)
    s = block.bf16((0.3 + rng.random((experts, rows, cols // group))).astype(np.float32) / (5 * np.sqrt(cols)))
    s[0, 0, 0] = 0.0
    return q, s


def _pack(C, which, q, s):
    buf = torch.full((moe.moe_packed_bytes(C, which),), 0xEE, dtype=torch.uint8, device=DEV)
    moe.moe_pack_quantized(C, which, _dev(block.pack_nibbles(q)), _bf16_dev(s), buf)
    return buf


class Layer:
    def __init__(self, wd, H, E, K, I, Is, seed=0):
        g, rng = GROUP[wd], np.random.default_rng(seed)
        self.C = moe.config(H, E, 1, 1, K, I, Is, 1.0, "bf16", wd)
        self.H, self.E, self.K, self.I, self.Is = H, E, K, I, Is
        m = {"w13": _matrix(rng, E, 2 * I, H, g), "w2": _matrix(rng, E, H, I, g)}
        if Is:
            m["ws13"], m["ws2"] = _matrix(rng, 1, 2 * Is, H, g), _matrix(rng, 1, H, Is, g)
        self.w = {k: block.dequantize_int4(*v, g) for k, v in m.items()}
        which = {"w13": moe.MOE_W13, "w2": moe.MOE_W2, "ws13": moe.MOE_WS13, "ws2": moe.MOE_WS2}
        self.packed = {k: _pack(self.C, which[k], *v) for k, v in m.items()}

    def check(self, T, idx, seed=1):
        N = T * self.K
        x = block.bf16(np.random.default_rng(seed).standard_normal((T, self.H)).astype(np.float32))
        c = synth.C1.replace(name="int4", T=T, E=self.E, G=1, TG=1, K=self.K)
        _, off, perm, _, _ = run_permute(c, idx)
        y = torch.full((N, self.H), float("nan"), dtype=torch.bfloat16, device=DEV)
        ys = torch.full((T, self.H), float("nan"), dtype=torch.bfloat16, device=DEV) if self.Is else None
        ws = torch.full((moe.moe_workspace_bytes(self.C, T),), 0xFF, dtype=torch.uint8, device=DEV)
        W = moe.weights(packed=True, **self.packed)
        moe.moe_expert_ffn(self.C, T, _bf16_dev(x), _dev(perm), _dev(off), W, y, ys, ws)
        sync()
        ref = np.zeros((N, self.H))
        for e in range(self.E):
            r = slice(off[e], off[e + 1])
            if off[e + 1] > off[e]:
                ref[r] = block.swiglu(x[perm[r] // self.K], self.w["w13"][e], self.w["w2"][e])
        bad = worst_row_rel(host(y), ref)
        log(f"int4 T={T} routed worst row {bad:.2e}")
        assert bad <= TOL
        if self.Is:
            assert worst_row_rel(host(ys), block.swiglu(x, self.w["ws13"][0], self.w["ws2"][0])) <= TOL
        y2 = torch.empty_like(y)
        ys2 = None if ys is None else torch.empty_like(ys)
        moe.moe_expert_ffn(self.C, T, _bf16_dev(x), _dev(perm), _dev(off), W, y2, ys2, ws)
        sync()
        assert torch.equal(y, y2) and (ys is None or torch.equal(ys, ys2))


# Tokens around the 16-row blocks of the few-row kernel; K steps that do not divide by four.
@pytest.mark.parametrize("wd", ["int4g128", "int4g32"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 150])
def test_rows(wd, T):
    L = Layer(wd, H=640, E=8, K=2, I=256, Is=384)
    L.check(T, random_routing(T, 2, 8, seed=T, skew=True))     # expert 0 has all T rows


# More than 8 rows per expert on average and enough output tiles to fill the GPU: the kernels with
# tiles of 32 (up to 28 rows on average) and of 64 rows, with an odd number of k steps and of output tiles.
# Expert 0 has all T rows, so tiles of every height up to the full one occur, alone and side by side.
@pytest.mark.parametrize("wd", ["int4g128", "int4g32"])
@pytest.mark.parametrize("T", [150, 400, 700])
def test_tall_tiles(wd, T):
    L = Layer(wd, H=384, E=32, K=2, I=2048, Is=128)
    L.check(T, random_routing(T, 2, 32, seed=T, skew=True))


def test_tall_tiles_with_few_workgroups():
    """1024 rows an expert: the tall-tile kernel although its grid is small."""
    L = Layer("int4g128", H=256, E=4, K=4, I=256, Is=128)
    L.check(1024, random_routing(1024, 4, 4, seed=11))


@pytest.mark.parametrize("wd", ["int4g128", "int4g32"])
@pytest.mark.parametrize("H,I,Is", [(128, 128, 0), (128, 128, 128), (256, 384, 128), (1024, 128, 640), (384, 512, 0)])
def test_widths(wd, H, I, Is):
    L = Layer(wd, H, E=4, K=1, I=I, Is=Is)
    L.check(21, random_routing(21, 1, 4, seed=H))


def test_large_widths():
    Layer("int4g128", H=7168, E=2, K=1, I=2048, Is=2048).check(5, random_routing(5, 1, 2, seed=3))


@pytest.mark.parametrize("wd", ["int4g128", "int4g32"])
def test_few_rows_on_average_many_in_one_expert(wd):
    """The few-row kernel with an expert cut into several 16-row tiles."""
    L = Layer(wd, 384, E=32, K=1, I=256, Is=128)
    idx = random_routing(100, 1, 32, seed=8)
    idx[20:] = 5
    L.check(100, idx)


def test_more_rows_than_tokens():
    """A caller's routing may name one expert twice for a token: more rows than the tile of a small batch."""
    L = Layer("int4g128", 256, E=4, K=4, I=128, Is=0)
    L.check(16, np.zeros((16, 4), np.int32))
    L.check(1, np.array([[2, 2, 2, 2]], np.int32))


def test_row_isolation():
    """Non-finite values of one token's row stay in that token's outputs."""
    L = Layer("int4g32", 256, E=4, K=1, I=128, Is=128)
    T = 20
    idx = random_routing(T, 1, 4, seed=9)
    c = synth.C1.replace(name="int4", T=T, E=4, G=1, TG=1, K=1)
    _, off, perm, pos, _ = run_permute(c, idx)
    x = torch.randn(T, 256, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    W = moe.weights(packed=True, **L.packed)
    outs = []
    for bad in (False, True):
        xx = x.clone()
        if bad:
            xx[3, 9], xx[7, 200] = float("inf"), float("nan")
        y, ys = torch.empty_like(x), torch.empty_like(x)
        ws = torch.empty(moe.moe_workspace_bytes(L.C, T), dtype=torch.uint8, device=DEV)
        moe.moe_expert_ffn(L.C, T, xx, _dev(perm), _dev(off), W, y, ys, ws)
        sync()
        outs.append((host(y)[pos], host(ys)))
    keep = [t for t in range(T) if t not in (3, 7)]
    for a, b in zip(*outs):
        assert np.array_equal(a[keep], b[keep]) and np.all(np.isnan(b[[3, 7]]).any(axis=1))


@pytest.mark.parametrize("wd", ["int4g128", "int4g32"])
@pytest.mark.parametrize("which", ["w13", "w2", "ws13", "ws2"])
def test_quantize_weight(wd, which):
    H, E, I, Is, g = 256, 3, 384, 128, GROUP[wd]
    C = moe.config(H, E, 1, 1, 1, I, Is, 1.0, "bf16", wd)
    shape = {"w13": (E, 2 * I, H), "w2": (E, H, I), "ws13": (1, 2 * Is, H), "ws2": (1, H, Is)}[which]
    w = block.bf16(np.random.default_rng(4).standard_normal(shape).astype(np.float32) * 0.02)
    w[0, 0, :g] = 0.0
    w[0, 1, 0], w[0, 2, g - 1] = 100.0, -3e38
    codes = torch.full((shape[0], shape[1], shape[2] // 2), 0x77, dtype=torch.uint8, device=DEV)
    scales = torch.full((shape[0], shape[1], shape[2] // g), 5.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_quantize_weight(C, getattr(moe, "MOE_" + which.upper()), _bf16_dev(w), codes, scales)
    sync()
    q, s = block.quantize_int4(w.reshape(-1, shape[2]), g)
    assert np.array_equal(host(scales).reshape(s.shape), s)
    assert np.array_equal(host(codes).reshape(-1, shape[2] // 2), block.pack_nibbles(q))


@pytest.mark.parametrize("wd", ["int4g128", "int4g32"])
@pytest.mark.parametrize("T", [3, 24, 100])
def test_forward_is_its_steps(wd, T):
    """moe_forward, its no-allocation and two-stream forms, and a replayed graph against the steps one by one."""
    cfg = synth.C3.replace(name="int4-forward", T=T, H=512, E=16, G=4, TG=2, K=4, I=256, Is=128, rho=2.5, wdtype=wd)
    src = synth.gen_inputs(cfg.replace(wdtype="bf16"))
    dev = sd.to_device(src)
    C, g = sd.moe_config(cfg), GROUP[wd]
    packed = {}
    for k, which in (("w13", moe.MOE_W13), ("w2", moe.MOE_W2), ("ws13", moe.MOE_WS13), ("ws2", moe.MOE_WS2)):
        m = dev[k]
        codes = torch.empty((*m.shape[:-1], m.shape[-1] // 2), dtype=torch.uint8, device=DEV)
        scales = torch.empty((*m.shape[:-1], m.shape[-1] // g), dtype=torch.bfloat16, device=DEV)
        moe.moe_quantize_weight(C, which, m, codes, scales)
        packed[k] = torch.empty(moe.moe_packed_bytes(C, which), dtype=torch.uint8, device=DEV)
        moe.moe_pack_quantized(C, which, codes, scales, packed[k])
    W = moe.weights(gate_w=dev["gate_w"], bias=dev["bias"], packed=True, **packed)
    N = T * cfg.K
    f32, i32 = dict(dtype=torch.float32, device=DEV), dict(dtype=torch.int32, device=DEV)
    idx, w, perm = torch.empty((T, cfg.K), **i32), torch.empty((T, cfg.K), **f32), torch.empty(N, **i32)
    ws, out = sd.workspace(cfg, T), torch.empty_like(dev["x"])
    moe.moe_forward(C, T, dev["x"], W, out, ws, topk_idx=idx, topk_w=w, perm=perm)
    assert moe.moe_get_device_error(ws) == moe.MOE_OK
    counts, off, pos = torch.empty(cfg.E, **i32), torch.empty(cfg.E + 1, **i32), torch.empty(N, **i32)
    y, ys, want = torch.empty((N, cfg.H), dtype=torch.bfloat16, device=DEV), torch.empty_like(out), torch.empty_like(out)
    moe.moe_permute(C, T, idx, counts, off, perm, pos, ws)
    moe.moe_expert_ffn(C, T, dev["x"], perm, off, W, y, ys, ws)
    moe.moe_combine(C, T, y, ys, pos, w, want)
    sync()
    assert torch.equal(out, want)
    other = torch.empty_like(out)
    moe.moe_forward_noalloc(C, T, dev["x"], W, other)
    sync()
    assert torch.equal(other, want)
    s = torch.cuda.Stream()
    other.zero_()
    moe.moe_forward_overlap(C, T, dev["x"], W, other, ws, s)
    sync()
    assert torch.equal(other, want)
    # the whole serving step in a graph, replayed with eager work between
    gamma = torch.ones(cfg.H, device=DEV)
    stream, normed = torch.empty_like(out), torch.empty_like(out)

    def step():
        moe.moe_add_rmsnorm(C, T, dev["x"], out, gamma, 1e-6, sum=stream, y=normed)
        moe.moe_forward(C, T, normed, W, other, ws)

    step()
    sync()
    eager = other.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        other.zero_()
        stream.zero_()
        normed.zero_()
        sync()
        graph.replay()
        sync()
        assert torch.equal(other, eager)


@pytest.mark.parametrize("wd", ["fp8", "fp8e8m0"])
def test_experts_on_e4m3_rows(wd):
    """The e4m3 rows of the quantiser through moe_expert_ffn_quantized: the bits of moe_expert_ffn."""
    cfg = synth.C5.replace(name="q-rows", T=40, H=256, E=8, G=2, TG=2, K=2, I=128, Is=128, rho=1.0, wdtype=wd)
    dev = sd.packed_copy(sd.to_device(synth.gen_inputs(cfg)))
    C, T, W = sd.moe_config(cfg), cfg.T, sd.weights_struct(dev)
    c = synth.C1.replace(name="q-rows", T=T, E=8, G=1, TG=1, K=2)
    _, off, perm, _, _ = run_permute(c, random_routing(T, 2, 8, seed=5))
    new = lambda n: torch.full((n, cfg.H), float("nan"), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    a, b = (new(2 * T), new(T)), (new(2 * T), new(T))
    ws = sd.workspace(cfg, T)
    moe.moe_expert_ffn(C, T, dev["x"], _dev(perm), _dev(off), W, *a, ws)
    xq = torch.empty((T, cfg.H), dtype=torch.uint8, device=DEV)
    xs = torch.empty((T, cfg.H // 128), device=DEV)
    moe.moe_quantize_act(C, T, dev["x"], xq, xs)
    ws.fill_(0xFF)
    moe.moe_expert_ffn_quantized(C, T, xq, xs, _dev(perm), _dev(off), W, *b, ws)
    sync()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# Routed experts and the shared one in one launch and each in its own (moe_forward_overlap): the rows of the whole
# layer name the kernel, so that the sums have one order.  More than 8 rows an expert and enough tiles of the whole
# layer for 32 (T = 600) and 64 rows (T = 1000), where the shared expert's tiles alone would be too few.
@pytest.mark.parametrize("wd", ["int4g128", "int4g32"])
@pytest.mark.parametrize("T", [600, 1000])
def test_overlap_has_the_bits_of_forward(wd, T):
    cfg = synth.C3.replace(name="int4-overlap", T=T, H=512, E=32, G=4, TG=2, K=1, I=2048, Is=2048, rho=2.5, wdtype=wd)
    C, g, rng = sd.moe_config(cfg), GROUP[wd], np.random.default_rng(T)
    which = {"w13": (moe.MOE_W13, cfg.E, 2 * cfg.I, cfg.H), "w2": (moe.MOE_W2, cfg.E, cfg.H, cfg.I),
             "ws13": (moe.MOE_WS13, 1, 2 * cfg.Is, cfg.H), "ws2": (moe.MOE_WS2, 1, cfg.H, cfg.Is)}
    packed = {k: _pack(C, i, *_matrix(rng, e, n, m, g)) for k, (i, e, n, m) in which.items()}
    gate = torch.from_numpy(rng.standard_normal((cfg.E, cfg.H)).astype(np.float32) / np.float32(np.sqrt(cfg.H))).to(DEV)
    bias = torch.zeros(cfg.E, device=DEV)
    W = moe.weights(gate_w=gate, bias=bias, packed=True, **packed)
    x = _bf16_dev(rng.standard_normal((T, cfg.H)))
    out, other, ws, s = torch.empty_like(x), torch.empty_like(x), sd.workspace(cfg, T), torch.cuda.Stream()
    moe.moe_forward(C, T, x, W, out, ws)
    sync()
    moe.moe_forward_overlap(C, T, x, W, other, ws, s)
    sync()
    assert torch.equal(out, other)


@pytest.mark.parametrize("wd", ["int4g128", "int4g32"])
def test_prompt_rows(wd):
    """A prompt of 2048 tokens at full width, all of them on one expert too; the first and last rows of every
    expert and some between against 64 bits."""
    T, H, E, K, I, Is, g = 2048, 7168, 3, 2, 2048, 2048, GROUP[wd]
    C, rng = moe.config(H, E, 1, 1, K, I, Is, 1.0, "bf16", wd), np.random.default_rng(12)
    m = {"w13": _matrix(rng, E, 2 * I, H, g), "w2": _matrix(rng, E, H, I, g),
         "ws13": _matrix(rng, 1, 2 * Is, H, g), "ws2": _matrix(rng, 1, H, Is, g)}
    which = {"w13": moe.MOE_W13, "w2": moe.MOE_W2, "ws13": moe.MOE_WS13, "ws2": moe.MOE_WS2}
    W_keep = {k: _pack(C, which[k], *v) for k, v in m.items()}
    x = block.bf16(rng.standard_normal((T, H)).astype(np.float32))
    c = synth.C1.replace(name="int4", T=T, E=E, G=1, TG=1, K=K)
    _, off, perm, _, _ = run_permute(c, random_routing(T, K, E, seed=13, skew=True))   # expert 0 has every token
    y = torch.full((T * K, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    ys = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.full((moe.moe_workspace_bytes(C, T),), 0xFF, dtype=torch.uint8, device=DEV)
    moe.moe_expert_ffn(C, T, _bf16_dev(x), _dev(perm), _dev(off), moe.weights(packed=True, **W_keep), y, ys, ws)
    sync()
    y, ys = host(y), host(ys)
    assert np.all(np.isfinite(y)) and np.all(np.isfinite(ys))
    for e in range(E + 1):
        rows = np.arange(off[e], off[e + 1]) if e < E else np.arange(T)
        rows = np.unique(np.concatenate([rows[:2], rows[rng.integers(0, len(rows), 8)], rows[-2:]]))
        k13, k2, i = ("w13", "w2", e) if e < E else ("ws13", "ws2", 0)
        w13, w2 = (block.dequantize_int4(m[k][0][i], m[k][1][i], g) for k in (k13, k2))
        got, tok = (y[rows], perm[rows] // K) if e < E else (ys[rows], rows)
        bad = worst_row_rel(got, block.swiglu(x[tok], w13, w2))
        log(f"int4 prompt {k13} {e} worst row {bad:.2e}")
        assert bad <= TOL
