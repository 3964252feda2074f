"""Cases of the operators around and inside the MoE layer, for timing and comparison:

  norm         residual add + RMS norm, with an e4m3 copy (1x128 scales) where asked for
  norm_grad    its backward
  tokens       token rows sorted by expert (bf16 or fp32 rows, or e4m3 rows with their scales)
  tokens_grad  the backward of the weighted combine and of the sorting, as a training step calls them
  experts      the SwiGLU expert products on 4-bit weights with group scales (routed and shared)

`run` computes them in plain torch (32-bit arithmetic, rounded once) or, with `own` set, through
the library.  `exact` is the definition in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the norm in front of one decode step of the 32-token batch, e4m3 copy with power-of-two scales: latency
        {"name": "norm-decode-T32-fp8e8m0", "op": "norm", "T": 32, "H": 7168, "act": "bf16", "q": "fp8e8m0"},
        # the norm in front of the FP8 layer's prompt batch: bf16 rows for the gate, e4m3 rows for the experts
        {"name": "norm-T8192-fp8", "op": "norm", "T": 8192, "H": 7168, "act": "bf16", "q": "fp8"},
        # a training step of one 4096-token sequence
        {"name": "norm-grad-T4096-bf16", "op": "norm_grad", "T": 4096, "H": 7168, "act": "bf16"},
        # fp32 training of a small layer, an odd number of tokens
        {"name": "norm-grad-T777-f32", "op": "norm_grad", "T": 777, "H": 1024, "act": "f32"},
        # a small odd batch handed to experts outside the library
        {"name": "tokens-T509-bf16", "op": "tokens", "T": 509, "H": 2048, "E": 64, "K": 4, "act": "bf16", "q": ""},
        # FP8 dispatch of the prompt batch: codes and 1x128 scales
        {"name": "tokens-T8192-fp8", "op": "tokens", "T": 8192, "H": 7168, "E": 256, "K": 8, "act": "bf16", "q": "fp8"},
        # the two ends of the expert backward of a 4096-token training step
        {"name": "tokens-grad-T4096-bf16", "op": "tokens_grad", "T": 4096, "H": 7168, "E": 256, "K": 8, "act": "bf16"},
        # the same in fp32, small and odd
        {"name": "tokens-grad-T261-f32", "op": "tokens_grad", "T": 261, "H": 1024, "E": 64, "K": 8, "act": "f32"},
        # one new token of one user: eight routed experts and the shared one
        {"name": "experts-T1-g128", "op": "experts", "T": 1, "H": 7168, "E": 256, "K": 8, "I": 2048, "Is": 2048, "g": 128, "skew": 0.0},
        # the 32-token decode batch with skewed expert loads
        {"name": "experts-T32-g128", "op": "experts", "T": 32, "H": 7168, "E": 256, "K": 8, "I": 2048, "Is": 2048, "g": 128, "skew": 1.2},
        # a smaller layer, odd batch, fine groups
        {"name": "experts-T201-g32", "op": "experts", "T": 201, "H": 1024, "E": 32, "K": 4, "I": 256, "Is": 384, "g": 32, "skew": 0.5},
        # a large serving batch (many users, or a short prompt chunk): every expert has rows
        {"name": "experts-T1024-g128", "op": "experts", "T": 1024, "H": 7168, "E": 256, "K": 8, "I": 2048, "Is": 2048, "g": 128, "skew": 0.3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    while True:
        h = max(lo, _log(rng, lo, hi) // step * step)
        if h != 3072:
            return h


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "tokens", "tokens_grad", "experts", "experts"])
    if op == "experts":
        E = rng.choice([8, 16, 32, 64, 128, 256])
        c = {"op": op, "T": _log(rng, 1, 1024), "H": _width(rng, 256, 7168, 128), "E": E, "K": rng.randint(1, 8),
             "I": _width(rng, 128, 2048, 128), "Is": rng.choice([0, 128, 384, 1024, 2048]), "g": rng.choice([32, 128]),
             "skew": rng.choice([0.0, 0.5, 1.2])}
    else:
        c = {"op": op, "T": _log(rng, 1, 8192), "H": _width(rng, 128, 7168, 128), "act": rng.choice(["bf16", "bf16", "f32"])}
        if op.startswith("tokens"):
            c["E"], c["K"] = rng.choice([8, 16, 64, 256]), rng.randint(1, 8)
        if op in ("norm", "tokens"):
            c["q"] = rng.choice(["", "fp8", "fp8e8m0" if c["T"] <= 64 else "fp8"]) if c["act"] == "bf16" else ""
        if c["act"] == "f32":
            c["T"] = min(c["T"], 4096)
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed, device=DEV):
    return torch.Generator(device=device).manual_seed(1000003 * (seed % 100003) + 17)


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _choose(c, seed, device):
    """Routing [T, K]: distinct experts from noisy scores, expert loads falling with their rank."""
    g = _gen(seed + 7, device)
    s = -torch.log(-torch.log(torch.rand(c["T"], c["E"], generator=g, device=device).clamp_(1e-9, 1 - 1e-7)))
    rank = torch.randperm(c["E"], generator=g, device=device).float() + 1
    return torch.topk(s - c.get("skew", 0.0) * torch.log(rank), c["K"], dim=1).indices


def _sorted(idx, E):
    """The stable order by expert: offsets, perm, pos (int32)."""
    flat = idx.reshape(-1)
    perm = torch.argsort(flat, stable=True)
    pos = torch.empty_like(perm)
    pos[perm] = torch.arange(perm.numel(), device=perm.device)
    off = torch.zeros(E + 1, dtype=torch.int32, device=perm.device)
    off[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    return off, perm.int(), pos.int()


def _codes(g, experts, rows, cols, group):
    """4-bit codes (two a byte, the even column low) and bf16 scales of a weight matrix of about N(0, 1/cols)."""
    q = torch.randint(0, 256, (experts, rows, cols // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = (0.7 + 0.6 * torch.rand(experts, rows, cols // group, generator=g, device=DEV)) / (4.6 * math.sqrt(cols))
    return q, s.to(torch.bfloat16)


def _quant_rows(y, pow2):
    """e4m3 values and fp32 scales of y [T, H] fp32 in tiles of 128 columns."""
    t = y.reshape(y.shape[0], -1, 128)
    a = t.abs().amax(dim=2)
    if pow2:
        m, e = torch.frexp(a.double() / 448.0)
        e = torch.where(m == 0.5, e - 1, e).clamp(-126, 127)
        s = torch.ldexp(torch.ones_like(a), e)
    else:
        s = a / 448.0
    s = torch.where(a > 0, s, torch.ones_like(s))
    q = (t / s[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.reshape(y.shape), s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _prepare_own(s, case)
    return s


def _inputs(c, seed):
    g = _gen(seed)
    op, T, H = c["op"], c["T"], c["H"]
    s = {"c": c, "T": T, "H": H}
    act = DT[c.get("act", "bf16")]
    if op in ("norm", "norm_grad"):
        s["weight"] = 1.0 + 0.2 * torch.randn(H, generator=g, device=DEV)
        s["x"] = _randn(g, T, H, dtype=act)                  # the block's output, or its incoming gradient
        s["residual"] = _randn(g, T, H, dtype=act, std=2.0)  # the residual stream
        if op == "norm_grad":
            s["dsum"] = _randn(g, T, H, dtype=act)           # the gradient that the stream carries past the layer
    else:
        K, E = c["K"], c["E"]
        s["K"], s["E"] = K, E
        s["off"], s["perm"], s["pos"] = _sorted(_choose(c, seed, DEV), E)
        if op == "tokens":
            x = _randn(g, T, H, dtype=act)
            if c["q"]:
                q, s["xs"] = _quant_rows(x.float(), c["q"] == "fp8e8m0")
                s["xq"] = q.view(torch.uint8)
            else:
                s["x"] = x
        elif op == "tokens_grad":
            s["dout"] = _randn(g, T, H, dtype=act)
            s["y"] = _randn(g, T * K, H, dtype=act, std=0.5)
            s["drows"] = _randn(g, T * K, H, dtype=act, std=0.5)
            s["dx_add"] = _randn(g, T, H, dtype=act)         # the shared expert's input gradient
            w = torch.rand(T, K, generator=g, device=DEV) + 0.1
            s["w"] = 2.5 * w / w.sum(1, keepdim=True)
        else:
            s["x"] = _randn(g, T, H, dtype=act)
            I, Is = c["I"], c["Is"]
            s["w13"], s["w2"] = _codes(g, E, 2 * I, H, c["g"]), _codes(g, E, H, I, c["g"])
            if Is:
                s["ws13"], s["ws2"] = _codes(g, 1, 2 * Is, H, c["g"]), _codes(g, 1, H, Is, c["g"])
    return s


def _prepare_own(s, c):
    """The library's config, and the output buffers, workspace and packed weights that a program keeps."""
    import sparse_mixture_experts_30_amd as moe
    op, T, H = c["op"], c["T"], c["H"]
    act = c.get("act", "bf16")
    dt = DT[act]

    def new(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device=DEV)

    wd = c.get("q") or act
    if op == "experts":
        wd = "int4g%d" % c["g"]
    s["cfg"] = C = moe.config(H, c.get("E", 2), 1, 1, c.get("K", 1), c.get("I", 128), c.get("Is", 0), 1.0, act, wd)
    if op == "norm":
        s["sum"], s["out"] = new(T, H), new(T, H)
        if c["q"]:
            s["yq"], s["ys"] = new(T, H, dtype=torch.uint8), new(T, H // 128, dtype=torch.float32)
    elif op == "norm_grad":
        s["dx"], s["dweight"] = new(T, H), new(H, dtype=torch.float32)
        s["ws"] = new(moe.moe_add_rmsnorm_backward_workspace_bytes(C, T), dtype=torch.uint8)
    elif op == "tokens":
        N = T * c["K"]
        if c["q"]:
            s["rows_q"], s["rows_s"] = new(N, H, dtype=torch.uint8), new(N, H // 128, dtype=torch.float32)
        else:
            s["rows"] = new(N, H)
    elif op == "tokens_grad":
        s["dy"], s["dx"], s["dw"] = new(T * c["K"], H), new(T, H), new(T, c["K"], dtype=torch.float32)
    else:
        packed = {}
        for name, which in (("w13", moe.MOE_W13), ("w2", moe.MOE_W2), ("ws13", moe.MOE_WS13), ("ws2", moe.MOE_WS2)):
            if name in s:
                buf = new(moe.moe_packed_bytes(C, which), dtype=torch.uint8)
                moe.moe_pack_quantized(C, which, s[name][0], s[name][1], buf)
                packed[name] = buf
        for name in packed:
            s[name] = packed[name]
        s["W"] = moe.weights(packed=True, **packed)
        s["out"], s["out_shared"] = new(T * c["K"], H), new(T, H) if c["Is"] else None
        s["ws"] = new(moe.moe_workspace_bytes(C, T), dtype=torch.uint8)


# ---------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)[state["c"]["op"]](state)


def _own_norm(s):
    import sparse_mixture_experts_30_amd as moe
    moe.moe_add_rmsnorm(s["cfg"], s["T"], s["x"], s["residual"], s["weight"], EPS, sum=s["sum"], y=s["out"],
                        yq=s.get("yq"), ys=s.get("ys"))
    out = {"sum": s["sum"], "y": s["out"]}
    if "yq" in s:
        out["yq"], out["ys"] = s["yq"].view(torch.float8_e4m3fn), s["ys"]
    return out


def _own_norm_grad(s):
    import sparse_mixture_experts_30_amd as moe
    moe.moe_add_rmsnorm_backward(s["cfg"], s["T"], s["residual"], s["weight"], EPS, s["x"], s["dx"], s["dweight"],
                                 s["ws"], dsum=s["dsum"])
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _own_tokens(s):
    import sparse_mixture_experts_30_amd as moe
    if "xq" in s:
        moe.moe_dispatch_quantized(s["cfg"], s["T"], s["xq"], s["xs"], s["pos"], s["rows_q"], s["rows_s"])
        return {"rows_q": s["rows_q"].view(torch.float8_e4m3fn), "rows_s": s["rows_s"]}
    moe.moe_dispatch(s["cfg"], s["T"], s["x"], s["pos"], s["rows"])
    return {"rows": s["rows"]}


def _own_tokens_grad(s):
    import sparse_mixture_experts_30_amd as moe
    moe.moe_combine_backward(s["cfg"], s["T"], s["dout"], s["y"], s["pos"], s["w"], s["dy"], s["dw"])
    moe.moe_dispatch_backward(s["cfg"], s["T"], s["drows"], s["pos"], s["dx"], dx_add=s["dx_add"])
    return {"dy": s["dy"], "dw": s["dw"], "dx": s["dx"]}


def _own_experts(s):
    import sparse_mixture_experts_30_amd as moe
    moe.moe_expert_ffn(s["cfg"], s["T"], s["x"], s["perm"], s["off"], s["W"], s["out"], s["out_shared"], s["ws"])
    return {"y": s["out"], "y_shared": s["out_shared"]}


def _plain_norm(s):
    x, c = s["x"], s["c"]
    r = (x.float() + s["residual"].float()).to(x.dtype)  # the stream as it is stored is what the norm reads
    f = r.float()
    y = f * torch.rsqrt((f * f).mean(dim=1, keepdim=True) + EPS) * s["weight"]
    out = {"sum": r, "y": y.to(x.dtype)}
    if c["q"]:
        out["yq"], out["ys"] = _quant_rows(y, c["q"] == "fp8e8m0")
    return out


def _plain_norm_grad(s):
    r, dy, w = s["residual"].float(), s["x"].float(), s["weight"]
    rstd = torch.rsqrt((r * r).mean(dim=1, keepdim=True) + EPS)
    n = r * rstd
    gw = dy * w
    dx = rstd * (gw - n * (gw * n).mean(dim=1, keepdim=True)) + s["dsum"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * n).sum(dim=0)}


def _plain_tokens(s):
    tok = (s["perm"] // s["K"]).long()
    if "xq" in s:
        return {"rows_q": s["xq"][tok].view(torch.float8_e4m3fn), "rows_s": s["xs"][tok]}
    return {"rows": s["x"][tok]}


def _plain_tokens_grad(s):
    T, K, H = s["T"], s["K"], s["H"]
    pos = s["pos"].long()
    dout = s["dout"].float()
    dy = torch.empty_like(s["y"])
    dy[pos] = (s["w"][:, :, None] * dout[:, None, :]).to(dy.dtype).reshape(T * K, H)
    dw = (dout[:, None, :] * s["y"][pos].reshape(T, K, H).float()).sum(dim=2)
    dx = s["dx_add"].float() + s["drows"][pos].reshape(T, K, H).float().sum(dim=1)
    return {"dy": dy, "dw": dw, "dx": dx.to(s["dx_add"].dtype)}


def _dequant(q, sc, group):
    """[experts, rows, cols] fp32 of 4-bit codes and group scales."""
    v = torch.stack((q & 15, q >> 4), dim=-1).reshape(*q.shape[:2], -1).float() - 8.0
    return (v.reshape(*sc.shape, group) * sc.float()[..., None]).reshape(v.shape)


def _swiglu(w13, w2, xt, group):
    """[experts, H, n] = W2 (silu(Wg x) * (Wu x)) for xt [experts, H, n] fp32."""
    gu = torch.bmm(_dequant(*w13, group), xt)
    I = gu.shape[1] // 2
    h = gu[:, :I] / (1.0 + torch.exp(-gu[:, :I])) * gu[:, I:]
    return torch.bmm(_dequant(*w2, group), h.contiguous())


def _plain_experts(s):
    """Every expert that has rows, on its rows, padded to the longest expert's."""
    T, K, group = s["T"], s["K"], s["c"]["g"]
    N = T * K
    counts = (s["off"][1:] - s["off"][:-1]).long()
    active = counts.nonzero()[:, 0]
    n = counts[active]
    e = torch.repeat_interleave(torch.arange(active.numel(), device=DEV), n, output_size=N)
    at = torch.arange(N, device=DEV) - s["off"][active].long()[e]
    xt = torch.zeros(active.numel(), s["H"], int(n.max()), device=DEV)
    xt[e, :, at] = s["x"].float()[(s["perm"] // K).long()]
    w13, w2 = (tuple(t[active] for t in s[name]) for name in ("w13", "w2"))
    y = _swiglu(w13, w2, xt, group)[e, :, at]
    ys = None
    if s["c"]["Is"]:
        ys = _swiglu(s["ws13"], s["ws2"], s["x"].float().t().contiguous()[None], group)[0].t().contiguous().to(s["x"].dtype)
    return {"y": y.to(s["x"].dtype), "y_shared": ys}


_own = {"norm": _own_norm, "norm_grad": _own_norm_grad, "tokens": _own_tokens, "tokens_grad": _own_tokens_grad,
        "experts": _own_experts}
_plain = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "tokens": _plain_tokens,
          "tokens_grad": _plain_tokens_grad, "experts": _plain_experts}


# ---------------------------------------------------------------- what a pass has to move and compute

def work(case):
    c = case
    op, T, H = c["op"], c["T"], c["H"]
    a = 2 if c.get("act", "bf16") == "bf16" else 4
    if op == "norm":
        q = T * H + T * H // 128 * 4 if c["q"] else 0
        return {"bytes": 4 * T * H * a + 4 * H + q, "flops": 6 * T * H}
    if op == "norm_grad":
        return {"bytes": 4 * T * H * a + 8 * H, "flops": 12 * T * H}
    N = T * c["K"]
    if op == "tokens":
        row = H + H // 128 * 4 if c["q"] else H * a
        return {"bytes": (T + N) * row + 4 * N, "flops": 0}
    if op == "tokens_grad":
        return {"bytes": (3 * T + 3 * N) * H * a + 16 * N, "flops": 4 * N * H}
    I, Is = c["I"], c["Is"]
    active = int(torch.unique(_choose(c, 0, "cpu")).numel())  # experts that a batch of this kind reaches
    weights = 3 * H * (active * I + Is) * (0.5 + 2.0 / c["g"])
    return {"bytes": weights + T * H * 2 + (N + (T if Is else 0)) * H * 2 + 4 * N,
            "flops": 6 * H * (N * I + T * Is)}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    c, T, H = case, case["T"], case["H"]
    d = lambda t: t.to(torch.float64)  # noqa: E731
    if c["op"] == "norm":
        r = d(s["x"]) + d(s["residual"])
        y = r / torch.sqrt(torch.sum(r ** 2, 1, keepdim=True) / H + EPS) * d(s["weight"])
        out = {"sum": r, "y": y}
        if c["q"]:
            out["yq"] = out["ys"] = None  # rounded to eight bits: the plain form says which values
        return out
    if c["op"] == "norm_grad":
        r, g, w = d(s["residual"]), d(s["x"]), d(s["weight"])
        m = torch.sum(r ** 2, 1, keepdim=True) / H + EPS
        dot = torch.sum(g * w * r, 1, keepdim=True) / H
        return {"dx": g * w * m ** -0.5 - r * dot * m ** -1.5 + d(s["dsum"]), "dweight": torch.sum(g * r * m ** -0.5, 0)}
    if c["op"] == "tokens":
        return None  # copies of rows
    K = c["K"]
    if c["op"] == "tokens_grad":
        if T * K * H > 300_000_000:
            return None
        dout, pos = d(s["dout"]), s["pos"].long().reshape(T, K)
        dy = torch.empty(T * K, H, dtype=torch.float64, device=DEV)
        dw = torch.empty(T, K, dtype=torch.float64, device=DEV)
        dx = d(s["dx_add"])
        for k in range(K):
            dy[pos[:, k]] = d(s["w"][:, k:k + 1]) * dout
            dw[:, k] = torch.sum(dout * d(s["y"][pos[:, k]]), 1)
            dx = dx + d(s["drows"][pos[:, k]])
        return {"dy": dy, "dw": dw, "dx": dx}

    def matrix(q, sc):
        m = torch.empty(q.shape[0], q.shape[1] * 2, dtype=torch.float64, device=DEV)
        m[:, 0::2] = d(q % 16) - 8
        m[:, 1::2] = d(q // 16) - 8
        return m * d(sc).repeat_interleave(c["g"], dim=1)

    def ffn(w13, w2, e, x):
        gu = x @ matrix(w13[0][e], w13[1][e]).T
        n = gu.shape[1] // 2
        return (gu[:, n:] * gu[:, :n] * torch.sigmoid(gu[:, :n])) @ matrix(w2[0][e], w2[1][e]).T

    x, off = d(s["x"]), s["off"].tolist()
    tok = s["perm"].long() // K
    y = torch.empty(T * K, H, dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        if off[e + 1] > off[e]:
            y[off[e]:off[e + 1]] = ffn(s["w13"], s["w2"], e, x[tok[off[e]:off[e + 1]]])
    return {"y": y, "y_shared": ffn(s["ws13"], s["ws2"], 0, x) if c["Is"] else None}
