"""The operators around the FP8 linears of a decoder layer, as measured work.

Four operators: residual addition + RMSNorm + FP8 output (``norm``), the scaled GEMM with
bias, activation and residual in its epilogue (``gemm``), the append of new K/V tokens to
a paged FP8 cache with one scale per page and KV head (``append``), and causal attention
over that cache (``attend``).  ``run`` computes each in plain torch operations, or, where
``own`` is true, through the package's entry points."""
import math
import random

import torch

own = False

F_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
DTYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of a served sequence entering a layer: latency
        dict(name="norm-1x8192", op="norm", rows=1, cols=8192, mode="row", fmt="e4m3", residual=True),
        # an odd batch of tokens in front of an MXFP8 linear, first layer (no residual yet)
        dict(name="norm-mx-odd", op="norm", rows=1021, cols=5152, mode="mx", fmt="e4m3", residual=False),
        # a long prompt in front of a block-scaled linear
        dict(name="norm-block-16k", op="norm", rows=16384, cols=8192, mode="block", fmt="e4m3", residual=True),
        # the down projection of a 16-token decode batch, added to the residual stream
        dict(name="gemm-decode-down", op="gemm", M=16, N=8192, K=28672, mode="row", fmt="e4m3", act="none",
             bias=False, residual=True, out="bf16"),
        # ragged sizes, every option, MXFP8 operands
        dict(name="gemm-mx-odd", op="gemm", M=333, N=2050, K=1056, mode="mx", fmt="e4m3", act="gelu", bias=True,
             residual=True, out="bf16"),
        # the up projection of a 4096-token prompt with its activation, FP8 output for the next linear
        dict(name="gemm-prefill-up", op="gemm", M=4096, N=28672, K=8192, mode="row", fmt="e4m3", act="silu", bias=True,
             residual=False, out="fp8"),
        # one decode step of 64 sequences: one new token each
        dict(name="append-decode", op="append", batch=64, max_q=1, max_kv=4096, spread=0.5, kv_heads=8, dim=128,
             page=64, fmt="e4m3", lens=1),
        # prompts of several lengths that end inside pages
        dict(name="append-prompts", op="append", batch=7, max_q=4096, max_kv=8000, spread=0.9, kv_heads=8, dim=128,
             page=32, fmt="e5m2", lens=2),
        # one short sequence, one KV head (a rank's share): latency
        dict(name="attend-short", op="attend", batch=1, max_q=1, max_kv=333, spread=0.0, heads=8, kv_heads=1, dim=128,
             page=16, fmt="e4m3", lens=3),
        # a full decode batch, sequences of many lengths
        dict(name="attend-decode", op="attend", batch=64, max_q=1, max_kv=8192, spread=0.6, heads=64, kv_heads=8,
             dim=128, page=64, fmt="e4m3", lens=4),
        # two long contexts: rows are few and the cache is long
        dict(name="attend-long", op="attend", batch=2, max_q=1, max_kv=100001, spread=0.3, heads=32, kv_heads=4,
             dim=128, page=128, fmt="e5m2", lens=5),
        # prompt chunks over what the cache already holds
        dict(name="attend-prompts", op="attend", batch=3, max_q=2048, max_kv=6001, spread=0.5, heads=32, kv_heads=8,
             dim=128, page=64, fmt="e4m3", lens=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gemm", "append", "attend"])
    if op == "norm":
        cols = 32 * _log(rng, 4, 512)
        rows = min(_log(rng, 1, 16384), 16384 * 8192 // cols)
        # E4M3, as the activations of a forward pass are held
        return dict(op=op, rows=rows, cols=cols, mode=rng.choice(["row", "block", "mx"]), fmt="e4m3",
                    residual=rng.random() < 0.7)
    if op == "gemm":
        M, N, K = _log(rng, 1, 4096), _log(rng, 64, 28672), 32 * _log(rng, 8, 896)
        while M * N * K > 4096 * 28672 * 8192:
            M, N = max(1, M // 2), max(64, N // 2)
        out = rng.choice(["bf16", "bf16", "fp8"])
        mode = rng.choice(["row", "block", "mx"])
        return dict(op=op, M=M, N=N, K=K, mode=mode, fmt="e4m3", act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                    bias=rng.random() < 0.5, residual=rng.random() < 0.6, out=out)
    dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    kv_heads, fmt = rng.choice([1, 2, 4, 8]), rng.choice(["e4m3", "e5m2"])
    lens = rng.randrange(1 << 20)
    if op == "append":
        max_q = rng.choice([1, 1, _log(rng, 2, 4096)])
        batch = _log(rng, 1, 256 if max_q == 1 else 8)
        max_kv = max(max_q, _log(rng, 16, 8192))
        return dict(op=op, batch=batch, max_q=max_q, max_kv=max_kv, spread=rng.uniform(0.0, 0.9), kv_heads=kv_heads,
                    dim=dim, page=page, fmt=fmt, lens=lens)
    group = rng.choice([1, 2, 4, 7, 8])
    max_q = rng.choice([1, 1, rng.randrange(2, 9), _log(rng, 9, 2048)])
    batch = _log(rng, 1, 64 if max_q < 9 else 4)
    max_kv = max(max_q, _log(rng, 1, 65536 if max_q < 9 else 6144))
    # the plain form pads the batch: bounded by what it holds at once
    while batch > 1 and (batch * max_kv * kv_heads * dim > 1 << 29 or batch * max_q * max_kv * group * kv_heads > 1 << 30):
        batch -= 1
    return dict(op=op, batch=batch, max_q=max_q, max_kv=max_kv, spread=rng.uniform(0.0, 0.9), heads=group * kv_heads,
                kv_heads=kv_heads, dim=dim, page=page, fmt=fmt, lens=lens)


def _lengths(case):
    """(new tokens, tokens in the cache after them) of every sequence: the case's own, whatever the seed."""
    rng = random.Random(case["lens"])
    kv = [max(1, int(round(case["max_kv"] * (1.0 - case["spread"] * rng.random())))) for _ in range(case["batch"])]
    kv[0] = case["max_kv"]
    q = [1 if case["max_q"] == 1 else min(kv[b], rng.randrange(max(1, case["max_q"] // 4), case["max_q"] + 1))
         for b in range(case["batch"])]
    q[0] = case["max_q"]
    return q, kv


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        scales = {"row": 4 * case["rows"], "block": 4 * case["rows"] * -(-case["cols"] // 128), "mx": n // 32}[case["mode"]]
        return {"bytes": n * (2 + 1 + (4 if case["residual"] else 0)) + 2 * case["cols"] + scales, "flops": 6 * n}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        scales = {"row": 4 * (M + N), "block": 4 * (M + -(-N // 128)) * -(-K // 128), "mx": (M + N) * K // 32}[case["mode"]]
        out = M * N * (1 if case["out"] == "fp8" else 2)
        extra = (2 * M * N if case["residual"] else 0) + (2 * N if case["bias"] else 0)
        return {"bytes": (M + N) * K + scales + out + extra, "flops": 2 * M * N * K}
    q, kv = _lengths(case)
    if case["op"] == "append":
        n = sum(q) * case["kv_heads"] * case["dim"]
        return {"bytes": 2 * (2 + 1) * n, "flops": 4 * n}
    io = 2 * 2 * sum(q) * case["heads"] * case["dim"]
    seen = sum(n * (k - n) + n * (n + 1) // 2 for n, k in zip(q, kv))
    return {"bytes": 2 * sum(kv) * case["kv_heads"] * case["dim"] + io, "flops": 4 * seen * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ elementary pieces
def _grouped(y, mode, fmt):
    """(codes as FP8 values, scales) of y along its rows: one scale per row, 128 or 32 elements."""
    rows, cols = y.shape
    size = {"row": cols, "block": 128, "mx": 32}[mode]
    n = -(-cols // size)
    z = torch.zeros((rows, n * size), dtype=y.dtype, device=y.device)
    z[:, :cols] = y
    z = z.view(rows, n, size)
    amax = z.abs().amax(2)
    if mode == "mx":
        s = torch.exp2(((torch.frexp(amax)[1] - 1).clamp(min=-119) - 8).to(y.dtype))
    else:
        s = amax.clamp(min=1e-12) / F_MAX[fmt]
    c = (z / s[:, :, None]).clamp(-F_MAX[fmt], F_MAX[fmt]).view(rows, n * size)[:, :cols]
    return c, s.view(rows) if mode == "row" else s


def _e8m0(s):
    return (torch.frexp(s)[1] - 1 + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _spread_scales(s, mode, rows, cols):
    """The scale of every element, from a buffer of one per row, per 128 x 128 block, per 128 or per 32 elements."""
    if mode == "row":
        return s.view(rows, 1)
    if mode == "block128":
        return s.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return s.repeat_interleave(128 if mode == "block" else 32, 1)[:, :cols]


def _activate(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return v / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


# ------------------------------------------------------------------ inputs
def _weight(g, N, K, mode, fmt, device):
    w = torch.randn((N, K), generator=g, device=device) * 0.02
    if mode == "block":
        nb, kb = -(-N // 128), -(-K // 128)
        z = torch.zeros((nb * 128, kb * 128), device=device)
        z[:N, :K] = w
        s = z.view(nb, 128, kb, 128).abs().amax((1, 3)).clamp(min=1e-12) / F_MAX[fmt]
        c = (w / _spread_scales(s, "block128", N, K)).clamp(-F_MAX[fmt], F_MAX[fmt])
        return c.to(DTYPE[fmt]), s
    c, s = _grouped(w, mode, fmt)
    return c.to(DTYPE[fmt]), _e8m0(s) if mode == "mx" else s


def _activations(g, rows, cols, device):
    """N(0, 1) with a few channels fifty times as large, as the linears' inputs have."""
    x = torch.randn((rows, cols), generator=g, device=device)
    x[:, torch.randperm(cols, generator=g, device=device)[:max(1, cols // 1000)]] *= 50.0
    return x


def prepare(case, seed):
    d = "cuda"
    g = torch.Generator(device=d).manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        rows, cols, mode = case["rows"], case["cols"], case["mode"]
        s["x"] = _activations(g, rows, cols, d).bfloat16()
        s["weight"] = (1.0 + 0.2 * torch.randn(cols, generator=g, device=d)).bfloat16()
        if case["residual"]:
            s["residual"] = (4.0 * torch.randn((rows, cols), generator=g, device=d)).bfloat16()
            s["h"] = torch.empty_like(s["x"])
        s["q"] = torch.empty((rows, cols), dtype=torch.uint8, device=d)
        shape = {"row": (rows,), "block": (rows, -(-cols // 128)), "mx": (rows, cols // 32)}[mode]
        s["scale"] = torch.empty(shape, dtype=torch.uint8 if mode == "mx" else torch.float32, device=d)
        return s
    if case["op"] == "gemm":
        M, N, K, mode, fmt = case["M"], case["N"], case["K"], case["mode"], case["fmt"]
        a, sa = _grouped(_activations(g, M, K, d), mode, fmt)
        s["a"], s["sa"] = a.to(DTYPE[fmt]), _e8m0(sa) if mode == "mx" else sa
        s["b"], s["sb"] = _weight(g, N, K, mode, fmt, d)
        if case["bias"]:
            s["bias"] = torch.randn(N, generator=g, device=d).bfloat16()
        if case["residual"]:
            s["residual"] = (4.0 * torch.randn((M, N), generator=g, device=d)).bfloat16()
        if case["out"] == "fp8":
            s["yq"] = torch.empty((M, N), dtype=torch.uint8, device=d)
            s["yq_scale"] = torch.full((1,), 0.05, device=d)
        else:
            s["y"] = torch.empty((M, N), dtype=torch.bfloat16, device=d)
        return s
    # the paged cache: every sequence's pages lie anywhere in the pool
    B, H, D, P, fmt = case["batch"], case["kv_heads"], case["dim"], case["page"], case["fmt"]
    q, kv = _lengths(case)
    per_seq = [-(-n // P) for n in kv]
    pages = sum(per_seq) + 3
    order = torch.randperm(pages, generator=g, device=d).to(torch.int32)
    first = torch.tensor([sum(per_seq[:b]) for b in range(B)], device=d)
    slot = torch.arange(max(per_seq), device=d)
    s["table"] = order[(first[:, None] + slot[None, :]).clamp(max=pages - 1)].contiguous()
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=d)
    s["cu_q"] = torch.tensor([sum(q[:b]) for b in range(B + 1)], dtype=torch.int32, device=d)
    T = sum(q)
    for name in ("k", "v"):
        x = torch.randn((pages, H, P, D), generator=g, device=d)
        x *= torch.exp(0.5 * torch.randn((pages, H, 1, 1), generator=g, device=d))
        scale = _page_scale(x.abs().amax((2, 3)), fmt)
        s[name + "_codes"] = (x / scale[:, :, None, None]).to(DTYPE[fmt]).view(torch.uint8)
        s[name + "_scale"] = scale
        del x
    if case["op"] == "append":
        # K and V as the QKV projection leaves them: side by side in one row per token
        rows = torch.randn((T, 2 * H * D), generator=g, device=d).bfloat16()
        s["k"], s["v"] = rows[:, :H * D].view(T, H, D), rows[:, H * D:].view(T, H, D)
    else:
        s["q"] = torch.randn((T, case["heads"], D), generator=g, device=d).bfloat16()
        s["out"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------------ plain forms
def _norm(s, dt):
    """h, y, the scaled values before their rounding to 8 bits, the scales."""
    case = s["case"]
    h = s["x"].to(dt)
    if case["residual"]:
        h = h + s["residual"].to(dt)
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].to(dt)
    return (h, *_grouped(y, case["mode"], case["fmt"]))


def _plain_norm(s):
    h, c, scale = _norm(s, torch.float32)
    out = {"q": c.to(DTYPE[s["case"]["fmt"]]), "scale": _e8m0(scale) if s["case"]["mode"] == "mx" else scale}
    if s["case"]["residual"]:
        out["h"] = h.bfloat16()
    return out


def _plain_gemm(s):
    case, f32 = s["case"], torch.float32
    bmode = "block128" if case["mode"] == "block" else case["mode"]
    a = s["a"].to(f32) * _spread_scales(s["sa"].to(f32), case["mode"], *s["a"].shape)
    b = s["b"].to(f32) * _spread_scales(s["sb"].to(f32), bmode, *s["b"].shape)
    v = a @ b.T
    if case["bias"]:
        v = v + s["bias"].to(f32)
    v = _activate(v, case["act"])
    if case["residual"]:
        v = v + s["residual"].to(f32)
    y = v.bfloat16()
    if case["out"] == "fp8":
        f = F_MAX[case["fmt"]]
        return {"yq": (y.to(f32) / s["yq_scale"]).clamp(-f, f).to(DTYPE[case["fmt"]])}
    return {"y": y}


def _page_scale(amax, fmt):
    """The least power of two s with max(amax, 1e-12) <= F_max s, F_max being 0.875 of a power of two."""
    m, e = torch.frexp(amax.clamp(min=1e-12))
    top = 9 if fmt == "e4m3" else 16
    return torch.ldexp(torch.ones_like(m), e - top + (m > 0.875).to(e.dtype))


def _token_places(s):
    """Of every new token: its page, its slot in it, and whether the page held tokens before the call."""
    P, dev = s["case"]["page"], s["table"].device
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    t = torch.arange(s["k"].shape[0], device=dev)
    b = torch.searchsorted(cu, t, right=True) - 1
    start = kv[b] - (cu[b + 1] - cu[b])
    pos = start + t - cu[b]
    return s["table"].long()[b, pos // P], pos % P, start, pos // P * P


def _plain_append(s):
    case = s["case"]
    dt, P = DTYPE[case["fmt"]], case["page"]
    page, slot, start, page_start = _token_places(s)
    held = (start - page_start).clamp(min=0)            # tokens that the page held before the call
    pages = s["k_scale"].shape[0]
    touched = torch.zeros(pages, dtype=torch.bool, device=page.device)
    touched[page] = True
    old = torch.zeros(pages, dtype=torch.long, device=page.device)
    old[page] = held
    out = {}
    for name in ("k", "v"):
        x, codes, scale = s[name].float(), s[name + "_codes"], s[name + "_scale"]
        amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(2), "amax")
        new = _page_scale(amax, case["fmt"])
        new = torch.where(old[:, None] > 0, torch.maximum(new, scale), new)
        new = torch.where(touched[:, None], new, scale)
        again = codes.view(dt).float() * (scale / new)[:, :, None, None]
        move = (torch.arange(P, device=page.device)[None, :] < old[:, None])[:, None, :, None]
        codes.copy_(torch.where(move, again.to(dt).view(torch.uint8), codes))
        scale.copy_(new)
        codes.permute(0, 2, 1, 3)[page, slot] = (x / new[page][:, :, None]).to(dt).view(torch.uint8)
        out[name], out[name + "_scale"] = codes.view(dt), scale
    return out


def _attend(s, dt):
    case = s["case"]
    B, H, D, P = case["batch"], case["kv_heads"], case["dim"], case["page"]
    G, Q = case["heads"] // H, case["max_q"]
    cu, kv, dev = s["cu_q"].long(), s["kv_lens"].long(), s["q"].device
    n = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=dev)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].to(dt)[rows].view(B, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
    table = s["table"].long()
    L = table.shape[1] * P
    seen = torch.arange(L, device=dev)[None, None, :] <= (kv - n)[:, None, None] + i[None, :, None]
    seen = seen & (torch.arange(L, device=dev)[None, None, :] < kv[:, None, None])
    values = {}
    for name in ("k", "v"):
        x = s[name + "_codes"].view(DTYPE[case["fmt"]]).to(dt) * s[name + "_scale"].to(dt)[:, :, None, None]
        values[name] = x[table].permute(0, 2, 1, 3, 4).reshape(B, H, L, D)
    scores = (q @ values["k"].transpose(2, 3)) * (1.0 / math.sqrt(D))
    scores = scores.view(B, H, Q, G, L).masked_fill_(~seen[:, None, :, None, :], -math.inf).view(B, H, Q * G, L)
    top = scores.amax(3, keepdim=True)
    p = scores.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = p.sum(3, keepdim=True)
    o = (p @ values["v"]) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(B, H, Q, G, D).permute(0, 2, 1, 3, 4).reshape(B, Q, H * G, D)
    return o[i[None, :] < n[:, None]]


def _plain_attend(s):
    return {"out": _attend(s, torch.float32).bfloat16()}


# ------------------------------------------------------------------ the package's calls
def _own_norm(s):
    from fp8_dynamic_scaled_b200 import binding as f8
    case = s["case"]
    fmt = f8.FP8_E4M3 if case["fmt"] == "e4m3" else f8.FP8_E5M2
    mode = {"row": f8.FP8_SCALE_ROW, "block": f8.FP8_SCALE_BLOCK_1x128, "mx": f8.FP8_SCALE_MX32}[case["mode"]]
    f8.fp8_rmsnorm_quantize(s["x"], s["weight"], EPS, fmt, mode, s["q"], s["scale"], residual=s.get("residual"),
                            sum_out=s.get("h"))
    out = {"q": s["q"].view(DTYPE[case["fmt"]]),
           "scale": s["scale"].view(torch.float8_e8m0fnu) if case["mode"] == "mx" else s["scale"]}
    if case["residual"]:
        out["h"] = s["h"]
    return out


def _own_gemm(s):
    from fp8_dynamic_scaled_b200 import binding as f8
    case = s["case"]
    E4 = f8.FP8_E4M3
    am, bm = {"row": (f8.FP8_SCALE_ROW, f8.FP8_SCALE_ROW), "mx": (f8.FP8_SCALE_MX32, f8.FP8_SCALE_MX32),
              "block": (f8.FP8_SCALE_BLOCK_1x128, f8.FP8_SCALE_BLOCK_128x128)}[case["mode"]]
    act = {"none": f8.FP8_ACT_NONE, "relu": f8.FP8_ACT_RELU, "gelu": f8.FP8_ACT_GELU,
           "gelu_tanh": f8.FP8_ACT_GELU_TANH, "silu": f8.FP8_ACT_SILU}[case["act"]]
    f8.fp8_scaled_gemm_act(s["a"].view(torch.uint8), s["sa"], am, E4, s["b"].view(torch.uint8), s["sb"], bm, E4,
                           s.get("y"), bias=s.get("bias"), activation=act, residual=s.get("residual"), yq=s.get("yq"),
                           yq_scale=s.get("yq_scale"), yq_fmt=E4)
    return {"yq": s["yq"].view(DTYPE["e4m3"])} if case["out"] == "fp8" else {"y": s["y"]}


def _cache(s):
    if "cache" not in s:
        from fp8_dynamic_scaled_b200 import binding as f8
        s["cache"] = f8.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"],
                                f8.FP8_E4M3 if s["case"]["fmt"] == "e4m3" else f8.FP8_E5M2)
    return s["cache"]


def _own_append(s):
    from fp8_dynamic_scaled_b200 import binding as f8
    case, dt = s["case"], DTYPE[s["case"]["fmt"]]
    f8.fp8_kv_append(s["k"], s["v"], _cache(s), s["table"], s["kv_lens"], cu_q=s["cu_q"], max_q_len=case["max_q"])
    return {"k": s["k_codes"].view(dt), "k_scale": s["k_scale"], "v": s["v_codes"].view(dt), "v_scale": s["v_scale"]}


def _own_attend(s):
    from fp8_dynamic_scaled_b200 import binding as f8
    case = s["case"]
    if "workspace" not in s:
        s["workspace"] = f8.kv_attention_workspace(s["q"], _cache(s), case["batch"], case["max_q"], case["max_kv"])
    f8.fp8_kv_attention(s["q"], _cache(s), s["table"], s["kv_lens"], s["out"], cu_q=s["cu_q"], max_q_len=case["max_q"],
                        max_kv_len=case["max_kv"], workspace=s["workspace"])
    return {"out": s["out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "gemm": _own_gemm, "append": _own_append, "attend": _own_attend}[op](state)
    return {"norm": _plain_norm, "gemm": _plain_gemm, "append": _plain_append, "attend": _plain_attend}[op](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    """What the norm and the GEMM round to 8 bits stands here unrounded, as what they round to 16 does; the cache's
    codes are rounded, since a page's later scale starts from them."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        h = s["x"].to(f64) + (s["residual"].to(f64) if case["residual"] else 0.0)
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].to(f64)
        rows, cols = y.shape
        size = {"row": cols, "block": 128, "mx": 32}[case["mode"]]
        a = torch.nn.functional.pad(y, (0, -cols % size)).view(rows, -1, size).abs().amax(2)
        if case["mode"] == "mx":
            scale = torch.pow(2.0, torch.floor(torch.log2(a.clamp(min=2.0 ** -119))) - 8)
        else:
            scale = a.clamp(min=1e-12) / F_MAX[case["fmt"]]
        # an MX value over F_max is clipped, by definition
        q = (y / scale.repeat_interleave(size, 1)[:, :cols]).clamp(-F_MAX[case["fmt"]], F_MAX[case["fmt"]])
        out = {"q": q, "scale": scale.view(rows) if case["mode"] == "row" else scale}
        return {**out, "h": h} if case["residual"] else out
    if case["op"] == "gemm":
        a, b, sa, sb = (s[k].to(torch.float32).to(f64) for k in ("a", "b", "sa", "sb"))
        (M, K), N = a.shape, b.shape[0]
        if case["mode"] == "row":
            v = (a @ b.T) * sa[:, None] * sb[None, :]
        else:
            step = 128 if case["mode"] == "block" else 32
            a = a * sa.repeat_interleave(step, 1)[:, :K]
            sb = sb.repeat_interleave(128, 0)[:N] if case["mode"] == "block" else sb
            v = a @ (b * sb.repeat_interleave(step, 1)[:, :K]).T
        v = v + (s["bias"].to(f64) if case["bias"] else 0.0)
        if case["act"] == "relu":
            v = v.clamp(min=0.0)
        elif case["act"] == "gelu":
            v = v * torch.special.ndtr(v)
        elif case["act"] == "gelu_tanh":
            v = 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
        elif case["act"] == "silu":
            v = v * torch.sigmoid(v)
        v = v + (s["residual"].to(f64) if case["residual"] else 0.0)
        if case["out"] == "fp8":
            return {"yq": (v / s["yq_scale"].to(f64)).clamp(-448.0, 448.0)}
        return {"y": v}
    P, H, D = case["page"], case["kv_heads"], case["dim"]
    new, kv = _lengths(case)
    table = s["table"].cpu().tolist()
    if case["op"] == "append":
        top = 448.0 if case["fmt"] == "e4m3" else 57344.0
        out = {}
        for name in ("k", "v"):
            scale = s[name + "_scale"].to(f64)
            value = s[name + "_codes"].view(DTYPE[case["fmt"]]).to(f64) * scale[:, :, None, None]
            x, t = s[name].to(f64), 0
            for b in range(case["batch"]):
                at = kv[b] - new[b]
                while at < kv[b]:
                    page, n = table[b][at // P], min(P - at % P, kv[b] - at)
                    part = x[t:t + n].transpose(0, 1)
                    a = part.abs().amax((1, 2)).clamp(min=1e-12)
                    need = torch.pow(2.0, torch.ceil(torch.log2(a / top)))
                    scale[page] = torch.maximum(scale[page], need) if at % P else need
                    value[page, :, at % P:at % P + n] = part
                    at, t = at + n, t + n
            value = value / scale[:, :, None, None]         # exact: the scales are powers of two
            out[name], out[name + "_scale"] = value.to(DTYPE[case["fmt"]]).to(f64), scale
        return out
    if max(new) * max(kv) * case["heads"] > 1 << 30:
        return None
    parts, t, G = [], 0, case["heads"] // H
    for b in range(case["batch"]):
        pages = s["table"][b, :-(-kv[b] // P)].long()
        k, v = ((s[n + "_codes"][pages].view(DTYPE[case["fmt"]]).to(f64) * s[n + "_scale"][pages].to(f64)[:, :, None, None])
                .transpose(0, 1).reshape(H, -1, D)[:, :kv[b]] for n in ("k", "v"))
        q = s["q"][t:t + new[b]].to(f64)
        hidden = torch.ones((new[b], kv[b]), dtype=torch.bool, device=q.device).triu(kv[b] - new[b] + 1)
        o = torch.empty_like(q)
        for h in range(case["heads"]):
            z = (q[:, h] @ k[h // G].T / math.sqrt(D)).masked_fill(hidden, -math.inf)
            o[:, h] = torch.softmax(z, 1) @ v[h // G]
        parts.append(o)
        t += new[b]
    return {"out": torch.cat(parts)}
