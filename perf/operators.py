"""The operators of a transformer decode block around the mixture-of-experts layer, as cases to
be measured: their inputs, their plain forms and their definitions in 64 bits.

    nvfp4_linear              y = W x with a dense NVFP4 matrix (E2M1 codes, an E4M3 scale per 16
                              elements of a row, one float32 scale), 1 to 64 tokens
    kv_append                 rotary embedding of q and k, and k and v into a paged cache (bf16, or
                              E4M3 with a scale)
    paged_decode_attention    attention of one new token per sequence over that cache
    residual_norm             r' = r + scale * gate * norm(y), x' = norm(r'): the norm after a
                              block, the gated residual sum and the norm before the next block
    residual_norm_backward    its gradient

`own` chooses between the plain forms (elementary torch operations in 32 bits) and the
framework's calls. A case is a dict of plain values; `prepare` makes its inputs from a seed.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
_SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}
EPS = 1e-6


def listed():
    return [
        # -- dense NVFP4 products of a decode step ------------------------------------------
        # the fused q, k, v projection of one token (32 + 2 * 8 heads of 128)
        dict(name="linear one token", op="linear", T=1, N=6144, K=4096, out="bf16"),
        # the attention's output projection for a decode batch
        dict(name="linear batch of 32", op="linear", T=32, N=4096, K=4096, out="bf16"),
        # next-token logits of a few sequences, a vocabulary of odd size, kept in float32
        dict(name="linear logits", op="linear", T=5, N=100003, K=4096, out="f32"),
        # -- rotary embedding and cache append ----------------------------------------------
        # one decode step of four sequences
        dict(name="append four tokens", op="append", T=4, Hq=32, Hkv=8, D=128, R=128, page=16,
             cache="bf16", prompt=False, past=2048),
        # a prompt chunk of odd length into an 8-bit cache, half of each head rotated
        dict(name="append prompt", op="append", T=4093, Hq=32, Hkv=8, D=128, R=64, page=64,
             cache="e4m3", prompt=True, past=1000),
        # -- attention of one new token per sequence ----------------------------------------
        # a single conversation, one that just began: latency
        dict(name="attention short", op="attention", B=1, L=777, ragged=False, Hq=32, Hkv=8,
             D=128, page=16, cache="bf16", window=0),
        # a serving batch of ragged lengths (some sequences empty), 8-bit cache
        dict(name="attention ragged batch", op="attention", B=48, L=8192, ragged=True, Hq=64,
             Hkv=8, D=128, page=64, cache="e4m3", window=0),
        # three long contexts: the cache's length is split over the GPU
        dict(name="attention long", op="attention", B=3, L=131072, ragged=True, Hq=32, Hkv=8,
             D=128, page=16, cache="bf16", window=0),
        # -- norms, gate and residual sum ---------------------------------------------------
        # between two blocks of a decode step of one token
        dict(name="norm one token", op="norm", T=1, H=4096, res="bf16", post=True, pre=True,
             gate="token"),
        # a prompt or a training batch, the residual stream kept in float32
        dict(name="norm batch", op="norm", T=8191, H=4096, res="f32", post=True, pre=True,
             gate="channel"),
        # gradients: a small batch with an elementwise gate
        dict(name="norm gradient small", op="norm_backward", T=509, H=4096, res="bf16", post=True,
             pre=True, gate="element"),
        # gradients of a training batch
        dict(name="norm gradient batch", op="norm_backward", T=8192, H=8192, res="bf16", post=True,
             pre=True, gate="channel"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "append", "attention", "attention", "attention", "norm",
                     "norm_backward"])
    if op == "linear":
        K = 32 * _log(rng, 8, 512)
        N = _log(rng, 64, min(100003, 100003 * 4096 // K))
        return dict(op=op, T=_log(rng, 1, 64), N=N, K=K, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "append":
        D = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        return dict(op=op, T=_log(rng, 1, max(8, 4093 * 6144 // ((Hq + 2 * Hkv) * D) // 2)),
                    Hq=Hq, Hkv=Hkv, D=D, R=rng.choice([0, D // 2, D]),
                    page=rng.choice([16, 24, 32, 64]), cache=rng.choice(["bf16", "e4m3"]),
                    prompt=rng.random() < 0.5, past=rng.randrange(0, 3000))
    if op == "attention":
        D = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8, 16])
        L = _log(rng, 1, 131072)
        # at most half of the largest listed cache, ragged or not
        B = _log(rng, 1, max(1, min(256, 100_000_000 // (L * Hkv * D))))
        return dict(op=op, B=B, L=L, ragged=rng.random() < 0.6, Hq=Hq, Hkv=Hkv, D=D,
                    page=rng.choice([16, 24, 32, 64, 128]), cache=rng.choice(["bf16", "e4m3"]),
                    window=rng.choice([0, 0, 1 + rng.randrange(4096)]))
    H = 8 * _log(rng, 8, 2048)
    T = _log(rng, 1, max(2, (1 << 25) // H))
    post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
    return dict(op=op, T=T, H=H, res=rng.choice(["bf16", "bf16", "f32"]), post=post, pre=pre,
                gate=rng.choice(["none", "channel", "token", "element"]))


def _lengths(case):
    """Sequence lengths, a function of the case alone. Ragged: one full, about one in eight
    empty, the rest spread."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    r = random.Random(B * 1000003 + L)
    lens = [0 if r.random() < 0.125 else r.randint(max(1, L // 8), L) for _ in range(B)]
    lens[r.randrange(B)] = L
    return lens


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _e4m3(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _quantize(g, N, K):
    """N(0, 0.02) weights in NVFP4: (codes u8 [N, K/2], scales u8 [N, K/16], float32 [1])."""
    w = _randn(g, N, K // 16, 16).mul_(0.02)
    gscale = (w.abs().amax() / (6.0 * 448.0)).reshape(1)
    s = _e4m3(w.abs().amax(-1, keepdim=True) / (6.0 * gscale))
    w = (w / (s.float() * gscale).clamp_min(1e-30)).reshape(N, K)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(w.abs(), mid, out_int32=True).to(torch.uint8)
    code |= (w < 0).to(torch.uint8) << 3
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    return codes.contiguous(), s.view(torch.uint8).reshape(N, K // 16).contiguous(), gscale


def _pages(g, counts, width):
    """A block table int32 [len(counts), width]: pages in random order, -1 past a sequence's own."""
    total = sum(counts)
    order = torch.randperm(total + 3, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32)
    at = torch.cat([torch.arange(n) + i * width for i, n in enumerate(counts)]).cuda()
    table = table.cuda()
    table.view(-1)[at] = order
    return table, total + 3


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], {"case": case}
    if op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        s["x"] = _randn(g, T, K).bfloat16()
        s["w"] = _quantize(g, N, K)
        s["out"] = torch.empty((T, N), dtype=_DT[case["out"]], device="cuda")
        if own:
            from nvfp4_mixture_experts_02_gb300 import ftmoe
            s["weight"] = ftmoe.NvFP4Linear(*s["w"])
    elif op == "append":
        T, Hq, Hkv, D, R, ps = (case[n] for n in ("T", "Hq", "Hkv", "D", "R", "page"))
        past = case["past"]
        qkv = _randn(g, T, Hq + 2 * Hkv, D).bfloat16()   # one projection's output, used in place
        s["q"], s["k"], s["v"] = qkv.split([Hq, Hkv, Hkv], 1)
        if case["prompt"]:   # T tokens of one sequence
            s["pos"] = torch.arange(past, past + T, dtype=torch.int32, device="cuda")
            s["seq"] = torch.zeros(T, dtype=torch.int32, device="cuda")
            counts, top = [-(-(past + T) // ps)], past + T
        else:                # the next token of T sequences
            r = random.Random(T * 7919 + past)
            lens = [r.randint(past // 2, past) for _ in range(T)]
            s["pos"] = torch.tensor(lens, dtype=torch.int32).cuda()
            s["seq"] = None
            counts, top = [n // ps + 1 for n in lens], past + 1
        s["table"], P = _pages(g, counts, max(counts))
        s["scales"] = (0.021, 0.017) if case["cache"] == "e4m3" else (1.0, 1.0)
        cast = _e4m3 if case["cache"] == "e4m3" else (lambda v: v.bfloat16())
        s["kc"] = cast(_randn(g, P, ps, Hkv, D))
        s["vc"] = cast(_randn(g, P, ps, Hkv, D))
        if R:
            inv = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
            ang = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * inv
            s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        else:
            s["rope"] = None
        s["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        if own:
            from nvfp4_mixture_experts_02_gb300 import ftmoe
            s["cache"] = ftmoe.PagedKVCache(s["kc"], s["vc"], *s["scales"])
    elif op == "attention":
        B, Hq, Hkv, D, ps = (case[n] for n in ("B", "Hq", "Hkv", "D", "page"))
        lens = _lengths(case)
        counts = [-(-n // ps) for n in lens]
        s["table"], P = _pages(g, counts, max(counts))
        s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        s["q"] = _randn(g, B, Hq, D).bfloat16()
        s["scales"] = (0.021, 0.017) if case["cache"] == "e4m3" else (1.0, 1.0)
        cast = ((lambda v, c: _e4m3(v / c)) if case["cache"] == "e4m3"
                else (lambda v, c: v.bfloat16()))
        s["kc"] = cast(_randn(g, P, ps, Hkv, D), s["scales"][0])
        s["vc"] = cast(_randn(g, P, ps, Hkv, D), s["scales"][1])
        s["out"] = torch.empty((B, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((B, Hq), dtype=torch.float32, device="cuda")
        if own:
            from nvfp4_mixture_experts_02_gb300 import ftmoe
            s["cache"] = ftmoe.PagedKVCache(s["kc"], s["vc"], *s["scales"])
    else:
        T, H, rt = case["T"], case["H"], _DT[case["res"]]
        s["y"] = _randn(g, T, H).bfloat16()
        s["r"] = _randn(g, T, H).mul_(3.0).to(rt)
        s["w_post"] = (1 + 0.1 * _randn(g, H)).bfloat16() if case["post"] else None
        s["w_pre"] = (1 + 0.1 * _randn(g, H)).bfloat16() if case["pre"] else None
        shape = {"none": None, "channel": (H,), "token": (T, 1), "element": (T, H)}[case["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(_randn(g, *shape)).bfloat16()
        s["scale"] = 0.7
        if op == "norm_backward":
            s["dr"] = _randn(g, T, H).to(rt)
            s["dx"] = _randn(g, T, H).bfloat16() if case["pre"] else None
    return s


# ---------------------------------------------------------------- the plain forms
def _plain_linear(s):
    codes, scales, gscale = s["w"]
    N, K = codes.shape[0], codes.shape[1] * 2
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float32, device="cuda")
    values = torch.cat([mags, -mags])
    w = values[torch.stack([codes & 15, codes >> 4], -1).int()].reshape(N, K // 16, 16)
    w = (w * scales.view(torch.float8_e4m3fn).float()[..., None]).reshape(N, K)
    y = (s["x"].float() @ w.T) * gscale
    return {"y": y.to(s["out"].dtype)}


def _rotate(v, rope, pos):
    if rope is None:
        return v.float()
    h = rope.shape[1] // 2
    c, sn = rope[pos.long(), None, :h], rope[pos.long(), None, h:]
    v = v.float()
    a, b = v[..., :h], v[..., h:2 * h]
    return torch.cat([a * c - b * sn, b * c + a * sn, v[..., 2 * h:]], -1)


def _plain_append(s):
    ps, pos = s["kc"].shape[1], s["pos"].long()
    seq = s["seq"].long() if s["seq"] is not None else torch.arange(len(pos), device="cuda")
    page = s["table"][seq, pos // ps].long()
    for_cache = ((lambda v, c: _e4m3(v / c).view(torch.uint8)) if s["kc"].dtype != torch.bfloat16
                 else (lambda v, c: v.bfloat16()))
    bits = (lambda c: c.view(torch.uint8)) if s["kc"].dtype != torch.bfloat16 else (lambda c: c)
    bits(s["kc"])[page, pos % ps] = for_cache(_rotate(s["k"], s["rope"], s["pos"]), s["scales"][0])
    bits(s["vc"])[page, pos % ps] = for_cache(s["v"].float(), s["scales"][1])
    return {"q": _rotate(s["q"], s["rope"], s["pos"]).bfloat16(), "k": s["kc"], "v": s["vc"]}


def _plain_attention(s):
    case = s["case"]
    B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
    table, lens = s["table"].clamp_min(0).long(), s["lens"][:, None].long()
    n = table.shape[1] * case["page"]
    at = torch.arange(n, device="cuda")[None]
    seen = at < lens
    if case["window"]:
        seen = seen & (at >= lens - case["window"])
    k = s["kc"][table].reshape(B, n, Hkv, D).float() * s["scales"][0]
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, D)
    a = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))       # [B, Hkv, G, n]
    a = a.masked_fill(~seen[:, None, None], -math.inf)
    m = a.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(a - m)
    l = p.sum(-1, keepdim=True)
    v = s["vc"][table].reshape(B, n, Hkv, D).float() * s["scales"][1]
    v = v.masked_fill(~seen[:, :, None, None], 0.0)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(l > 0, l, 1.0)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)
    return {"out": o.reshape(B, Hq, D).bfloat16(), "lse": lse.reshape(B, Hq)}


def _norm_parts(y, r, w_post, w_pre, gate, scale):
    """z, r' and the reciprocal rms of y and r', in the type of y."""
    s1 = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    z = y * s1 * w_post if w_post is not None else y
    out = r + scale * (z if gate is None else gate * z)
    s2 = torch.rsqrt(out.square().mean(-1, keepdim=True) + EPS)
    return z, out, s1, s2


def _cast(t, dtype):
    return None if t is None else t.to(dtype)


def _plain_norm(s):
    w_pre = _cast(s["w_pre"], torch.float32)
    _, r, _, s2 = _norm_parts(s["y"].float(), s["r"].float(), _cast(s["w_post"], torch.float32),
                              w_pre, _cast(s["gate"], torch.float32), s["scale"])
    return {"r": r.to(s["r"].dtype),
            "x": None if w_pre is None else (r * s2 * w_pre).bfloat16()}


def _norm_gradient(s, dt):
    y, r, w_post, w_pre, gate, dr, dx = (_cast(s[n], dt) for n in
                                         ("y", "r", "w_post", "w_pre", "gate", "dr", "dx"))
    z, out, s1, s2 = _norm_parts(y, r, w_post, w_pre, gate, s["scale"])
    got = dict(dw_post=None, dw_pre=None, dgate=None)
    if w_pre is not None:
        d = dx * w_pre
        dr = dr + s2 * (d - out * s2.square() * (d * out).mean(-1, keepdim=True))
        got["dw_pre"] = (dx * out * s2).sum(0)
    dz = s["scale"] * (dr if gate is None else gate * dr)
    if gate is not None:
        dg = s["scale"] * z * dr
        got["dgate"] = (dg.sum(0) if gate.dim() == 1 else
                        dg.sum(1, keepdim=True) if gate.shape[1] == 1 else dg)
    dy = dz
    if w_post is not None:
        got["dw_post"] = (dz * y * s1).sum(0)
        d = dz * w_post
        dy = s1 * (d - y * s1.square() * (d * y).mean(-1, keepdim=True))
    return dict(got, dy=dy, dr=dr)


def _plain_norm_backward(s):
    got = _norm_gradient(s, torch.float32)
    got["dy"], got["dr"] = got["dy"].bfloat16(), got["dr"].to(s["r"].dtype)
    if s["case"]["gate"] == "element":
        got["dgate"] = got["dgate"].bfloat16()
    return got


_PLAIN = {"linear": _plain_linear, "append": _plain_append, "attention": _plain_attention,
          "norm": _plain_norm, "norm_backward": _plain_norm_backward}


# ---------------------------------------------------------------- the framework's calls
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    from nvfp4_mixture_experts_02_gb300 import ftmoe
    if op == "linear":
        return {"y": ftmoe.nvfp4_linear(s["x"], s["weight"], out=s["out"])}
    if op == "append":
        q = ftmoe.kv_append(s["k"], s["v"], s["cache"], s["table"], s["pos"], seq_ids=s["seq"],
                            q=s["q"], rope=s["rope"], q_out=s["q_out"])
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    if op == "attention":
        out, lse = ftmoe.paged_decode_attention(s["q"], s["cache"], s["table"], s["lens"],
                                                window=s["case"]["window"], out=s["out"],
                                                lse=s["lse"])
        return {"out": out, "lse": lse}
    if op == "norm":
        r, x = ftmoe.residual_norm(s["y"], s["r"], w_post=s["w_post"], w_pre=s["w_pre"],
                                   gate=s["gate"], scale=s["scale"], eps=EPS)
        return {"r": r, "x": x}
    d = ftmoe.residual_norm_backward(s["y"], s["r"], s["dr"], s["dx"], w_post=s["w_post"],
                                     w_pre=s["w_pre"], gate=s["gate"], scale=s["scale"], eps=EPS)
    return {"dy": d.dy, "dr": d.dresidual, "dw_post": d.dw_post, "dw_pre": d.dw_pre,
            "dgate": d.dgate}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": N * K * 9 // 16 + 4 + 2 * T * K + T * N * _SIZE[case["out"]],
                "flops": 2.0 * T * N * K}
    if op == "append":
        T, Hq, Hkv, D = (case[n] for n in ("T", "Hq", "Hkv", "D"))
        b = T * D * (2 * (2 * Hq + 2 * Hkv) + 2 * Hkv * _SIZE[case["cache"]])
        return {"bytes": b + T * (4 * case["R"] + 12), "flops": 3.0 * T * (Hq + Hkv) * case["R"]}
    if op == "attention":
        Hq, Hkv, D = (case[n] for n in ("Hq", "Hkv", "D"))
        keys = sum(min(n, case["window"] or n) for n in _lengths(case))
        pages = sum(-(-min(n, case["window"] or n) // case["page"]) for n in _lengths(case))
        return {"bytes": 2 * keys * Hkv * D * _SIZE[case["cache"]] + case["B"] * Hq * (4 * D + 4)
                + 4 * pages + 4 * case["B"], "flops": 4.0 * keys * Hq * D}
    T, H, rs = case["T"], case["H"], _SIZE[case["res"]]
    gate = {"none": 0, "channel": H, "token": T, "element": T * H}[case["gate"]]
    if op == "norm":
        vectors = 2 * H * (case["post"] + case["pre"]) + 2 * gate
        return {"bytes": T * H * (2 + 2 * rs + 2 * case["pre"]) + vectors, "flops": 10.0 * T * H}
    vectors = 6 * H * (case["post"] + case["pre"])
    vectors += {"none": 0, "channel": 6 * H, "token": 6 * T, "element": 4 * T * H}[case["gate"]]
    return {"bytes": T * H * (4 + 3 * rs + 2 * case["pre"]) + vectors, "flops": 30.0 * T * H}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        codes, scales, gscale = s["w"]
        c = torch.empty((codes.shape[0], codes.shape[1], 2), dtype=torch.uint8, device="cuda")
        c[..., 0], c[..., 1] = codes & 15, codes >> 4
        y = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        x = s["x"].double()
        for a in range(0, c.shape[0], 8192):   # rows at a time: the matrix in 64 bits is large
            part = c[a:a + 8192].reshape(-1, x.shape[1])
            e, m = ((part >> 1) & 3).double(), (part & 1).double()
            mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e - 1))
            mag = torch.where((part & 8) != 0, -mag, mag)
            b = scales[a:a + 8192].to(torch.int32)
            se, sm = ((b >> 3) & 15).double(), (b & 7).double()
            sc = torch.where(se == 0, sm * 2.0 ** -9, (1 + sm / 8) * torch.exp2(se - 7))
            y[:, a:a + 8192] = x @ (mag * sc.repeat_interleave(16, 1)).T
        return {"y": y * gscale.double()}
    if op == "append":
        T, R, ps = case["T"], case["R"], case["page"]
        pos = s["pos"].long()

        def turned(v):
            v = v.double().clone()
            if R:
                c = s["rope"][pos].double()
                z = torch.complex(v[..., :R // 2], v[..., R // 2:R])
                z = z * torch.complex(c[:, :R // 2], c[:, R // 2:])[:, None]
                v[..., :R // 2], v[..., R // 2:R] = z.real, z.imag
            return v
        seq = s["seq"].long() if s["seq"] is not None else torch.arange(T, device="cuda")
        at = s["table"][seq, pos // ps].long() * ps + pos % ps
        k = s["kc"].double().reshape(-1, *s["kc"].shape[2:])
        v = s["vc"].double().reshape(-1, *s["vc"].shape[2:])
        k[at] = turned(s["k"]) / s["scales"][0]
        v[at] = s["v"].double() / s["scales"][1]
        if case["cache"] == "e4m3":
            k, v = k.clamp(-448, 448), v.clamp(-448, 448)
        return {"q": turned(s["q"]), "k": k.reshape(s["kc"].shape), "v": v.reshape(s["vc"].shape)}
    if op == "attention":
        B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
        G = Hq // Hkv
        out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
        ps = case["page"]
        for b, n in enumerate(_lengths(case)):
            first = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            at = torch.arange(first, n, device="cuda")
            page = s["table"][b].long()[at // ps]
            k = s["kc"][page, at % ps].double() * s["scales"][0]
            v = s["vc"][page, at % ps].double() * s["scales"][1]
            for h in range(Hkv):
                q = s["q"][b, h * G:(h + 1) * G].double() / math.sqrt(D)
                a = (q[:, None, :] * k[None, :, h]).sum(-1) if G * len(at) < 4096 else q @ k[:, h].T
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(a, -1)
                out[b, h * G:(h + 1) * G] = torch.softmax(a, -1) @ v[:, h]
        return {"out": out, "lse": lse}
    y, r, gate = (_cast(s[n], torch.float64) for n in ("y", "r", "gate"))
    w_post, w_pre = (_cast(s[n], torch.float64) for n in ("w_post", "w_pre"))
    leaf = [t.requires_grad_() for t in (y, r, gate, w_post, w_pre) if t is not None]
    with torch.enable_grad():
        norm = lambda v, w: v / (v.square().mean(-1, keepdim=True) + EPS).sqrt() * w  # noqa: E731
        z = norm(y, w_post) if w_post is not None else y
        out = r + s["scale"] * z * (1.0 if gate is None else gate)
        x = norm(out, w_pre) if w_pre is not None else None
        if op == "norm":
            return {"r": out.detach(), "x": None if x is None else x.detach()}
        total = (out * s["dr"].double()).sum()
        if x is not None:
            total = total + (x * s["dx"].double()).sum()
        torch.autograd.backward(total, inputs=leaf)
    grad = lambda t: None if t is None else t.grad  # noqa: E731
    return {"dy": y.grad, "dr": r.grad, "dw_post": grad(w_post), "dw_pre": grad(w_pre),
            "dgate": grad(gate)}
