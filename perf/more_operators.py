"""The operators of a key-value cache held in 4 bits, and rotary positions with several axes, as cases
to be measured: their inputs, their plain forms and their definitions in 64 bits.

    append      rotary embedding of q and k, and k and v into a paged cache. NVFP4 caches: a block of
                16 elements x of a head is stored as E2M1 codes under an E4M3 scale s and the
                tensor's float scale g: s = e4m3(max|x| / (6 g)), code = e2m1(x / (s g)); the tokens
                are then read back, so that what is stored shows as the values it stands for.
                Several axes: pair i of a head turns by the position on its own axis.
    gather      cached tokens back as dense bf16 keys and values
    attention   attention of one new token per sequence over an NVFP4 cache

`own` chooses between the plain forms (elementary torch operations in 32 bits) and the framework's
calls. A case is a dict of plain values; `prepare` makes its inputs from a seed.
"""
import math
import random

import torch

own = False

_SIZE = {"bf16": 2.0, "e4m3": 1.0, "nvfp4": 9 / 16}   # bytes of a cached element
_G = {"bf16": (1.0, 1.0), "e4m3": (0.021, 0.017), "nvfp4": (0.0021, 0.0017)}   # scales of k, v


def listed():
    return [
        # -- rotary embedding and cache append, read back -----------------------------------
        # one decode step of four sequences: latency
        dict(name="append step", op="append", T=4, Hq=32, Hkv=8, D=128, R=128, page=16,
             order="slot", cache="nvfp4", prompt=False, past=2000, axes="one"),
        # a chunk of a prompt behind an earlier one
        dict(name="append prompt", op="append", T=4093, Hq=32, Hkv=8, D=128, R=128, page=64,
             order="slot", cache="nvfp4", prompt=True, past=1001, axes="one"),
        # the next tokens of 37 conversations about images: three axes, taken in turn by the pairs
        dict(name="axes step", op="append", T=37, Hq=28, Hkv=4, D=128, R=128, page=16,
             order="slot", cache="e4m3", prompt=False, past=5000, axes="interleaved"),
        # a prompt of text, images and a video, a section of each head for each axis
        dict(name="axes prompt", op="append", T=9001, Hq=32, Hkv=8, D=128, R=128, page=32,
             order="head", cache="nvfp4", prompt=True, past=0, axes="sections"),
        # -- cached tokens read back --------------------------------------------------------
        # a short prefix, for the attention of what follows it
        dict(name="gather prefix", op="gather", B=1, L=613, ragged=False, Hkv=8, D=128, page=16,
             order="slot", cache="nvfp4"),
        # the contexts of a few long conversations
        dict(name="gather long", op="gather", B=5, L=40000, ragged=True, Hkv=8, D=128, page=64,
             order="slot", cache="nvfp4"),
        # -- attention ----------------------------------------------------------------------
        # a single conversation that just began: latency
        dict(name="attention short", op="attention", B=1, L=777, ragged=False, Hq=32, Hkv=8,
             D=128, page=16, order="slot", window=0),
        # a serving batch of ragged lengths, some sequences empty
        dict(name="attention ragged batch", op="attention", B=48, L=8192, ragged=True, Hq=64,
             Hkv=8, D=128, page=64, order="slot", window=0),
        # three long contexts: the cache's length is split over the GPU
        dict(name="attention long", op="attention", B=3, L=131072, ragged=True, Hq=32, Hkv=8,
             D=128, page=16, order="head", window=0),
        # small heads in groups of seven, layers that look back over a window
        dict(name="attention window", op="attention", B=200, L=5001, ragged=True, Hq=28, Hkv=4,
             D=64, page=32, order="slot", window=1023),
        # wide heads, sixteen queries to a key head
        dict(name="attention wide", op="attention", B=13, L=24001, ragged=True, Hq=32, Hkv=2,
             D=256, page=64, order="head", window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "gather", "attention", "attention", "attention"])
    D = rng.choice([64, 128, 128, 256])
    page, order = rng.choice([16, 24, 32, 64, 128]), rng.choice(["slot", "slot", "head"])
    if op == "append":
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        prompt = rng.random() < 0.5
        # half of the listed prompt's values, or the next tokens of a batch over a pool of a few GB
        top = (9001 * 48 * 128 // ((Hq + 2 * Hkv) * D) // 2 if prompt
               else min(512, 400_000_000 // (3000 * Hkv * D)))
        axes = rng.choice(["one", "sections", "interleaved"])
        R = rng.choice([D // 2, D] if axes != "one" else [0, D // 2, D])
        return dict(op=op, T=_log(rng, 1, min(max(top, 8), 20000)), Hq=Hq, Hkv=Hkv, D=D, R=R, page=page,
                    order=order, cache=rng.choice(["nvfp4", "nvfp4", "bf16", "e4m3"]),
                    prompt=prompt, past=rng.randrange(0, 3000), axes=axes)
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "gather":
        L = _log(rng, 1, 40000)
        B = _log(rng, 1, max(1, min(64, 60_000_000 // (L * Hkv * D))))
        return dict(op=op, B=B, L=L, ragged=rng.random() < 0.6, Hkv=Hkv, D=D, page=page,
                    order=order, cache=rng.choice(["nvfp4", "nvfp4", "bf16", "e4m3"]))
    Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8, 16])
    L = _log(rng, 1, 131072)
    B = _log(rng, 1, max(1, min(256, 100_000_000 // (L * Hkv * D))))
    return dict(op=op, B=B, L=L, ragged=rng.random() < 0.6, Hq=Hq, Hkv=Hkv, D=D, page=page,
                order=order, window=rng.choice([0, 0, 1 + rng.randrange(4096)]))


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


def _pair_axes(case):
    """The axis of each of the R/2 rotary pairs: a quarter time, the rest height and width, as
    consecutive sections or in turn while an axis has pairs left."""
    n = case["R"] // 2
    time = n // 4 if case["axes"] == "sections" else n - 2 * (n * 5 // 16)
    height = (n - time) // 2
    left = [time, height, n - time - height]
    if case["axes"] == "sections":
        return [0] * left[0] + [1] * left[1] + [2] * left[2]
    axes = []
    for i in range(n):
        a = i % 3 if left[i % 3] else next(j for j in range(3) if left[j])
        left[a] -= 1
        axes.append(a)
    return axes


def _axis_positions(T, past, r):
    """Positions int32 [3, T] of a prompt of text runs, images and videos: text advances all axes
    together, the patches of a grid (t, h, w) lie on it, and what follows begins past its largest."""
    parts, at, got = [], past, 0
    while got < T:
        if len(parts) % 2 == 0:
            n = r.randint(9, 90)
            p = (at + torch.arange(n)).expand(3, n)
        else:
            t, h, w = r.choice([1, 1, 1, 7]), r.randint(5, 29), r.randint(5, 29)
            p = torch.stack(torch.meshgrid(torch.arange(t), torch.arange(h), torch.arange(w),
                                           indexing="ij")).reshape(3, -1) + at
        parts.append(p)
        got += p.shape[1]
        at = int(p.max()) + 1
    return torch.cat(parts, 1)[:, :T].to(torch.int32).contiguous()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _e4m3(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _pages(g, counts, width):
    """A block table int32 [len(counts), width]: pages in random order, -1 past a sequence's own."""
    total = sum(counts)
    order = torch.randperm(total + 3, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32)
    at = torch.cat([torch.arange(n) + i * width for i, n in enumerate(counts)]).cuda()
    table = table.cuda()
    table.view(-1)[at] = order
    return table, total + 3


def _quantize(x, g):
    """float32 [..., D] -> (codes u8 [..., D/2], scales E4M3 [..., D/16]); ties to the even code."""
    g = torch.tensor(g, dtype=torch.float32, device=x.device)
    b = x.reshape(*x.shape[:-1], -1, 16)
    s = _e4m3(b.abs().amax(-1) * (1.0 / (6.0 * g)))
    d = s.float() * g
    y = b * torch.where(d > 0, 1.0 / d, 0.0)[..., None]
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = (code | ((y < 0).to(torch.uint8) << 3)).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def _dequantize(codes, scales, g):
    """float32 values of codes u8 [..., D/2] under E4M3 scales [..., D/16]."""
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float32, device=codes.device)
    values = torch.cat([mags, -mags])
    v = torch.stack([values[(codes & 15).int()], values[(codes >> 4).int()]], -1)
    v = v.reshape(*scales.shape, 16) * scales.float()[..., None] * g
    return v.reshape(*codes.shape[:-1], -1)


def _pool(case, P, g, scale):
    """A pool of P pages of N(0, 1) keys or values, [P, page, Hkv, ..] (stored in the case's
    order): (values or codes, block scales or None)."""
    Hkv, D, ps = case["Hkv"], case["D"], case["page"]
    slot = case["order"] == "slot"
    x = _randn(g, P, ps, Hkv, D) if slot else _randn(g, P, Hkv, ps, D)
    kind = case.get("cache", "nvfp4")
    if kind == "nvfp4":
        parts = [_quantize(x[a:a + 4096], scale) for a in range(0, P, 4096)]
        got = [torch.cat([p[0] for p in parts]), torch.cat([p[1].view(torch.uint8) for p in parts])]
        got[1] = got[1].view(torch.float8_e4m3fn)
    else:
        got = [_e4m3(x / scale) if kind == "e4m3" else x.bfloat16(), None]
    return [t if slot or t is None else t.permute(0, 2, 1, 3) for t in got]


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], {"case": case}
    ps, D, Hkv = case["page"], case["D"], case["Hkv"]
    kind = case.get("cache", "nvfp4")
    s["scales"] = _G[kind]
    if op == "append":
        T, Hq, R, past = (case[n] for n in ("T", "Hq", "R", "past"))
        qkv = _randn(g, T, Hq + 2 * Hkv, D).bfloat16()   # one projection's output, used in place
        s["q"], s["k"], s["v"] = qkv.split([Hq, Hkv, Hkv], 1)
        r = random.Random(T * 7919 + past)
        if case["prompt"]:   # T tokens of one sequence
            places = list(range(past, past + T))
            s["seq"] = torch.zeros(T, dtype=torch.int32, device="cuda")
            counts = [-(-(past + T) // ps)]
        else:                # the next token of T sequences
            places = [r.randint(past // 2, past) for _ in range(T)]
            s["seq"] = None
            counts = [n // ps + 1 for n in places]
        s["pos"] = torch.tensor(places, dtype=torch.int32).cuda()
        s["turn"], s["axes"], top = None, None, max(places) + 1
        if case["axes"] != "one":
            s["axes"] = _pair_axes(case)
            if case["prompt"]:
                s["turn"] = _axis_positions(T, past, r).cuda()
            else:   # text behind pictures: an equal, earlier position on each axis
                turn = torch.tensor([n - r.randint(0, n // 2) for n in places], dtype=torch.int32)
                s["turn"] = turn.expand(3, T).contiguous().cuda()
            top = max(top, int(s["turn"].max()) + 1)
        s["table"], P = _pages(g, counts, max(counts))
        if R:
            inv = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
            ang = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * inv
            s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        else:
            s["rope"] = None
        s["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    else:
        lens = _lengths(case)
        counts = [-(-n // ps) for n in lens]
        s["table"], P = _pages(g, counts, max(counts))
        if op == "gather":
            s["pos"] = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
            s["seq"] = torch.cat([torch.full((n,), b, dtype=torch.int32)
                                  for b, n in enumerate(lens)]).cuda()
        else:
            s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
            s["q"] = _randn(g, case["B"], case["Hq"], D).bfloat16()
            s["out"] = torch.empty((case["B"], case["Hq"], D), dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.empty((case["B"], case["Hq"]), dtype=torch.float32, device="cuda")
    (s["kc"], s["ks"]), (s["vc"], s["vs"]) = (_pool(case, P, g, c) for c in s["scales"])
    if op == "gather" or (op == "append" and kind == "nvfp4"):
        n = len(s["pos"])
        s["k_out"], s["v_out"] = (torch.empty((n, Hkv, D), dtype=torch.bfloat16, device="cuda")
                                  for _ in range(2))
    if own:
        from nvfp4_mixture_experts_02_gb300 import ftmoe
        if kind == "nvfp4":
            s["cache"] = ftmoe.NvFP4KVCache(s["kc"], s["vc"], s["ks"], s["vs"], *s["scales"])
        else:
            s["cache"] = ftmoe.PagedKVCache(s["kc"], s["vc"], *s["scales"])
        if s.get("axes") is not None:
            s["axes"] = ftmoe.RopeAxes(s["axes"])
    return s


# ---------------------------------------------------------------- the plain forms
def _turned(s, v):
    rope, v = s["rope"], v.float()
    if rope is None:
        return v
    h = rope.shape[1] // 2
    pair = torch.arange(h, device="cuda")
    if s["axes"] is None:
        at = s["pos"].long()[:, None].expand(-1, h)
    else:
        at = s["turn"].long().T[:, torch.tensor(s["axes"]).cuda()]
    c, sn = rope[at, pair][:, None], rope[at, pair + h][:, None]
    a, b = v[..., :h], v[..., h:2 * h]
    return torch.cat([a * c - b * sn, b * c + a * sn, v[..., 2 * h:]], -1)


def _places(s):
    pos = s["pos"].long()
    seq = s["seq"].long() if s["seq"] is not None else torch.arange(len(pos), device="cuda")
    ps = s["kc"].shape[1]
    return s["table"][seq, pos // ps].long(), pos % ps


def _bits(t):
    return t if t.dtype == torch.bfloat16 else t.view(torch.uint8)


def _plain_append(s):
    at = _places(s)
    got = {"q": _turned(s, s["q"]).bfloat16()}
    for n, x in (("k", _turned(s, s["k"])), ("v", s["v"].float())):
        g = s["scales"][n == "v"]
        pool, scales = s[n + "c"], s[n + "s"]
        if scales is not None:
            codes, sc = _quantize(x, g)
            pool[at] = codes
            _bits(scales)[at] = _bits(sc)
            got[n] = _dequantize(pool[at], _bits(scales)[at].view(sc.dtype), g).bfloat16()
            got[n + "_scales"] = scales
        else:
            to = _e4m3(x * (1.0 / torch.tensor(g, device="cuda"))) if pool.dtype != torch.bfloat16 else x.bfloat16()
            _bits(pool)[at] = _bits(to)
            got[n] = pool
    return got


def _plain_gather(s):
    at = _places(s)
    got = {}
    for n in "kv":
        g, x = s["scales"][n == "v"], _bits(s[n + "c"])[at]
        if s[n + "s"] is not None:
            x = _dequantize(x, _bits(s[n + "s"])[at].view(torch.float8_e4m3fn), g)
        else:
            x = x.view(s[n + "c"].dtype).float() * g
        got[n] = x.bfloat16()
    return got


def _plain_attention(s):
    case = s["case"]
    B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
    table, lens = s["table"].clamp_min(0).long(), s["lens"][:, None].long()
    n = table.shape[1] * case["page"]
    at = torch.arange(n, device="cuda")[None]
    seen = at < lens
    if case["window"]:
        seen = seen & (at >= lens - case["window"])
    k, v = (_dequantize(s[c + "c"][table], _bits(s[c + "s"])[table].view(torch.float8_e4m3fn), g)
            .reshape(B, n, Hkv, D) for c, g in zip("kv", s["scales"]))
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, D)
    a = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))       # [B, Hkv, G, n]
    a = a.masked_fill(~seen[:, None, None], -math.inf)
    m = a.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(a - m)
    l = p.sum(-1, keepdim=True)
    v = v.masked_fill(~seen[:, :, None, None], 0.0)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(l > 0, l, 1.0)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)
    return {"out": o.reshape(B, Hq, D).bfloat16(), "lse": lse.reshape(B, Hq)}


_PLAIN = {"append": _plain_append, "gather": _plain_gather, "attention": _plain_attention}


# ---------------------------------------------------------------- the framework's calls
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    from nvfp4_mixture_experts_02_gb300 import ftmoe
    if op == "append":
        q = ftmoe.kv_append(s["k"], s["v"], s["cache"], s["table"], s["pos"], seq_ids=s["seq"],
                            q=s["q"], rope=s["rope"], rope_positions=s["turn"], rope_axes=s["axes"],
                            q_out=s["q_out"])
        if s["ks"] is None:
            return {"q": q, "k": s["kc"], "v": s["vc"]}
    if op != "attention":
        k, v = ftmoe.kv_gather(s["cache"], s["table"], s["pos"], seq_ids=s["seq"], k_out=s["k_out"],
                               v_out=s["v_out"])
        if op == "gather":
            return {"k": k, "v": v}
        return {"q": q, "k": k, "v": v, "k_scales": s["ks"], "v_scales": s["vs"]}
    out, lse = ftmoe.paged_decode_attention(s["q"], s["cache"], s["table"], s["lens"],
                                            window=s["case"]["window"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    size = _SIZE[case.get("cache", "nvfp4")]
    if op == "append":
        T, Hq = case["T"], case["Hq"]
        # written: q and the cache; an NVFP4 cache is then read back, as bf16
        b = T * D * (2 * (2 * Hq + 2 * Hkv) + 2 * Hkv * size)
        if case["cache"] == "nvfp4":
            b += T * D * 2 * Hkv * (size + 2)
        tables = 4 * case["R"] + 12 + (0 if case["axes"] == "one" else 12)
        return {"bytes": b + T * tables, "flops": 3.0 * T * (Hq + Hkv) * case["R"]}
    keys = sum(min(n, case.get("window") or n) for n in _lengths(case))
    pages = sum(-(-min(n, case.get("window") or n) // case["page"]) for n in _lengths(case))
    if op == "gather":
        return {"bytes": 2 * keys * Hkv * D * (size + 2) + 8 * keys + 4 * pages,
                "flops": 4.0 * keys * Hkv * D}
    Hq = case["Hq"]
    return {"bytes": 2 * keys * Hkv * D * size + case["B"] * Hq * (4 * D + 4) + 4 * pages + 4 * case["B"],
            "flops": 4.0 * keys * Hq * D}


# ---------------------------------------------------------------- the definitions in 64 bits
def _nearest(v, bits, low, top):
    """The nearest number of `bits` significant bits, steps no finer than those at 2^low, of a
    magnitude up to `top`; ties to even."""
    e = torch.frexp(v).exponent.double() - 1
    step = torch.exp2(e.clamp_min(low) - (bits - 1))
    return (torch.round(v / step) * step).clamp(-top, top)


def _stored(pool, scales, at):
    """Values without the tensor's scale of the slots `at` of an NVFP4 cache, in 64 bits."""
    page, slot = at
    c = pool[page, slot]
    part = torch.empty((*c.shape, 2), dtype=torch.int64, device="cuda")
    part[..., 0], part[..., 1] = c % 16, c // 16
    e, m = (part // 2 % 4).double(), (part % 2).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e - 1))
    mag = torch.where(part >= 8, -mag, mag).reshape(*c.shape[:-1], -1)
    b = scales.view(torch.uint8)[page, slot].to(torch.int64)
    se, sm = (b // 8 % 16).double(), (b % 8).double()
    sc = torch.where(se == 0, sm * 2.0 ** -9, (1 + sm / 8) * torch.exp2(se - 7))
    return mag * sc.repeat_interleave(16, -1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, ps = case["op"], case["page"]
    if op == "attention":
        B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
        G = Hq // Hkv
        out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lengths(case)):
            first = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            at = torch.arange(first, n, device="cuda")
            at = (s["table"][b].long()[at // ps], at % ps)
            k = _stored(s["kc"], s["ks"], at) * s["scales"][0]
            v = _stored(s["vc"], s["vs"], at) * s["scales"][1]
            for h in range(Hkv):
                q = s["q"][b, h * G:(h + 1) * G].double() / math.sqrt(D)
                a = q @ k[:, h].T
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(a, -1)
                out[b, h * G:(h + 1) * G] = torch.softmax(a, -1) @ v[:, h]
        return {"out": out, "lse": lse}
    pos = s["pos"].long()
    seq = s["seq"].long() if s["seq"] is not None else torch.arange(len(pos), device="cuda")
    at = (s["table"][seq, pos // ps].long(), pos % ps)
    if op == "gather":
        got = {}
        for n, g in zip("kv", s["scales"]):
            if case["cache"] == "nvfp4":
                got[n] = _stored(s[n + "c"], s[n + "s"], at) * g
            else:
                got[n] = s[n + "c"].double()[at] * g
        return got
    R = case["R"]

    def turned(v):
        v = v.double().clone()
        if R:
            # which position each pair turns by: the token's place, or the one on the pair's axis
            which = torch.zeros(R // 2, dtype=torch.int64) if s["axes"] is None else torch.tensor(s["axes"])
            rows = (s["pos"][None] if s["axes"] is None else s["turn"]).long()[which.cuda()]   # [R/2, T]
            table = s["rope"].double()
            c, sn = (t.T.gather(1, rows).T[:, None] for t in (table[:, :R // 2], table[:, R // 2:]))
            z = torch.complex(v[..., :R // 2], v[..., R // 2:R]) * torch.complex(c, sn)
            v[..., :R // 2], v[..., R // 2:R] = z.real, z.imag
        return v
    got = {"q": turned(s["q"])}
    for n, x, g in (("k", turned(s["k"]), s["scales"][0]), ("v", s["v"].double(), s["scales"][1])):
        if case["cache"] == "nvfp4":
            b = x.unflatten(-1, (-1, 16))
            sc = _nearest(b.abs().amax(-1) / (6 * g), 4, -6, 448.0)
            d = sc[..., None] * g
            code = torch.where(d > 0, _nearest(b / d.clamp_min(1e-300), 2, 0, 6.0), 0.0)
            got[n] = (code * d).flatten(-2)
            got[n + "_scales"] = s[n + "s"].double()
            got[n + "_scales"][at] = sc
        else:
            got[n] = s[n + "c"].double()
            got[n][at] = (x / g).clamp(-448, 448) if case["cache"] == "e4m3" else x
    return got
