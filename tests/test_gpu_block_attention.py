"""GPU parity of the cache append and of paged attention against float64 (append: bit-exact against
float32 arithmetic).

Attention tolerance: scores of D products in float32 are within (D/16 + 4) 2^-23 of their sum of
magnitudes, about 1e-5 for the normal q and k here; the weights add 2^-16 (two bf16) or 2^-11 (f16,
E4M3 caches), numerator and denominator: rel = 2^-14 or 2^-10 of sum p|v|, then one bf16 rounding.
"""
import math

import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.block_util import bf16, close, f64
from tests.layer_util import ftmoe

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def paged(rng, lens, page, Hkv, D, dtype, order="slot", spare=3, width=None):
    """(cache k, cache v, table, keys, values): pages in random order in a pool whose unused slots
    are NaN, and the sequences' float32 keys and values as stored."""
    counts = [-(-n // page) for n in lens]
    P = sum(counts) + spare
    perm = rng.permutation(P)
    table = np.full((len(lens), width or max(max(counts), 1)), -7, np.int32)
    shape = (P, page, Hkv, D) if order == "slot" else (P, Hkv, page, D)
    pools, seqs = [], [[], []]
    for which in range(2):
        pool = torch.full(shape, float("nan")).to(dtype)
        view = pool if order == "slot" else pool.permute(0, 2, 1, 3)
        at = 0
        for b, n in enumerate(lens):
            vals = torch.from_numpy(rng.standard_normal((n, Hkv, D)).astype(np.float32)).to(dtype)
            for i in range(counts[b]):
                part = vals[i * page:(i + 1) * page]
                view[int(perm[at])].view(torch.uint8 if dtype == F8 else torch.int16)[:len(part)] = \
                    part.view(torch.uint8 if dtype == F8 else torch.int16)
                table[b, i] = perm[at]
                at += 1
            seqs[which].append(vals.double().numpy())
        pools.append(pool.cuda() if order == "slot" else pool.cuda().permute(0, 2, 1, 3))
    return pools[0], pools[1], torch.from_numpy(table).cuda(), seqs[0], seqs[1]


def check(lens, page, Hq, Hkv, D, dtype, seed, order="slot", window=0, scales=(1.0, 1.0), scale=None):
    m = ftmoe()
    rng = np.random.default_rng(seed)
    kc, vc, table, ks, vs = paged(rng, lens, page, Hkv, D, dtype, order)
    q = bf16(rng.standard_normal((len(lens), Hq, D)))
    cache = m.PagedKVCache(kc, vc, *scales)
    n = m.paged_attention_workspace_bytes(len(lens), D)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")   # NaN patterns
    ws = ws[(-ws.data_ptr()) % 256:][:n]
    ws[:1024] = 0
    out, lse = m.paged_decode_attention(q.cuda(), cache, table, torch.tensor(lens, dtype=torch.int32).cuda(),
                                        scale=scale, window=window, workspace=ws)
    assert m.get_error(ws) == 0
    sc = D ** -0.5 if scale is None else scale
    got_lse = f64(lse)
    for b, n in enumerate(lens):
        ref, rlse, mag = ob.attention(f64(q[b]), ks[b] * float(np.float32(scales[0])),
                                      vs[b] * float(np.float32(scales[1])), n, sc, window)
        close(out[b], ref, mag, 2.0 ** -14 if dtype == torch.bfloat16 else 2.0 ** -10, f"b={b} len={n}")
        if n == 0:
            assert np.all(got_lse[b] == -np.inf) and not f64(out[b]).any()
        else:
            assert np.all(np.abs(got_lse[b] - rlse) <= 2.0 ** -22 * np.abs(rlse) + 4e-5)
    again, _ = m.paged_decode_attention(q.cuda(), cache, table, torch.tensor(lens, dtype=torch.int32).cuda(),
                                        scale=scale, window=window)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    return out


EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0, 255, 257, 700]


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 24, 64])
def test_lengths_around_tiles_and_pages(dtype, D, page):
    check(EDGES, page, 8, 2, D, dtype, D + page, scales=(0.5, 0.25) if dtype == F8 else (1.0, 1.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (7, 7), (10, 2), (16, 1), (27, 3), (40, 2), (64, 1)])
def test_head_layouts(dtype, Hq, Hkv):
    check([33, 0, 290], 16, Hq, Hkv, 128, dtype, Hq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("page", [1, 7, 100, 4096])
def test_page_sizes_and_head_major_pages(dtype, page):
    check([1, 50, 999], page, 4, 2, 64, dtype, page, order="head")


@pytest.mark.parametrize("window", [1, 16, 100, 5000])
@pytest.mark.parametrize("D", [64, 256])
def test_windows(window, D):
    check([0, 1, 99, 100, 101, 1300], 16, 4, 1, D, torch.bfloat16, window, window=window)
    check([0, 1, 99, 100, 101, 1300], 32, 16, 1, D, F8, window, window=window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
def test_split_over_the_length(dtype):
    check([20011], 16, 4, 1, 128, dtype, 1)          # one segment over every block
    check([9000, 3, 0, 4500], 64, 16, 2, 128, dtype, 2)


def test_many_short_sequences():
    rng = np.random.default_rng(3)
    check([int(n) for n in rng.integers(0, 40, 700)], 16, 2, 2, 64, torch.bfloat16, 4)


@pytest.mark.parametrize("D,dtype,Hq,Hkv,window", [
    (128, torch.bfloat16, 32, 8, 0), (128, F8, 64, 8, 0), (128, F8, 4, 2, 0), (128, torch.bfloat16, 6, 6, 777),
    (128, F8, 9, 3, 0), (64, torch.bfloat16, 16, 4, 0), (64, F8, 16, 8, 0), (64, F8, 44, 4, 1501),
    (256, torch.bfloat16, 8, 4, 0), (256, F8, 34, 2, 0), (128, torch.bfloat16, 80, 4, 0)])
def test_several_key_heads_of_a_block(D, dtype, Hq, Hkv, window):
    # work enough for long runs on every block; sequences that end and begin inside them
    unit = 256 if D == 64 and dtype == F8 else 128
    segments = Hkv * -(-Hq // Hkv // 16)
    keys = 1900 * unit // segments
    lens = [int(keys * x) + 1 for x in (0.4, 0.13, 0.2, 0.17, 0.1)] + [0, 1, 130]
    if window:
        lens = [n + 3 * window // 2 for n in lens] + [window + 5] * (keys // window)
    check(lens, 48, Hq, Hkv, D, dtype, D + Hq, window=window)


def test_large_scores_do_not_overflow():
    check([40, 300], 16, 4, 2, 64, torch.bfloat16, 5, scale=0.0)
    m = ftmoe()
    q = torch.full((1, 2, 64), 3e4, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((20, 16, 1, 64), dtype=torch.bfloat16, device="cuda")
    k[3, 5] = 3e4                                     # one score of 5.8e10, the others 0
    v = torch.randn((20, 16, 1, 64), device="cuda").bfloat16()
    table = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    out, lse = m.paged_decode_attention(q, m.PagedKVCache(k, v), table,
                                        torch.tensor([320], dtype=torch.int32, device="cuda"), scale=1.0)
    assert torch.equal(out[0, 0], v[3, 5, 0]) and torch.isfinite(lse).all()
    # every score -inf: no weight at all
    k.fill_(float("-inf"))
    q.fill_(1.0)
    out, lse = m.paged_decode_attention(q, m.PagedKVCache(k, v), table,
                                        torch.tensor([320], dtype=torch.int32, device="cuda"))
    assert not out.any() and torch.isneginf(lse).all()


def test_strided_queries_side_stream_and_graph():
    m = ftmoe()
    rng = np.random.default_rng(8)
    lens = [70, 300]
    kc, vc, table, ks, vs = paged(rng, lens, 16, 2, 128, torch.bfloat16)
    wide = bf16(rng.standard_normal((2, 12, 128))).cuda()
    q = wide[:, 3:11]
    cache, n = m.PagedKVCache(kc, vc), torch.tensor(lens, dtype=torch.int32).cuda()
    want, _ = m.paged_decode_attention(q.contiguous(), cache, table, n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = m.paged_decode_attention(q, cache, table, n)
    s.synchronize()
    assert torch.equal(got, want)
    out, lse = torch.empty_like(want), torch.empty((2, 8), device="cuda")
    ws = m.default_workspace  # the default workspace exists: nothing is allocated in the capture
    assert ws is not None
    graph = torch.cuda.CUDAGraph()
    work = torch.zeros(m.paged_attention_workspace_bytes(2, 128) + 256, dtype=torch.uint8, device="cuda")
    work = work[(-work.data_ptr()) % 256:]
    with torch.cuda.graph(graph):
        m.paged_decode_attention(q, cache, table, n, out=out, lse=lse, workspace=work)
    n.copy_(torch.tensor([64, 1], dtype=torch.int32))     # other lengths: the same graph
    graph.replay()
    torch.cuda.synchronize()
    ref, _, mag = ob.attention(f64(q[1]), ks[1], vs[1], 1, 128 ** -0.5)
    close(out[1], ref, mag, 2.0 ** -14)


def test_bad_pages_are_flagged_and_not_followed():
    m = ftmoe()
    rng = np.random.default_rng(9)
    kc, vc, table, ks, vs = paged(rng, [40, 40], 16, 1, 64, torch.bfloat16)
    table[0, 1] = kc.shape[0]
    q = bf16(rng.standard_normal((2, 4, 64))).cuda()
    n = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    ws = torch.zeros(m.paged_attention_workspace_bytes(2, 64) + 256, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:]
    out, _ = m.paged_decode_attention(q, m.PagedKVCache(kc, vc), table, n, workspace=ws)
    assert m.get_error(ws) == 6 and m.get_error(ws) == 0
    ref, _, mag = ob.attention(f64(q[1]), ks[1], vs[1], 40, 0.125)
    close(out[1], ref, mag, 2.0 ** -14)                    # the other sequence is as ever
    table[0, 1] = 0
    n[1] = 48                                              # the table's three pages, then lengths past them
    kc.nan_to_num_()
    vc.nan_to_num_()
    want, _ = m.paged_decode_attention(q, m.PagedKVCache(kc, vc), table, n, workspace=ws)
    assert m.get_error(ws) == 0
    for past in (49, 1 << 20, (1 << 31) - 1):
        n[1] = past
        out, _ = m.paged_decode_attention(q, m.PagedKVCache(kc, vc), table, n, workspace=ws)
        assert m.get_error(ws) == 6 and torch.equal(out, want)
    out, lse = m.paged_decode_attention(q, m.PagedKVCache(kc, vc), table[:, :0].contiguous(), n, workspace=ws)
    assert m.get_error(ws) == 6 and not out.any() and torch.isneginf(lse).all()


def test_offsets_past_32_bits():
    """Pages beyond 2^32 bytes (and 2^31 elements) of the pool."""
    m = ftmoe()
    rng = np.random.default_rng(10)
    P, page, D = 36000, 64, 256                           # 2^31 elements at page 32768 + ...
    kc = torch.empty((P, page, 4, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((P, page, 4, D), dtype=torch.bfloat16, device="cuda")
    cache = m.PagedKVCache(kc, vc)
    pages = [35999, 33333, 2]
    table = torch.tensor([pages], dtype=torch.int32, device="cuda")
    k, v = (bf16(rng.standard_normal((150, 4, D))) for _ in range(2))
    pos = torch.arange(150, dtype=torch.int32, device="cuda")
    m.kv_append(k.cuda(), v.cuda(), cache, table, pos,
                seq_ids=torch.zeros(150, dtype=torch.int32, device="cuda"))
    assert torch.equal(kc[35999].cpu(), k[:64]) and torch.equal(vc[33333].cpu(), v[64:128])
    q = bf16(rng.standard_normal((1, 8, D)))
    out, _ = m.paged_decode_attention(q.cuda(), cache, table, torch.tensor([150], dtype=torch.int32).cuda())
    ref, _, mag = ob.attention(f64(q[0]), f64(k), f64(v), 150, D ** -0.5)
    close(out[0], ref, mag, 2.0 ** -14)


# ---------------------------------------------------------------- append
def rope_table(rows, R):
    ang = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def rotate32(v, rope, pos):
    """float32 arithmetic, every product and sum rounded."""
    v = v.float().numpy().copy()
    if rope is None:
        return v
    h = rope.shape[1] // 2
    c, s = rope[pos, None, :h], rope[pos, None, h:]
    a, b = v[..., :h].copy(), v[..., h:2 * h].copy()
    v[..., :h], v[..., h:2 * h] = a * c - b * s, b * c + a * s
    return v


def as_stored(v, dtype, scale):
    v = torch.from_numpy(v)
    if dtype == torch.bfloat16:
        return v.bfloat16()
    return (v * float(np.float32(1) / np.float32(scale))).clamp(-448, 448).to(F8)


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("D,R,Hq,Hkv,page", [(64, 64, 4, 2, 16), (128, 64, 5, 1, 24), (256, 256, 3, 3, 7),
                                             (128, 0, 8, 2, 1), (64, 16, 0, 1, 64)])
@pytest.mark.parametrize("order", ["slot", "head"])
def test_append_is_exact(dtype, D, R, Hq, Hkv, page, order):
    m = ftmoe()
    rng = np.random.default_rng(D + R)
    T, B, P, width = 37, 5, 40, 8
    # tokens of five sequences at places that differ, two of them padding
    seq = rng.integers(0, B, T)
    pos = np.array([int(np.sum(seq[:t] == seq[t])) + min(3, page * width - T) for t in range(T)])
    P = max(P, B * width)
    table = rng.permutation(P)[:B * width].reshape(B, width).astype(np.int32)
    fits = pos // page < width
    pos[~fits] = -1
    pos[[4, 20]] = -1
    rope = rope_table(64, R) if R else None
    wide = bf16(3 * rng.standard_normal((T, Hq + 2 * Hkv, D)))
    wide[0, Hq] = 1e5                                    # saturates E4M3
    q, k, v = wide[:, :Hq], wide[:, Hq:Hq + Hkv], wide[:, Hq + Hkv:]
    shape = (P, page, Hkv, D) if order == "slot" else (P, Hkv, page, D)
    scales = (0.3, 0.02) if dtype == F8 else (1.0, 1.0)
    pools = [torch.zeros(shape, dtype=torch.uint8).to(dtype).cuda() for _ in range(2)]
    view = [p if order == "slot" else p.permute(0, 2, 1, 3) for p in pools]
    cache = m.PagedKVCache(*view, *scales)
    want = [p.cpu().clone() for p in view]
    kr, qr = rotate32(k, rope, np.maximum(pos, 0)), rotate32(q, rope, np.maximum(pos, 0))
    ks, vs = as_stored(kr, dtype, scales[0]), as_stored(v.float().numpy(), dtype, scales[1])
    for t in range(T):
        if pos[t] >= 0:
            p, s = table[seq[t], pos[t] // page], pos[t] % page
            raw = torch.uint8 if dtype == F8 else torch.int16
            want[0].view(raw)[p, s] = ks[t].view(raw)
            want[1].view(raw)[p, s] = vs[t].view(raw)
    wd = wide.cuda()
    ws = torch.zeros(1024 + 256, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:1024]
    got = m.kv_append(wd[:, Hq:Hq + Hkv], wd[:, Hq + Hkv:], cache, torch.from_numpy(table).cuda(),
                      torch.from_numpy(pos.astype(np.int32)).cuda(),
                      seq_ids=torch.from_numpy(seq.astype(np.int32)).cuda(),
                      q=wd[:, :Hq] if Hq else None, rope=None if rope is None else torch.from_numpy(rope).cuda(),
                      workspace=ws)
    assert m.get_error(ws) == 0
    assert np.array_equal(bits(view[0]), bits(want[0])) and np.array_equal(bits(view[1]), bits(want[1]))
    if Hq:
        ref = torch.from_numpy(qr).bfloat16()
        ref[torch.from_numpy(pos < 0)] = 0
        assert np.array_equal(bits(got), bits(ref))
    else:
        assert got is None


def test_append_flags_what_lies_outside():
    m = ftmoe()
    cache = m.PagedKVCache(*(torch.zeros((4, 16, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32, device="cuda")
    one = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    rope = torch.zeros((40, 64), dtype=torch.float32, device="cuda")
    ws = torch.zeros(1280, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:1024]
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")
    for seq, pos, bad in ((0, 3, False), (1, 17, True), (0, 32, True), (2, 0, True), (-1, 0, True),
                          (0, 40, True), (0, -1, False)):
        m.kv_append(one, one, cache, table, i32(pos), seq_ids=i32(seq), rope=rope, workspace=ws)
        assert m.get_error(ws) == (6 if bad else 0), (seq, pos)
    assert int(cache.v.sum()) == 64                       # only the first one was stored
    assert m.kv_append(one[:0], one[:0], cache, table, i32(0)[:0]) is None


def test_a_step_reads_what_the_step_appended():
    """Append, then attend, token by token: as one attention over the whole sequence."""
    m = ftmoe()
    rng = np.random.default_rng(12)
    n, Hq, Hkv, D = 35, 4, 2, 64
    rope = rope_table(64, D)
    x = bf16(rng.standard_normal((n, Hq + 2 * Hkv, D)))
    cache = m.PagedKVCache(*(torch.full((6, 16, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                             for _ in range(2)))
    table = torch.tensor([[4, 0, 3]], dtype=torch.int32, device="cuda")
    xd, rd = x.cuda(), torch.from_numpy(rope).cuda()
    ks, vs = [], []
    for t in range(n):
        at = torch.tensor([t], dtype=torch.int32, device="cuda")
        q = m.kv_append(xd[t:t + 1, Hq:Hq + Hkv], xd[t:t + 1, Hq + Hkv:], cache, table, at,
                        q=xd[t:t + 1, :Hq], rope=rd)
        out, _ = m.paged_decode_attention(q, cache, table, at + 1)
        ks.append(f64(torch.from_numpy(rotate32(x[t:t + 1, Hq:Hq + Hkv], rope, [t])).bfloat16())[0])
        vs.append(f64(x[t, Hq + Hkv:]))
        ref, _, mag = ob.attention(f64(q[0]), np.array(ks), np.array(vs), t + 1, D ** -0.5)
        close(out[0], ref, mag, 2.0 ** -14, f"token {t}")
