"""The calls on an NVFP4 cache together: steps of examples/decode_block.py with its caches in four bits against
the float64 oracles, eager and captured; append, attention and read-back on streams of their own.

Tolerance of the steps: that of the bf16 caches (about ten bf16 roundings: rel_fro <= 2e-2). A key or value that
float32 arithmetic moves over a tie between two codes, rare, changes one element of a cached row by a step.
"""
import numpy as np
import pytest
import torch

from examples import decode_block as ex
from oracle import block as ob
from oracle import moe as om
from tests.block_util import bf16, close, f64
from tests.layer_util import ftmoe
from tests.nvfp4_cache_util import paged
from tests.test_gpu_block_step import B, D, HKV, HQ, H, K, PAGE, ROOM, build, r16

pytestmark = pytest.mark.gpu
G = ex.KV_GSCALE


def four(m, order="slot"):
    """A cache whose every slot reads as NaN."""
    P = B * (ROOM // PAGE)
    shape = lambda w: (P, PAGE, HKV, w) if order == "slot" else (P, HKV, PAGE, w)  # noqa: E731
    pool = lambda w, byte: torch.full(shape(w), byte, dtype=torch.uint8, device="cuda")  # noqa: E731
    t = [pool(D // 2, 0xA5), pool(D // 2, 0xA5), pool(D // 16, 0x7F), pool(D // 16, 0x7F)]
    return m.NvFP4KVCache(*(x if order == "slot" else x.permute(0, 2, 1, 3) for x in t), G, G)


def stored(x):
    return ob.nvfp4_values(*ob.nvfp4_rows(np.asarray(x, np.float32), G), 1.0).astype(np.float64) * float(np.float32(G))


def reference(host, first, logits, rope, x_in, t, keys, values):
    """One step in float64; keys/values [layer][sequence] grow by the step's, as the cache holds them."""
    res, x = ob.residual_norm(x_in, None, None, first, None, 1.0, ex.EPS)
    x = r16(x)
    for i, h in enumerate(host):
        qkv = r16(ob.linear(x, *h["qkv"])[0]).reshape(B, HQ + 2 * HKV, D)
        q = r16(ob.rotate(qkv[:, :HQ], rope, [t] * B))
        k = stored(ob.rotate(qkv[:, HQ:HQ + HKV], rope, [t] * B))
        v = stored(qkv[:, HQ + HKV:])
        a = np.zeros((B, HQ, D))
        for b in range(B):
            keys[i][b].append(k[b])
            values[i][b].append(v[b])
            a[b] = ob.attention(q[b], np.array(keys[i][b]), np.array(values[i][b]), t + 1, D ** -0.5)[0]
        y = r16(ob.linear(r16(a.reshape(B, -1)), *h["o"])[0])
        res, x = ob.residual_norm(y, res, h["attn_post"], h["moe_pre"], None, 0.5, ex.EPS)
        x = r16(x)
        bits = bf16(x).view(torch.int16).numpy().view(np.uint16)
        scores = (x @ h["router"].T).astype(np.float32)
        y = r16(om.moe_layer(bits, scores, K, h["moe"])[0])
        res, x = ob.residual_norm(y, res, h["moe_post"], h["next_pre"], h["moe_gate"], 0.5, ex.EPS)
        x = r16(x)
    return ob.linear(x, *logits)[0]


@pytest.mark.parametrize("order", ["slot", "head"])
def test_steps_against_the_oracles_and_a_graph(order):
    m = ftmoe()
    rng = np.random.default_rng(31)
    step, host, first, logits, rope = build(rng, 1)
    step.caches = [four(m, order) for _ in host]
    keys, values = ([[[] for _ in range(B)] for _ in host] for _ in range(2))
    xs = [bf16(rng.standard_normal((B, H))) for _ in range(20)]
    x_in = xs[0].cuda()
    graph = None
    for t, x in enumerate(xs):
        x_in.copy_(x)
        if t < 2:
            got = step.step(x_in)
        else:
            if graph is None:        # from the third step on the captured step runs
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    got = step.step(x_in)
            graph.replay()
        ref = reference(host, first, logits, rope, f64(x), t, keys, values)
        off = np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)
        assert off <= 2e-2, (t, off)
    assert m.get_error(step.workspace) == 0
    # the first layer's cache read back: what the oracle stored, but for codes on the edge of another
    n = len(xs)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B)
    seq = torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(n)
    k, v = m.kv_gather(step.caches[0], step.table, pos, seq_ids=seq)
    for got, want in ((k, keys[0]), (v, values[0])):
        got, want = f64(got).reshape(B, n, HKV, D), np.array(want)
        far = np.abs(got - want) > 2.0 ** -8 * np.abs(want) + 1e-30
        assert far.mean() <= 0.02, far.mean()


def test_the_example_runs_with_a_cache_of_four_bits():
    torch.manual_seed(0)
    model = ex.random_model(2, 1, torch.device("cuda"), H=256, Hq=4, Hkv=2, D=64, E=8, k=2, I=128, cache="nvfp4")
    x = torch.randn(2, 256, device="cuda").bfloat16()
    for _ in range(3):
        assert torch.isfinite(model.step(x)).all()
    assert ftmoe().get_error(model.workspace) == 0


def test_strided_queries_side_stream_and_graph():
    m = ftmoe()
    rng = np.random.default_rng(8)
    lens = [70, 300]
    cache, table, ks, vs = paged(rng, lens, 16, 2, 128)
    wide = bf16(rng.standard_normal((2, 12, 128))).cuda()
    q = wide[:, 3:11]
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    want, _ = m.paged_decode_attention(q.contiguous(), cache, table, n)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, lse = m.paged_decode_attention(q, cache, table, n, stream=s)
    pos, seq = torch.tensor([5, 299], dtype=torch.int32).cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    k, v = m.kv_gather(cache, table, pos, seq_ids=seq, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and m.get_error(stream=s) == 0
    close(k, np.stack([ks[0][5], ks[1][299]]), np.zeros((2, 2, 128)), 0)
    close(v, np.stack([vs[0][5], vs[1][299]]), np.zeros((2, 2, 128)), 0)
    out, lse = torch.empty_like(want), torch.empty((2, 8), device="cuda")
    work = torch.zeros(m.paged_attention_workspace_bytes(2, 128) + 256, dtype=torch.uint8, device="cuda")
    work = work[(-work.data_ptr()) % 256:]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.paged_decode_attention(q, cache, table, n, out=out, lse=lse, workspace=work)
    n.copy_(torch.tensor([64, 1], dtype=torch.int32))     # other lengths: the same graph
    graph.replay()
    torch.cuda.synchronize()
    for b, length in ((0, 64), (1, 1)):
        ref, _, mag = ob.attention(f64(q[b]), ks[b], vs[b], length, 128 ** -0.5)
        close(out[b], ref, mag, 2.0 ** -10)


def test_most_sequences_that_a_call_takes():
    """4096 of them, with the widest heads in the largest groups: the running sums of units in shared memory."""
    m = ftmoe()
    rng = np.random.default_rng(5)
    for D2, Hq in ((256, 16), (256, 8), (128, 16), (128, 8), (64, 16), (64, 4)):
        lens = [0] * 4096
        for i in (0, 1, 77, 2048, 4000, 4095):
            lens[i] = int(rng.integers(1, 90))
        cache, table, ks, vs = paged(rng, lens, 16, 1, D2)
        q = bf16(rng.standard_normal((4096, Hq, D2)))
        out, lse = m.paged_decode_attention(q.cuda(), cache, table, torch.tensor(lens, dtype=torch.int32).cuda())
        for i in (0, 1, 77, 2048, 4000, 4095):
            ref, _, mag = ob.attention(f64(q[i]), ks[i], vs[i], lens[i], D2 ** -0.5)
            close(out[i], ref, mag, 2.0 ** -10, (D2, Hq, i))
        some = torch.tensor(lens).cuda() > 0
        assert not out[~some].any() and torch.isneginf(lse[~some]).all()


def test_keys_and_values_that_lie_otherwise():
    """Keys slot by slot, values head by head, in pools of other strides: offsets of their own."""
    m = ftmoe()
    rng = np.random.default_rng(13)
    Hkv, D2, page, P, n = 3, 128, 16, 9, 131
    x = bf16(rng.standard_normal((n, 2 * Hkv, D2)))
    pool = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    kc = pool(P, page, Hkv + 1, D2)[:, :, 1:, :D2 // 2]
    vc, vs = pool(P, Hkv, page, D2 // 2).permute(0, 2, 1, 3), pool(P, Hkv, page + 3, D2 // 16)[:, :, 3:].permute(0, 2, 1, 3)
    cache = m.NvFP4KVCache(kc, vc, pool(P, page, Hkv, 2 * (D2 // 16))[..., D2 // 16:], vs, 0.0021, 0.0017)
    table = torch.from_numpy(rng.permutation(P).astype(np.int32)[None]).cuda()
    pos, seq = torch.arange(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    xd = x.cuda()
    m.kv_append(xd[:, :Hkv], xd[:, Hkv:], cache, table, pos, seq_ids=seq)
    want = [ob.nvfp4_values(*ob.nvfp4_rows(h.float().numpy(), g), 1.0).astype(np.float64) * float(np.float32(g))
            for h, g in ((x[:, :Hkv], 0.0021), (x[:, Hkv:], 0.0017))]
    for got, w in zip(m.kv_gather(cache, table, pos, seq_ids=seq), want):
        close(got, w, np.zeros(w.shape), 0)
    q = bf16(rng.standard_normal((1, 6, D2)))
    out, _ = m.paged_decode_attention(q.cuda(), cache, table, torch.tensor([n], dtype=torch.int32).cuda())
    ref, _, mag = ob.attention(f64(q[0]), *want, n, D2 ** -0.5)
    close(out[0], ref, mag, 2.0 ** -10)


def test_a_scale_below_zero_and_large_scores():
    m = ftmoe()
    rng = np.random.default_rng(21)
    cache, table, ks, vs = paged(rng, [200], 16, 2, 128)
    q = bf16(rng.standard_normal((1, 8, 128)))
    n = torch.tensor([200], dtype=torch.int32).cuda()
    for scale in (-0.1, 3.0, 1e30):
        out, lse = m.paged_decode_attention(q.cuda(), cache, table, n, scale=scale)
        ref, rlse, mag = ob.attention(f64(q[0]), ks[0], vs[0], 200, scale)
        assert np.all(np.abs(f64(lse)[0] - rlse) <= 2.0 ** -18 * np.abs(rlse) + 4e-5)
        if scale != 3.0:                                  # scores of hundreds: float32 moves them by more than a weight's step
            close(out[0], ref, mag, 2.0 ** -10, scale)


def test_scores_whose_steps_are_larger_than_a_weights_range():
    """Scores of 2^27 in units of log 2, where neighbouring float32 lie 16 apart: a weight is 1 or at least 2^16 times
    another's, and no sum may overflow on the way from one to the other."""
    m = ftmoe()
    for ahead in (1, 2, 3):
        n, D2 = 96, 64
        codes = np.zeros((6, 16, 1, D2 // 2), np.uint8)
        scales = np.full((6, 16, 1, D2 // 16), 0x38, np.uint8)   # 1
        scales[..., 0] = 0x70                                    # 128
        codes[..., 0] = 6                                        # 4 * 128 = 512 in element 0
        late = codes.reshape(n, D2 // 2)
        late[40:80, 8] = 2 * 1                                   # 1 in element 16 of keys 40 to 79
        late[80:, 8] = (0, 2, 4, 5)[ahead]                       # 1, 2 or 3 in that of keys 80 on
        vals = np.random.default_rng(ahead).integers(0, 256, codes.shape).astype(np.uint8)
        q = torch.zeros((1, 1, D2))
        q[0, 0, 0], q[0, 0, 16] = 2.0 ** 14, 1.0                 # products of 2^23 and 1, 2 or 3
        cache = m.NvFP4KVCache(*(torch.from_numpy(a).cuda() for a in (codes, vals, scales, np.full_like(scales, 0x38))))
        table = torch.arange(6, dtype=torch.int32)[None].cuda()
        out, lse = m.paged_decode_attention(q.bfloat16().cuda(), cache, table, torch.tensor([n], dtype=torch.int32).cuda(),
                                            scale=16 * float(np.log(2)))
        vs = ob.nvfp4_values(vals, np.full_like(scales, 0x38), 1.0).reshape(n, 1, D2).astype(np.float64)
        # the keys with the largest product, all alike: the others' weights are 2^-16 of theirs at most
        best = slice(40, n) if ahead == 1 else slice(80, n)
        want, mag = vs[best, 0].mean(0), np.abs(vs[best, 0]).mean(0)
        close(out[0], want[None], np.maximum(mag, 6.0)[None], 2.0 ** -10 + 40 * 2.0 ** -16)
        assert torch.isfinite(lse).all()
