"""The decode block's calls together: steps of examples/decode_block.py against the float64 oracles, with
bf16 rounding where the calls' outputs are bf16, and the captured step against the eager one.

Tolerance: a value that float32 moves over a bf16 tie differs by 2^-8 of itself; about ten roundings lie
between a step's input and its logits: rel_fro <= 2e-2.
"""
import numpy as np
import pytest
import torch

from examples import decode_block as ex
from oracle import block as ob
from oracle import moe as om
from synth import LayerSpec, make_layer
from tests.block_util import bf16, f64
from tests.layer_util import experts_to_device, ftmoe
from tests.test_gpu_block_linear import matrix, on_gpu

pytestmark = pytest.mark.gpu
B, H, HQ, HKV, D, E, K, I, PAGE, ROOM = 3, 256, 4, 2, 64, 8, 2, 128, 16, 64


def r16(a):
    return f64(bf16(a))


def build(rng, layers):
    m = ftmoe()
    small = lambda n, k: tuple(a * s for a, s in zip(matrix(rng, n, k), (1, 1, 0.3)))  # noqa: E731
    vec = lambda n, s=0.1: f64(bf16(1 + s * rng.standard_normal(n)))  # noqa: E731
    dev = lambda a: bf16(a).cuda()  # noqa: E731
    host, on_dev, caches = [], [], []
    width = ROOM // PAGE
    for i in range(layers):
        moe = make_layer(LayerSpec(f"s{i}", seed=20 + i, T=1, E=E, k=K, H=H, I=I, w_sigma=0.1))
        h = dict(qkv=small((HQ + 2 * HKV) * D, H), o=small(H, HQ * D), moe=moe,
                 router=f64(bf16(0.2 * rng.standard_normal((E, H)))), attn_post=vec(H), moe_pre=vec(H),
                 moe_post=vec(H), moe_gate=vec(H, 0.3), next_pre=vec(H))
        host.append(h)
        f32 = lambda w: (w[0], w[1], w[2].astype(np.float32))  # noqa: E731
        experts, _ = experts_to_device(moe)
        on_dev.append(ex.Layer(on_gpu(m, *f32(h["qkv"])), on_gpu(m, *f32(h["o"])), dev(h["router"]), experts,
                               dev(h["attn_post"]), dev(h["moe_pre"]), dev(h["moe_post"]),
                               dev(h["moe_gate"]), dev(h["next_pre"]), K))
        pool = lambda: torch.full((B * width, PAGE, HKV, D), float("nan"), dtype=torch.bfloat16,  # noqa: E731
                                  device="cuda")
        caches.append(m.PagedKVCache(pool(), pool()))
    table = torch.from_numpy(rng.permutation(B * width).astype(np.int32).reshape(B, width)).cuda()
    rope = ex.rotary_table(ROOM, D, "cuda")
    first, logits = vec(H), small(77, H)
    step = ex.DecodeStep(on_dev, caches, table, rope, HQ, dev(first),
                         on_gpu(m, logits[0], logits[1], logits[2].astype(np.float32)), B, scale=0.5)
    return step, host, first, logits, rope.cpu().numpy()


def reference(host, first, logits, rope, x_in, t, keys, values):
    """One step in float64; keys/values [layer][sequence] grow by the step's."""
    res, x = ob.residual_norm(x_in, None, None, first, None, 1.0, ex.EPS)
    x = r16(x)
    for i, h in enumerate(host):
        qkv = r16(ob.linear(x, *h["qkv"])[0]).reshape(B, HQ + 2 * HKV, D)
        pos = [t] * B
        q = r16(ob.rotate(qkv[:, :HQ], rope, pos))
        k = r16(ob.rotate(qkv[:, HQ:HQ + HKV], rope, pos))
        a = np.zeros((B, HQ, D))
        for b in range(B):
            keys[i][b].append(k[b])
            values[i][b].append(qkv[b, HQ + HKV:])
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


def test_steps_against_the_oracles_and_a_graph():
    rng = np.random.default_rng(31)
    step, host, first, logits, rope = build(rng, 2)
    keys = [[[] for _ in range(B)] for _ in host]
    values = [[[] for _ in range(B)] for _ in host]
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
    assert step.positions.tolist() == [20] * B


def test_what_a_call_makes_belongs_to_the_stream_it_is_given():
    m = ftmoe()
    rng = np.random.default_rng(40)
    on = lambda *shape: bf16(rng.standard_normal(shape)).cuda()  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    lin, x = on_gpu(m, *matrix(rng, 300, 512)), on(20, 512)
    cache = m.PagedKVCache(on(8, 16, 2, 64), on(8, 16, 2, 64))
    table, q, k = i32([[0, 1, 2], [3, 4, 5]]), on(2, 4, 64), on(2, 2, 64)
    y, w = on(20, 512), on(512)

    def calls(stream):
        made = [m.nvfp4_linear(x, lin, stream=stream),
                m.kv_append(k, k, cache, table, i32([3, 40]), q=q, stream=stream),
                *m.paged_decode_attention(q, cache, table, i32([20, 41]), stream=stream),
                *m.residual_norm(y, x, w_post=w, w_pre=w, gate=w, stream=stream)]
        grads = m.residual_norm_backward(y, x, y, x, w_post=w, w_pre=w, gate=w, stream=stream)
        return made + list(grads)

    want = calls(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = calls(s)
    s.synchronize()
    home = {a: seg["stream"] for seg in torch.cuda.memory_snapshot()
            for a in range(seg["address"], seg["address"] + seg["total_size"], 512)}
    for a, b in zip(want, got):
        assert torch.equal(a, b)
        assert home[b.data_ptr()] == s.cuda_stream != home[a.data_ptr()]
