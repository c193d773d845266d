"""Calls that are given no workspace: from two threads on one stream, captured and then followed by a larger
call, and captured twice and replayed side by side."""
import threading

import numpy as np
import pytest
import torch

from synth import TINY, make_layer
from tests.block_util import bf16
from tests.layer_util import bf16_tensor, experts_to_device, ftmoe
from tests.test_gpu_block_linear import matrix, on_gpu

pytestmark = pytest.mark.gpu


def calls_of(m, seed, D=128, T=40, H=1032):
    """Functions of several launches each, and their outputs as tuples of tensors."""
    rng = np.random.default_rng(seed)
    on = lambda *s: bf16(rng.standard_normal(s)).cuda()  # noqa: E731
    n = 9000
    cache = m.PagedKVCache(on(n // 64 + 1, 64, 2, D), on(n // 64 + 1, 64, 2, D))
    table = torch.from_numpy(rng.permutation(n // 64 + 1).astype(np.int32))[None].cuda()
    q, length = on(1, 8, D), torch.tensor([n - 3], dtype=torch.int32, device="cuda")
    lin, x = on_gpu(m, *matrix(rng, 12000, 512)), on(T, 512)
    y, r, dr, dx, w = on(300, H), on(300, H), on(300, H), on(300, H), on(H)
    layer = make_layer(TINY)
    experts, shared = experts_to_device(layer)
    xl, logits = bf16_tensor(layer.x), torch.from_numpy(layer.logits).cuda()
    return [lambda: tuple(m.paged_decode_attention(q, cache, table, length)),
            lambda: (m.nvfp4_linear(x, lin),),
            lambda: tuple(t for t in m.residual_norm_backward(y, r, dr, dx, w_post=w, w_pre=w, gate=w)),
            lambda: (m.decode_routed(xl, logits, TINY.k, experts, shared),)]


def same(a, b):
    return all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))


def test_two_threads_on_one_stream():
    m = ftmoe()
    work = [calls_of(m, 1), calls_of(m, 2)]
    want = [[f() for f in calls] for calls in work]
    torch.cuda.synchronize()
    bad, together = [], threading.Barrier(2)

    def run(i):
        for f, w in zip(work[i], want[i]):
            together.wait()
            got = [f() for _ in range(150)]
            torch.cuda.synchronize()
            bad.extend(i for g in got if not same(g, w))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_a_captured_call_outlives_a_larger_one():
    m = ftmoe()
    small, large = calls_of(m, 3, D=64, T=20, H=520), calls_of(m, 4, D=256, T=64, H=8192)
    want = [f() for f in small]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for f, g, w in zip(small, large, want):
        with torch.cuda.stream(s):
            f()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = f()
        with torch.cuda.stream(s):
            g()                                  # needs more: the stream's own workspace is replaced
            others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
            graph.replay()
        s.synchronize()
        assert same(out, w)
        assert all(bool((t == 7).all()) for t in others)


def test_two_graphs_side_by_side():
    m = ftmoe()
    work = [calls_of(m, 5), calls_of(m, 6)]
    want = [[f() for f in calls] for calls in work]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for calls in work:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append([f() for f in calls])
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for order in ((0, 1), (1, 0)) * 5:
        for i in order:
            with torch.cuda.stream(streams[i]):
                for _ in range(4):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert all(same(a, b) for a, b in zip(out, w))


def test_the_workspace_belongs_to_the_stream_it_is_asked_for():
    m = ftmoe()
    layer = make_layer(TINY)
    experts, _ = experts_to_device(layer)
    s = torch.cuda.Stream()
    ws = m.default_workspace(TINY.T, TINY.k, experts, False, stream=s)
    assert ws is m.default_workspace(TINY.T, TINY.k, experts, False, stream=s)
    home = [seg["stream"] for seg in torch.cuda.memory_snapshot()
            if seg["address"] <= ws.data_ptr() < seg["address"] + seg["total_size"]]
    assert home == [s.cuda_stream]


def test_flags_of_calls_without_a_workspace_can_be_read():
    m = ftmoe()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = m.PagedKVCache(*(torch.zeros((4, 16, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    one = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    table = i32([[0, 9]])

    def append(pos):
        m.kv_append(one, one, cache, table, i32([pos]))

    def attend(n):
        m.paged_decode_attention(one, cache, table, i32([n]))

    m.get_error()                                     # what earlier tests of this thread left
    for f, arg, bad in ((append, 3, 0), (append, 17, 6), (append, 40, 6), (append, -1, 0), (attend, 4, 0),
                        (attend, 20, 6), (attend, 33, 6)):
        f(arg)
        assert m.get_error() == bad and m.get_error() == 0, (f, arg)
    append(17)                                        # another thread or stream has its own
    s, seen = torch.cuda.Stream(), []
    t = threading.Thread(target=lambda: seen.extend([m.get_error(), m.get_error(stream=s)]))
    t.start()
    t.join()
    assert seen == [0, 0] and m.get_error(stream=s) == 0
    with torch.cuda.stream(s):
        append(3)
        append(17)
        attend(4)                                     # a larger workspace takes the flags along
        assert m.get_error() == 6
    append(17)
    s.synchronize()
    assert m.get_error(stream=s) == 0 and m.get_error() == 6
