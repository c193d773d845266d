"""The cache append into NVFP4 pages, and with several rotary axes: bit-exact against float32 arithmetic (the
codes of a block with a NaN, which reads as NaN whatever they are, are left out)."""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.block_util import bf16
from tests.layer_util import ftmoe
from tests.nvfp4_cache_util import pool, to_gpu
from tests.test_gpu_block_attention import F8, as_stored, bits, rope_table, rotate32

pytestmark = pytest.mark.gpu
I32 = torch.int32


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def rotate_axes32(v, rope, positions, axis):
    """float32 arithmetic, every product and sum rounded."""
    v = v.float().numpy().copy()
    h = rope.shape[1] // 2
    at = np.asarray(positions)[np.asarray(axis)].T
    c, s = rope[at, np.arange(h)][:, None], rope[at, h + np.arange(h)][:, None]
    a, b = v[..., :h].copy(), v[..., h:2 * h].copy()
    v[..., :h], v[..., h:2 * h] = a * c - b * s, b * c + a * s
    return v


class Case:
    """Tokens of five sequences at places that differ, two of them padding, in a pool that is zero."""

    def __init__(self, D, R, Hq, Hkv, page, order, kind, T=37, seed=0):
        rng = self.rng = np.random.default_rng(D + R + page + seed)
        B, width = 5, -(-T // page) + 1
        self.T, self.order, self.kind = T, order, kind
        self.seq = rng.integers(0, B, T)
        self.pos = np.array([int(np.sum(self.seq[:t] == self.seq[t])) for t in range(T)])
        self.pos[[T // 9, T // 2]] = -1
        P = B * width + 3
        self.table = rng.permutation(P)[:B * width].reshape(B, width).astype(np.int32)
        self.rope = rope_table(max(64, T), R) if R else None
        wide = bf16(3 * rng.standard_normal((T, Hq + 2 * Hkv, D)) * 2.0 ** rng.integers(-20, 3, (T, Hq + 2 * Hkv, 1)))
        wide[0, Hq] = 1e5                                # saturates E4M3 and the block scales
        wide[1, Hq] = 0
        self.wide, self.Hq, self.Hkv, self.D = wide, Hq, Hkv, D
        self.q, self.k, self.v = wide[:, :Hq], wide[:, Hq:Hq + Hkv], wide[:, Hq + Hkv:]
        self.gs = {"nvfp4": (0.0021, 0.37), "e4m3": (0.3, 0.02), "bf16": (1.0, 1.0)}[kind]
        if kind == "nvfp4":
            self.pools = [pool(P, page, Hkv, D, order, False) for _ in range(2)]
        else:
            shape = (P, page, Hkv, D) if order == "slot" else (P, Hkv, page, D)
            z = [torch.zeros(shape, dtype=torch.uint8).to(F8 if kind == "e4m3" else torch.bfloat16) for _ in range(2)]
            self.pools = [[t if order == "slot" else t.permute(0, 2, 1, 3)] for t in z]
        self.page = page

    def run(self, m, turned_k, turned_q, **more):
        """The call, and its results against float32 arithmetic."""
        gpu = [[to_gpu(t, self.order) for t in p] for p in self.pools]
        if self.kind == "nvfp4":
            cache = m.NvFP4KVCache(gpu[0][0], gpu[1][0], gpu[0][1], gpu[1][1], *self.gs)
        else:
            cache = m.PagedKVCache(gpu[0][0], gpu[1][0], *self.gs)
        ws = torch.zeros(1024 + 256, dtype=torch.uint8, device="cuda")
        ws = ws[(-ws.data_ptr()) % 256:][:1024]
        wd = self.wide.cuda()
        Hq, Hkv = self.Hq, self.Hkv
        got = m.kv_append(wd[:, Hq:Hq + Hkv], wd[:, Hq + Hkv:], cache, i32(self.table), i32(self.pos),
                          seq_ids=i32(self.seq), q=wd[:, :Hq] if Hq else None,
                          rope=None if self.rope is None else torch.from_numpy(self.rope).cuda(), workspace=ws, **more)
        assert m.get_error(ws) == 0
        for which, x in enumerate((turned_k, self.v.float().numpy())):
            want = [t.clone() for t in self.pools[which]]
            if self.kind == "nvfp4":
                new = [torch.from_numpy(a) for a in ob.nvfp4_rows(x, self.gs[which])]
            else:
                new = [as_stored(x, F8 if self.kind == "e4m3" else torch.bfloat16, self.gs[which])]
            raw = torch.int16 if self.kind == "bf16" else torch.uint8
            for t in np.flatnonzero(self.pos >= 0):
                p, s = self.table[self.seq[t], self.pos[t] // self.page], self.pos[t] % self.page
                for w, n in zip(want, new):
                    w.view(raw)[p, s] = n[t].view(raw)
            have = [t.cpu() for t in gpu[which]]
            if self.kind == "nvfp4":   # codes under a NaN scale say nothing
                nan = (want[1] == 0x7F).repeat_interleave(8, -1)
                have[0], want[0] = have[0].masked_fill(nan, 0), want[0].masked_fill(nan, 0)
            for h, w in zip(have, want):
                assert np.array_equal(bits(h), bits(w)), "kv"[which]
        if Hq:
            ref = torch.from_numpy(turned_q).bfloat16()
            ref[torch.from_numpy(self.pos < 0)] = 0
            assert np.array_equal(bits(got), bits(ref))
        else:
            assert got is None
        return cache


@pytest.mark.parametrize("D,R,Hq,Hkv,page", [(64, 64, 4, 2, 16), (128, 64, 5, 1, 24), (256, 256, 3, 3, 7),
                                             (128, 0, 8, 2, 1), (64, 32, 0, 1, 64), (128, 128, 32, 8, 16),
                                             (256, 128, 40, 8, 5), (128, 96, 2, 1, 16)])
@pytest.mark.parametrize("order", ["slot", "head"])
def test_append_is_exact(D, R, Hq, Hkv, page, order):
    c = Case(D, R, Hq, Hkv, page, order, "nvfp4")
    at = np.maximum(c.pos, 0)
    c.run(ftmoe(), rotate32(c.k, c.rope, at), rotate32(c.q, c.rope, at))


@pytest.mark.parametrize("R", [0, 64])
def test_nan_and_infinity(R):
    c = Case(64, R, 2, 2, 16, "slot", "nvfp4")
    c.wide[5, 2:, 7] = float("nan")
    c.wide[6, 2:, 9] = float("inf")
    c.wide[7, 2:, 40] = float("-inf")
    c.wide[8, 2:, 3] = 3e38
    c.rope = None if not R else np.concatenate([np.ones((64, 32)), np.zeros((64, 32))], 1).astype(np.float32)
    if R:   # infinity times zero: the partners of infinities turn into NaN by the formula
        c.wide[6, 2:, 9] = c.wide[7, 2:, 40] = 1e30
    at = np.maximum(c.pos, 0)
    with np.errstate(all="ignore"):
        c.run(ftmoe(), rotate32(c.k, c.rope, at), rotate32(c.q, c.rope, at))


def test_one_token_and_none():
    m = ftmoe()
    for T in (1, 2):
        c = Case(128, 128, 3, 1, 16, "slot", "nvfp4", T=max(T, 2))
        c.pos[:] = 5
        c.seq[:] = [0, 1]
        c.run(m, rotate32(c.k, c.rope, c.pos), rotate32(c.q, c.rope, c.pos))
    kc, ks = (t.cuda() for t in pool(2, 16, 1, 64, "slot", False))
    cache = m.NvFP4KVCache(kc, kc.clone(), ks, ks.clone())
    one = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    assert m.kv_append(one[:0], one[:0], cache, i32([[0]]), i32([0])[:0]) is None
    k, v = m.kv_gather(cache, i32([[0]]), i32([0])[:0])
    assert k.shape == v.shape == (0, 1, 64)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("T,D,R,Hq,Hkv", [(1003, 128, 128, 32, 8), (1601, 256, 128, 20, 3), (2003, 64, 64, 50, 9), (1301, 128, 96, 64, 1)])
def test_prompts_of_many_tokens_a_block(kind, T, D, R, Hq, Hkv):
    c = Case(D, R, Hq, Hkv, 24, "head" if D == 256 else "slot", kind, T=T)
    at = np.maximum(c.pos, 0)
    c.run(ftmoe(), rotate32(c.k, c.rope, at), rotate32(c.q, c.rope, at))


def test_prompts_of_many_tokens_that_lie_outside():
    """Tokens without a place among many of a block: their neighbours are as ever."""
    m = ftmoe()
    c = Case(128, 128, 32, 8, 16, "slot", "nvfp4", T=1201)
    at = np.maximum(c.pos, 0)
    cache = c.run(m, rotate32(c.k, c.rope, at), rotate32(c.q, c.rope, at))
    before = cache.k.clone(), cache.k_scales.clone()
    wd = c.wide.cuda()
    args = (wd[:, 32:40], wd[:, 40:], cache, i32(c.table))
    kw = dict(seq_ids=i32(c.seq), q=wd[:, :32], rope=torch.from_numpy(c.rope).cuda())
    whole = m.kv_append(*args, i32(c.pos), **kw)
    assert m.get_error() == 0
    pos = c.pos.copy()
    pos[7] = c.rope.shape[0] + 5                           # past the table of angles
    pos[1100] = 1 << 30
    got = m.kv_append(*args, i32(pos), **kw)
    assert m.get_error() == 6
    assert not got[7].any() and not got[1100].any()
    keep = torch.ones(c.T, dtype=torch.bool)
    keep[[7, 1100]] = False
    assert torch.equal(got[keep.cuda()], whole[keep.cuda()])
    assert torch.equal(cache.k, before[0]) and torch.equal(cache.k_scales.view(torch.uint8), before[1].view(torch.uint8))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("D,R,sections,interleaved", [
    (128, 128, (16, 24, 24), False), (128, 128, (24, 20, 20), True), (64, 64, (8, 12, 12), False),
    (64, 32, (3, 7, 6), True), (256, 256, (32, 48, 48), False), (256, 64, (5, 9, 7, 11), False),
    (128, 64, (32,), False), (64, 64, (0, 1, 31), True)])
def test_several_axes_are_exact(kind, D, R, sections, interleaved):
    m = ftmoe()
    c = Case(D, R, 5, 2, 16, "head" if D == 128 else "slot", kind, seed=R)
    axes = m.RopeAxes.of_sections(sections, interleaved)
    assert len(axes.axes) == R // 2 and [axes.axes.count(a) for a in range(len(sections))] == list(sections)
    pos = c.rng.integers(0, 64, (max(axes.count, len(sections)), c.T)).astype(np.int32)
    pos[:, 3] = 9                                        # equal on every axis, as text is
    pos[:, c.pos < 0] = -5                               # not looked at for padding
    at = np.maximum(pos, 0)
    c.run(m, rotate_axes32(c.k, c.rope, at, axes.axes), rotate_axes32(c.q, c.rope, at, axes.axes),
          rope_positions=i32(pos), rope_axes=axes)


def test_equal_axes_are_one_axis():
    m = ftmoe()
    for kind in ("bf16", "e4m3", "nvfp4"):
        c = Case(128, 128, 4, 2, 16, "slot", kind)
        at = np.maximum(c.pos, 0)
        pos = np.broadcast_to(c.pos, (3, c.T))
        c.run(m, rotate32(c.k, c.rope, at), rotate32(c.q, c.rope, at), rope_positions=i32(pos),
              rope_axes=m.RopeAxes.of_sections((22, 21, 21), True))


def test_what_lies_outside_is_flagged():
    m = ftmoe()
    kc, ks = (t.cuda() for t in pool(4, 16, 1, 64, "slot", False))
    cache = m.NvFP4KVCache(kc, kc.clone(), ks, ks.clone())
    plain = m.PagedKVCache(*(torch.zeros((4, 16, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    table = i32([[0, 1], [2, 9]])
    one = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    rope = torch.zeros((40, 64), dtype=torch.float32, device="cuda")
    axes = m.RopeAxes.of_sections((8, 12, 12))
    ws = torch.zeros(1280, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:1024]
    for seq, pos, bad in ((0, 3, False), (1, 17, True), (0, 32, True), (2, 0, True), (-1, 0, True), (0, 40, True),
                          (0, -1, False)):
        m.kv_append(one, one, cache, table, i32([pos]), seq_ids=i32([seq]), rope=rope, workspace=ws)
        assert m.get_error(ws) == (6 if bad else 0), (seq, pos)
        k, v = m.kv_gather(cache, table, i32([pos]), seq_ids=i32([seq]), workspace=ws)
        # the place alone counts here: 17 of sequence 1 lies on page 9, the rest past the table
        assert m.get_error(ws) == (6 if bad else 0), (seq, pos)
        if pos != 3:
            assert not k.any() and not v.any()
    assert int((cache.v_scales != 0).sum()) == 4          # only the first one was stored
    for c in (cache, plain):
        for where, bad in (([1, 2, 3], False), ([1, 40, 3], True), ([-1, 2, 3], True), ([1, 2, 1 << 30], True)):
            turn = torch.tensor(where, dtype=I32, device="cuda")[:, None].contiguous()
            q = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
            got = m.kv_append(one, one, c, table, i32([7]), q=q, rope=rope, workspace=ws, rope_positions=turn,
                              rope_axes=axes)
            assert m.get_error(ws) == (6 if bad else 0), where
            assert not got.any()                          # a table of zeros, or a query without a place
            m.kv_append(one, one, c, table, i32([-7]), rope=rope, workspace=ws, rope_positions=turn, rope_axes=axes)
            assert m.get_error(ws) == 0                    # padding: its axes are not looked at
    m.kv_append(one, one, plain, table, i32([20]), rope=rope, workspace=ws, rope_positions=i32([[1], [1], [1]]),
                rope_axes=axes)
    assert m.get_error(ws) == 0
    rope20 = rope[:10]                                     # a place past the table of angles is none of its business
    m.kv_append(one, one, plain, table, i32([20]), rope=rope20, workspace=ws, rope_positions=i32([[1], [1], [1]]),
                rope_axes=axes)
    assert m.get_error(ws) == 0
