"""The cache append of one token, and of many tokens with several rotary axes, bit-exact against float32 arithmetic; what
becomes of the queries and of the cache where a token's place or one of its positions lies outside its table."""
import numpy as np
import pytest
import torch

from tests.block_util import bf16
from tests.layer_util import ftmoe
from tests.test_gpu_block_attention import rotate32
from tests.test_gpu_nvfp4_append import Case, i32, rotate_axes32

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "e4m3", "nvfp4"]


def axes_of(m, R):
    """Three axes in turn, the last pairs all on the first."""
    return m.RopeAxes(tuple(i % 3 if i < R // 2 - 3 else 0 for i in range(R // 2)))


def single(D, R, Hq, Hkv, order, kind, at):
    """A case of one token, at place `at` of its sequence."""
    c = Case(D, R, Hq, Hkv, 16, order, kind, T=30, seed=Hq)
    c.T, c.seq, c.pos = 1, c.seq[:1], np.array([at])
    c.wide = bf16(3 * c.rng.standard_normal((1, Hq + 2 * Hkv, D)))
    c.q, c.k, c.v = c.wide[:, :Hq], c.wide[:, Hq:Hq + Hkv], c.wide[:, Hq + Hkv:]
    return c


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,R,Hq,Hkv", [(64, 64, 1, 1), (64, 32, 0, 1), (128, 128, 3, 1), (128, 64, 0, 2), (256, 256, 8, 1),
                                        (256, 0, 2, 2), (128, 128, 40, 8)])
def test_one_token(kind, D, R, Hq, Hkv):
    m = ftmoe()
    for order, at in (("slot", 0), ("head", 17)):
        c = single(D, R, Hq, Hkv, order, kind, at)
        c.run(m, rotate32(c.k, c.rope, c.pos), rotate32(c.q, c.rope, c.pos))
        if R == 0:
            continue
        c = single(D, R, Hq, Hkv, order, kind, at)
        axes, pos = axes_of(m, R), c.rng.integers(0, 64, (3, 1)).astype(np.int32)
        c.run(m, rotate_axes32(c.k, c.rope, pos, axes.axes), rotate_axes32(c.q, c.rope, pos, axes.axes),
              rope_positions=i32(pos), rope_axes=axes)


# tokens of a block on 152 SMs: 3, 3, 8 times 2, 3 (two heads a thread), 21 times 6
MANY = [(1003, 128, 128, 32, 8), (1201, 128, 96, 32, 8), (6001, 64, 64, 4, 2), (2003, 128, 128, 40, 8), (64001, 64, 32, 1, 1)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,D,R,Hq,Hkv", MANY[:4])
def test_axes_of_many_tokens_a_block(kind, T, D, R, Hq, Hkv):
    m = ftmoe()
    c = Case(D, R, Hq, Hkv, 24, "head" if T % 2003 == 0 else "slot", kind, T=T)
    axes = axes_of(m, R)
    pos = c.rng.integers(0, len(c.rope), (3, T)).astype(np.int32)
    pos[:, c.pos < 0] = 1 << 30                          # not looked at for padding
    at = np.where(c.pos < 0, 0, pos)
    c.run(m, rotate_axes32(c.k, c.rope, at, axes.axes), rotate_axes32(c.q, c.rope, at, axes.axes),
          rope_positions=i32(pos), rope_axes=axes)


def device_case(kind, T, D, R, Hq, Hkv, several, seed=0):
    """(call(positions, seq_ids, turn) -> (q, [pools]), positions, seq_ids, turn, table, P): tokens of four sequences, on
    the GPU; the pools are fresh ones at each call."""
    m = ftmoe()
    g = torch.Generator(device="cuda").manual_seed(T + seed)
    page, B = 16, 4
    width = -(-T // (B * page)) + 2
    P = B * width + 2
    table = torch.randperm(P, device="cuda", generator=g)[:B * width].view(B, width).to(torch.int32)
    wide = torch.randn((T, Hq + 2 * Hkv, D), device="cuda", generator=g).bfloat16()
    angles = torch.rand((T + 64, R // 2), device="cuda", generator=g) * 6.28
    rope = torch.cat([angles.cos(), angles.sin()], 1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") // B
    seq = torch.arange(T, dtype=torch.int32, device="cuda") % B
    turn = torch.randint(0, T + 64, (3, T), dtype=torch.int32, device="cuda", generator=g) if several else None
    axes = axes_of(m, R) if several else None

    def call(pos, seq, turn):
        if kind == "nvfp4":
            t = [torch.zeros((P, page, Hkv, w), dtype=torch.uint8, device="cuda") for w in (D // 2, D // 2, D // 16, D // 16)]
            cache = m.NvFP4KVCache(*t, 0.002, 0.003)
        else:
            dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
            t = [torch.zeros((P, page, Hkv, D), dtype=dtype, device="cuda") for _ in range(2)]
            cache = m.PagedKVCache(*t)
        q, k, v = wide.split([Hq, Hkv, Hkv], 1)
        got = m.kv_append(k, v, cache, table, pos, seq_ids=seq, q=q, rope=rope, rope_positions=turn, rope_axes=axes)
        return got, [x.view(torch.uint8) for x in t]
    return call, pos, seq, turn, table, P


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("several", [False, True])
@pytest.mark.parametrize("T,D,R,Hq,Hkv", MANY + [(40, 128, 128, 8, 2), (1, 64, 64, 4, 1)])
def test_tokens_that_lie_outside(kind, several, T, D, R, Hq, Hkv):
    """Padding and a position past the table of angles give a zero query; a page, sequence or column outside its table
    leaves the rotated query. None of them stores anything, and the other tokens are as ever."""
    m = ftmoe()
    call, pos, seq, turn, table, P = device_case(kind, T, D, R, Hq, Hkv, several)
    whole, stored = call(pos, seq, turn)
    assert m.get_error() == 0 and whole.any(-1).all()
    where = sorted({i for i in (0, 3, 7, T // 2, T - 2, T - 1) if 0 <= i < T})

    def check(pos, seq, turn, zero, flagged):
        got, pools = call(pos, seq, turn)
        assert m.get_error() == (6 if flagged else 0)
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[where] = False
        assert torch.equal(got[keep].view(torch.int16), whole[keep].view(torch.int16))
        if zero:
            assert not got[where].any()
        else:
            assert torch.equal(got[where].view(torch.int16), whole[where].view(torch.int16)) and got[where].any()
        page = table[seq_ok.long(), pos_ok.long() // 16].long()
        for a, b in zip(pools, stored):
            want = b.clone()
            want[page[where], pos_ok[where].long() % 16] = 0
            assert torch.equal(a, want)

    pos_ok, seq_ok = pos, seq
    bad = pos.clone()
    bad[where] = -3
    check(bad, seq, turn, zero=True, flagged=False)
    if several:
        for axis in (0, 1, 2):
            off = turn.clone()
            off[axis, where] = torch.tensor([T + 64, -1, 1 << 30, (1 << 31) - 1, -(1 << 31), T + 65][:len(where)],
                                            dtype=torch.int32, device="cuda")
            check(pos, seq, off, zero=True, flagged=True)
    else:
        bad[where] = T + 64                              # past the table of angles (and of the block table)
        check(bad, seq, turn, zero=True, flagged=True)
    bad = seq.clone()
    for n in (4, -1, 1 << 30):
        bad[where] = n
        check(pos, bad, turn, zero=False, flagged=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("several", [False, True])
@pytest.mark.parametrize("T", [3, 1003])
def test_pages_that_lie_outside(kind, several, T):
    m = ftmoe()
    call, pos, seq, turn, table, P = device_case(kind, T, 128, 128, 32, 8, several, 1)
    whole, stored = call(pos, seq, turn)
    assert m.get_error() == 0
    n = 2 % T                                            # the pages of its neighbours on that page as well
    row, col = int(seq[n]), int(pos[n]) // 16
    kept = table[row, col].clone()
    for page in (P, -1, 1 << 30):
        table[row, col] = page
        got, pools = call(pos, seq, turn)
        assert m.get_error() == 6
        assert torch.equal(got.view(torch.int16), whole.view(torch.int16)) and got[n].any()
        for a, b in zip(pools, stored):
            want = b.clone()
            want[kept.long()] = 0
            assert torch.equal(a, want)
    # a place past the block table, its position on the table of angles or on the axes: the rotated query
    table[row, col] = kept
    if several:
        far = pos.clone()
        far[n] = 16 * table.shape[1]
        got, pools = call(far, seq, turn)
        assert m.get_error() == 6 and torch.equal(got.view(torch.int16), whole.view(torch.int16))
