"""The cache append without rotation and into pages of one slot, bit-exact against float32 arithmetic."""
import numpy as np
import pytest
import torch

from tests.block_util import bf16
from tests.layer_util import ftmoe
from tests.test_gpu_block_attention import F8, as_stored, bits, rope_table, rotate32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("D,R,Hq,Hkv,page", [(128, 0, 8, 2, 1), (128, 128, 8, 2, 1), (64, 0, 4, 4, 16), (256, 0, 2, 1, 5),
                                             (128, 0, 40, 8, 64)])
@pytest.mark.parametrize("order", ["slot", "head"])
def test_every_token_has_a_place(dtype, D, R, Hq, Hkv, page, order):
    m = ftmoe()
    rng = np.random.default_rng(D + R + page)
    T, B = 37, 5
    width = -(-T // page) + 1
    seq = rng.integers(0, B, T)
    pos = np.array([int(np.sum(seq[:t] == seq[t])) for t in range(T)])
    pos[[4, 20]] = -1                                     # padding
    assert (pos >= 0).sum() == T - 2 and (pos // page < width).all()
    P = B * width + 3
    table = rng.permutation(P)[:B * width].reshape(B, width).astype(np.int32)
    rope = rope_table(64, R) if R else None
    wide = bf16(3 * rng.standard_normal((T, Hq + 2 * Hkv, D)))
    q, k, v = wide[:, :Hq], wide[:, Hq:Hq + Hkv], wide[:, Hq + Hkv:]
    shape = (P, page, Hkv, D) if order == "slot" else (P, Hkv, page, D)
    scales = (0.3, 0.02) if dtype == F8 else (1.0, 1.0)
    pools = [torch.zeros(shape, dtype=torch.uint8).to(dtype).cuda() for _ in range(2)]
    view = [p if order == "slot" else p.permute(0, 2, 1, 3) for p in pools]
    want = [p.cpu().clone() for p in view]
    ks = as_stored(rotate32(k, rope, np.maximum(pos, 0)), dtype, scales[0])
    vs = as_stored(v.float().numpy(), dtype, scales[1])
    raw = torch.uint8 if dtype == F8 else torch.int16
    for t in np.flatnonzero(pos >= 0):
        p, s = table[seq[t], pos[t] // page], pos[t] % page
        want[0].view(raw)[p, s], want[1].view(raw)[p, s] = ks[t].view(raw), vs[t].view(raw)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    wd = wide.cuda()
    got = m.kv_append(wd[:, Hq:Hq + Hkv], wd[:, Hq + Hkv:], m.PagedKVCache(*view, *scales), i32(table), i32(pos),
                      seq_ids=i32(seq), q=wd[:, :Hq], rope=None if rope is None else torch.from_numpy(rope).cuda())
    assert m.get_error() == 0
    assert np.array_equal(bits(view[0]), bits(want[0])) and np.array_equal(bits(view[1]), bits(want[1]))
    ref = torch.from_numpy(rotate32(q, rope, np.maximum(pos, 0))).bfloat16()
    ref[torch.from_numpy(pos < 0)] = 0
    assert np.array_equal(bits(got), bits(ref))


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
def test_scales_of_the_cache_cancel(dtype):
    """What is appended under a scale is read back under it: powers of two change nothing."""
    m = ftmoe()
    rng = np.random.default_rng(7)
    n, D = 70, 64
    k, v = (bf16(rng.standard_normal((n, 2, D))).cuda() for _ in range(2))
    q = bf16(rng.standard_normal((1, 4, D))).cuda()
    table = torch.randperm(8).to(torch.int32)[None].cuda()
    pos, seq = torch.arange(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    outs = []
    for scales in ((1.0, 1.0), (0.25, 4.0)):
        cache = m.PagedKVCache(*(torch.zeros((8, 16, 2, D), dtype=torch.uint8).to(dtype).cuda() for _ in range(2)), *scales)
        m.kv_append(k, v, cache, table, pos, seq_ids=seq)
        outs.append(m.paged_decode_attention(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda")))
    if dtype == torch.bfloat16:
        assert torch.equal(outs[0][0], outs[1][0])
        assert (outs[0][1] - outs[1][1]).abs().max() <= 1e-5
    else:   # E4M3 rounds subnormals otherwise
        assert (outs[0][0].float() - outs[1][0].float()).abs().max() <= 0.02
