"""GPU parity of paged attention over an NVFP4 cache against float64.

Tolerance: scores of D products in float32 are within (D/16 + 4) 2^-23 of their sum of magnitudes, about
1e-5 for the normal q and k here; a weight rounded to 11 bits or more adds at most 2^-12 each to numerator
and denominator: rel = 2^-11 + 2^-14 < 2^-10 of sum p|v|, then one bf16 rounding.
"""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.block_util import bf16, close, f64
from tests.layer_util import ftmoe
from tests.nvfp4_cache_util import paged

pytestmark = pytest.mark.gpu
REL = 2.0 ** -10


def check(lens, page, Hq, Hkv, D, seed, order="slot", window=0, scale=None, sigma=1.0, gscale=(0.0021, 0.0017)):
    m = ftmoe()
    rng = np.random.default_rng(seed)
    cache, table, ks, vs = paged(rng, lens, page, Hkv, D, order, sigma=sigma, gscale=gscale)
    q = bf16(rng.standard_normal((len(lens), Hq, D)))
    n = m.paged_attention_workspace_bytes(len(lens), D)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")   # NaN patterns
    ws = ws[(-ws.data_ptr()) % 256:][:n]
    ws[:1024] = 0
    on_gpu = torch.tensor(lens, dtype=torch.int32).cuda()
    out, lse = m.paged_decode_attention(q.cuda(), cache, table, on_gpu, scale=scale, window=window, workspace=ws)
    assert m.get_error(ws) == 0
    sc = D ** -0.5 if scale is None else scale
    got_lse = f64(lse)
    for b, n in enumerate(lens):
        ref, rlse, mag = ob.attention(f64(q[b]), ks[b], vs[b], n, sc, window)
        close(out[b], ref, mag, REL, f"b={b} len={n}")
        if n == 0:
            assert np.all(got_lse[b] == -np.inf) and not f64(out[b]).any()
        else:
            assert np.all(np.abs(got_lse[b] - rlse) <= 2.0 ** -22 * np.abs(rlse) + 4e-5)
    again, _ = m.paged_decode_attention(q.cuda(), cache, table, on_gpu, scale=scale, window=window)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


EDGES = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 0, 255, 257, 700]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 24, 64])
def test_lengths_around_tiles_and_pages(D, page):
    check(EDGES, page, 8, 2, D, D + page)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 2), (5, 1), (7, 7), (10, 2), (16, 1), (27, 3), (40, 2), (64, 1)])
def test_head_layouts(Hq, Hkv, D):
    check([33, 0, 290], 16, Hq, Hkv, D, Hq + D)


@pytest.mark.parametrize("page", [1, 7, 100, 4096])
def test_page_sizes_and_head_major_pages(page):
    check([1, 50, 999], page, 4, 2, 64, page, order="head")
    check([1, 50, 499], page, 4, 2, 128, page, order="head")


@pytest.mark.parametrize("window", [1, 16, 100, 5000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_windows(window, D):
    check([0, 1, 99, 100, 101, 1300], 32, 16 if D == 128 else 4, 1, D, window, window=window)


def test_split_over_the_length():
    check([20011], 16, 4, 1, 128, 1)                     # one segment over every block
    check([9000, 3, 0, 4500], 64, 16, 2, 128, 2)
    check([9000, 3, 0, 4500], 64, 6, 2, 64, 2)
    check([5000, 3, 0, 4500], 64, 9, 1, 256, 2)


def test_many_short_sequences():
    rng = np.random.default_rng(3)
    check([int(n) for n in rng.integers(0, 40, 700)], 16, 2, 2, 64, 4)


@pytest.mark.parametrize("D,Hq,Hkv,window", [(128, 32, 8, 0), (128, 64, 8, 0), (128, 4, 2, 0), (128, 6, 6, 777), (128, 9, 3, 0),
                                             (64, 16, 4, 0), (64, 16, 8, 0), (64, 44, 4, 1501), (256, 8, 4, 0), (256, 34, 2, 0)])
def test_several_key_heads_of_a_block(D, Hq, Hkv, window):
    # work enough for long runs on every block; sequences that end and begin inside them
    unit = 256 if D == 64 else 128
    segments = Hkv * -(-Hq // Hkv // 16)
    keys = 1900 * unit // segments
    lens = [int(keys * x) + 1 for x in (0.4, 0.13, 0.2, 0.17, 0.1)] + [0, 1, 130]
    if window:
        lens = [n + 3 * window // 2 for n in lens] + [window + 5] * (keys // window)
    check(lens, 48, Hq, Hkv, D, D + Hq, window=window)


@pytest.mark.parametrize("gscale", [(2.0 ** -60, 2.0 ** 40), (3.0e4, 1.0e-20)])
def test_magnitudes_of_the_tensor_scales(gscale):
    # keys of magnitude 448 * 6 * gscale, with a softmax scale that undoes it
    check([1, 40, 300], 16, 8, 2, 128, 5, sigma=1.0, gscale=gscale, scale=0.0)


def test_small_and_large_block_scales():
    """Block scales down to the smallest subnormal and up to 448, in one key."""
    m = ftmoe()
    rng = np.random.default_rng(6)
    n, D = 48, 128
    codes = rng.integers(0, 256, (3, 16, 1, D // 2)).astype(np.uint8)
    for small in (True, False):
        s = np.tile(np.array([1, 2, 7, 8, 0x7E, 0x38, 0, 0x10], np.uint8), (3, 16, 1, 1))
        if small:
            s[..., 4] = 3
        cache = m.NvFP4KVCache(*(torch.from_numpy(a).cuda() for a in (codes, codes[::-1].copy(), s, s[:, ::-1].copy())))
        ks = ob.nvfp4_values(codes, s, 1.0).reshape(n, 1, D).astype(np.float64)
        vs = ob.nvfp4_values(codes[::-1], s[:, ::-1], 1.0).reshape(n, 1, D).astype(np.float64)
        q = bf16(rng.standard_normal((1, 4, D)))
        scale = 0.02 if small else 1e-4
        out, lse = m.paged_decode_attention(q.cuda(), cache, torch.arange(3, dtype=torch.int32).cuda()[None],
                                            torch.tensor([n], dtype=torch.int32).cuda(), scale=scale)
        ref, rlse, mag = ob.attention(f64(q[0]), ks, vs, n, scale)
        close(out[0], ref, mag, REL)
        assert np.all(np.abs(f64(lse)[0] - rlse) <= 2.0 ** -22 * np.abs(rlse) + 4e-5)


def test_masked_slots_nan_blocks_and_bad_pages():
    m = ftmoe()
    rng = np.random.default_rng(9)
    for D in (64, 128, 256):
        cache, table, ks, vs = paged(rng, [40, 40], 16, 1, D)
        q = bf16(rng.standard_normal((2, 4, D)))
        n = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
        ws = torch.zeros(m.paged_attention_workspace_bytes(2, D) + 256, dtype=torch.uint8, device="cuda")
        ws = ws[(-ws.data_ptr()) % 256:]
        want, _ = m.paged_decode_attention(q.cuda(), cache, table, n, workspace=ws)
        assert m.get_error(ws) == 0
        kept = table[0, 1].clone()
        table[0, 1] = cache.k.shape[0]
        out, _ = m.paged_decode_attention(q.cuda(), cache, table, n, workspace=ws)
        assert m.get_error(ws) == 6 and m.get_error(ws) == 0
        zeroed = [x[0].copy() for x in (ks, vs)]
        for z in zeroed:
            z[16:32] = 0                                  # reads as zeros
        ref, _, mag = ob.attention(f64(q[0]), zeroed[0], zeroed[1], 40, D ** -0.5)
        close(out[0], ref, mag, REL)
        assert torch.equal(out[1], want[1])               # the other sequence is as ever
        table[0, 1] = kept
        for past in (49, 1 << 20, (1 << 31) - 1):         # cut to the table, whose last slots are NaN
            n[1] = past
            out, _ = m.paged_decode_attention(q.cuda(), cache, table, n, workspace=ws)
            assert m.get_error(ws) == 6 and torch.equal(out[0], want[0]) and torch.isnan(out[1]).all()
        n[1] = 40
        cache.v_scales[int(table[0, 2]), 3, 0, 1] = 0x7F  # a NaN in the second block of elements
        out, _ = m.paged_decode_attention(q.cuda(), cache, table, n, workspace=ws)
        assert torch.isnan(out[0, :, 16:32]).all() and torch.equal(out[1], want[1])
        assert torch.equal(out[0, :, :16], want[0, :, :16]) and torch.equal(out[0, :, 32:], want[0, :, 32:])
        out, lse = m.paged_decode_attention(q.cuda(), cache, table[:, :0].contiguous(), n, workspace=ws)
        assert m.get_error(ws) == 6 and not out.any() and torch.isneginf(lse).all()


def test_offsets_past_32_bits():
    m = ftmoe()
    rng = np.random.default_rng(10)
    P, page, Hkv, D = 140000, 64, 4, 256
    zero = lambda w: torch.empty((P, page, Hkv, w), dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = m.NvFP4KVCache(zero(D // 2), zero(D // 2), zero(D // 16), zero(D // 16), 0.0021, 0.0017)
    table = torch.tensor([[139999, 133333, 2]], dtype=torch.int32, device="cuda")
    k, v = (bf16(rng.standard_normal((150, Hkv, D))) for _ in range(2))
    pos, seq = torch.arange(150, dtype=torch.int32, device="cuda"), torch.zeros(150, dtype=torch.int32, device="cuda")
    m.kv_append(k.cuda(), v.cuda(), cache, table, pos, seq_ids=seq)
    ks, vs = (ob.nvfp4_values(*ob.nvfp4_rows(x.float().numpy(), g), 1.0).astype(np.float64) * float(np.float32(g))
              for x, g in ((k, 0.0021), (v, 0.0017)))
    q = bf16(rng.standard_normal((1, 8, D)))
    out, _ = m.paged_decode_attention(q.cuda(), cache, table, torch.tensor([150], dtype=torch.int32).cuda())
    ref, _, mag = ob.attention(f64(q[0]), ks, vs, 150, D ** -0.5)
    close(out[0], ref, mag, REL)
