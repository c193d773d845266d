"""Paged attention over an NVFP4 cache where the rounding of the softmax weights shows: values that nearly cancel,
keys whose weights lie many powers of two apart.

Tolerance: a score of D products in float32 is within (D/16 + 4) 2^-23 of its sum of magnitudes, 2.4e-5 with heads
of 256 and normal q and k, and so is its weight; the denominator as much; a weight in two f16 adds 2^-22, or 2^-35 of
the largest key's weight where it is smaller than that allows: 2^-14 of sum p|v|, as for the other caches, and where
weights lie far apart 2^-35 of the largest one of sum |v|.
"""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.block_util import bf16, close, f64
from tests.layer_util import ftmoe
from tests.nvfp4_cache_util import paged, to_gpu

pytestmark = pytest.mark.gpu
REL = 2.0 ** -14


def lens_of(n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def cache_of(m, k, v, page, order, rng):
    """(cache, table, keys, values): k and v [n, Hkv, D] on pages in random order, and what is stored (float64)."""
    n, Hkv, D = k.shape
    count = -(-n // page)
    perm = rng.permutation(count + 2)[:count]
    pools, kept = [], []
    for a in (k, v):
        stored = ob.nvfp4_rows(a.astype(np.float32), 2.0 ** -7)
        for part in stored:
            flat = np.zeros((count * page, *part.shape[1:]), np.uint8)
            flat[:n] = part
            pool = np.zeros((count + 2, page, *part.shape[1:]), np.uint8)
            pool[perm] = flat.reshape(count, page, *part.shape[1:])
            t = torch.from_numpy(pool)
            pools.append(to_gpu(t if order == "slot" else t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3), order))
        kept.append(ob.nvfp4_values(*stored, 1.0).astype(np.float64) * 2.0 ** -7)
    cache = m.NvFP4KVCache(pools[0], pools[2], pools[1], pools[3], 2.0 ** -7, 2.0 ** -7)
    return cache, torch.from_numpy(perm.astype(np.int32))[None].cuda(), *kept


@pytest.mark.parametrize("order", ["slot", "head"])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 4, 128), (32, 2, 128), (32, 2, 64), (14, 2, 64), (4, 4, 256), (24, 2, 256)])
def test_weights_keep_their_bits_where_the_values_cancel(Hq, Hkv, D, order):
    """Two to five keys a sequence: in a few of a hundred dims the weighted values nearly cancel, so that the
    output's own rounding is small and that of the weights shows."""
    m = ftmoe()
    rng = np.random.default_rng(Hq + D)
    lens = [int(n) for n in rng.integers(2, 6, 48)]
    cache, table, ks, vs = paged(rng, lens, 8, Hkv, D, order)
    q = bf16(rng.standard_normal((48, Hq, D)))
    out, _ = m.paged_decode_attention(q.cuda(), cache, table, lens_of(lens))
    for b, n in enumerate(lens):
        ref, _, mag = ob.attention(f64(q[b]), ks[b], vs[b], n, D ** -0.5)
        close(out[b], ref, mag, REL, f"b={b}")


@pytest.mark.parametrize("n,D,Hq,Hkv", [(20011, 128, 8, 1), (20011, 128, 16, 1), (9001, 64, 8, 2), (30000, 64, 16, 1),
                                        (12001, 256, 4, 1), (12001, 256, 32, 2)])
def test_two_keys_of_different_pieces(n, D, Hq, Hkv):
    """All values but two are zero, and those two keys lie far apart: what the runs' pieces are joined from."""
    m = ftmoe()
    rng = np.random.default_rng(n + Hq)
    k, v = 0.3 * rng.standard_normal((n, Hkv, D)), np.zeros((n, Hkv, D))
    k[:, :, 0] = 0
    for at, gap in ((n // 5, 6.0), (n - 7, 5.5)):
        k[at], k[at, :, 0] = 0, gap
        v[at] = rng.standard_normal((Hkv, D))
    q = bf16(0.5 / np.sqrt(D) * rng.standard_normal((1, Hq, D)))
    q[:, :, 0] = torch.from_numpy(rng.uniform(0.6, 1.2, Hq)).bfloat16()
    cache, table, ks, vs = cache_of(m, k, v, 64, "slot", rng)
    out, _ = m.paged_decode_attention(q.cuda(), cache, table, lens_of([n]), scale=1.0)
    ref, _, mag = ob.attention(f64(q[0]), ks, vs, n, 1.0)
    close(out[0], ref, mag, REL)


@pytest.mark.parametrize("gap", [6, 10, 12, 14, 16, 18])
@pytest.mark.parametrize("n,D,Hq,Hkv", [(300, 64, 4, 2), (4001, 128, 16, 1), (3001, 256, 8, 1), (30000, 64, 8, 1)])
def test_small_weights_beside_a_large_one(gap, n, D, Hq, Hkv):
    """A key of large weight whose value is zero leaves the others' weights as the whole output."""
    m = ftmoe()
    rng = np.random.default_rng(n + gap)
    k, v = 0.5 * rng.standard_normal((n, Hkv, D)), np.abs(rng.standard_normal((n, Hkv, D)))
    k[:, :, 0] = 0
    at = n // 3                        # its score is about `gap` (of natural logarithm) above the others' mean
    k[at], v[at], k[at, :, 0] = 0, 0, gap
    q = bf16(0.5 / np.sqrt(D) * rng.standard_normal((1, Hq, D)))
    q[:, :, 0] = 1
    cache, table, ks, vs = cache_of(m, k, v, 64, "head", rng)
    out, lse = m.paged_decode_attention(q.cuda(), cache, table, lens_of([n]), scale=1.0)
    ref, rlse, mag = ob.attention(f64(q[0]), ks, vs, n, 1.0)
    largest = np.exp(np.einsum("hgd,hd->hg", f64(q[0]).reshape(Hkv, -1, D), ks[at]).reshape(Hq) - rlse)
    floor = 2.0 ** -35 * largest[:, None] * np.repeat(vs.sum(0), Hq // Hkv, 0)
    close(out[0], ref, mag + floor / REL, REL, f"gap {gap}")
    assert np.all(np.abs(f64(lse[0]) - rlse) <= 2.0 ** -22 * np.abs(rlse) + 4e-5)
