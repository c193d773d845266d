"""Paged attention where the softmax weights lie many powers of two apart: a key of large weight whose
value is zero leaves the others' weights as the whole output.

Tolerance as for the other attention tests: 2^-14 (bf16) or 2^-10 (E4M3 caches) of sum p|v|. A float32
score here is a product of at most 24 in magnitude, within 2e-5, and its weight as near.
"""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.block_util import bf16, close, f64
from tests.layer_util import ftmoe

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def cache_of(m, k, v, dtype, page, rng):
    """Keys and values [n, Hkv, D], exact in `dtype`, on pages in random order."""
    n, Hkv, D = k.shape
    count = -(-n // page)
    perm = rng.permutation(count + 2)[:count]
    pools = []
    for a in (k, v):
        pool = torch.zeros((count + 2, page, Hkv, D))
        flat = torch.zeros((count * page, Hkv, D))
        flat[:n] = a
        pool[torch.from_numpy(perm)] = flat.view(count, page, Hkv, D)
        pools.append(pool.to(dtype).cuda())
    return m.PagedKVCache(*pools), torch.from_numpy(perm.astype(np.int32))[None].cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("gap", [6, 10, 12, 14, 16, 18])
@pytest.mark.parametrize("n,D,Hq,Hkv", [(300, 64, 4, 2), (4001, 128, 16, 1), (60000, 64, 8, 1)])
def test_small_weights_beside_a_large_one(dtype, gap, n, D, Hq, Hkv):
    m = ftmoe()
    rng = np.random.default_rng(n + gap)
    k = torch.from_numpy(0.5 * rng.standard_normal((n, Hkv, D)).astype(np.float32)).to(dtype).float()
    v = torch.from_numpy(np.abs(rng.standard_normal((n, Hkv, D))).astype(np.float32)).to(dtype).float()
    k[:, :, 0] = 0
    at = n // 3                        # its score is `gap` (of natural logarithm) above the others' mean
    k[at] = 0
    k[at, :, 0] = gap
    v[at] = 0
    q = bf16(0.5 / np.sqrt(D) * rng.standard_normal((1, Hq, D)))
    q[:, :, 0] = 1
    cache, table = cache_of(m, k, v, dtype, 64, rng)
    out, lse = m.paged_decode_attention(q.cuda(), cache, table,
                                        torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0)
    ref, rlse, mag = ob.attention(f64(q[0]), f64(k), f64(v), n, 1.0)
    close(out[0], ref, mag, 2.0 ** -14 if dtype == torch.bfloat16 else 2.0 ** -10, f"gap {gap}")
    assert np.all(np.abs(f64(lse[0]) - rlse) <= 2.0 ** -22 * np.abs(rlse) + 4e-5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("power", [0, 4, 10, 16, 20, 21, 22, 23, 24, 28, 40, 80])
def test_scores_of_any_size_stay_finite(dtype, power):
    """Scores of +-2^power: the largest keys share the output, equal ones alike."""
    m = ftmoe()
    rng = np.random.default_rng(power)
    n, D = 333, 64
    k = torch.zeros((n, 1, D))
    k[:, 0, 0] = torch.from_numpy(rng.choice([-1.0, -0.5, 0.5], n)).float()
    top = [7, 150, 332]
    k[top, 0, 0] = 1.0
    v = torch.from_numpy(rng.standard_normal((n, 1, D)).astype(np.float32)).to(dtype).float()
    q = torch.zeros((1, 2, D))
    q[:, :, 0] = 2.0 ** power
    cache, table = cache_of(m, k, v, dtype, 16, rng)
    out, lse = m.paged_decode_attention(q.bfloat16().cuda(), cache, table,
                                        torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0)
    ref, rlse, mag = ob.attention(f64(q[0]), f64(k), f64(v), n, 1.0)
    close(out[0], ref, mag, 2.0 ** -14 if dtype == torch.bfloat16 else 2.0 ** -10)
    # log2 units and back: two constants, three products and two sums, each within 2^-24 of the score
    assert np.all(np.abs(f64(lse[0]) - rlse) <= 2.0 ** -21 * np.abs(rlse) + 4e-5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 4, 128), (32, 2, 64), (4, 4, 256)])
def test_weights_keep_their_bits_where_the_values_cancel(dtype, Hq, Hkv, D):
    """Two to five keys a sequence: in a few of a hundred dims the weighted values nearly cancel, so that the
    output's own rounding is small and that of the weights shows. 2^-14 of sum p|v| with either cache."""
    m = ftmoe()
    rng = np.random.default_rng(Hq)
    B, page = 48, 8
    lens = rng.integers(2, 6, B)
    draw = lambda: torch.from_numpy(rng.standard_normal((B, page, Hkv, D)).astype(np.float32)).to(dtype)  # noqa: E731
    k, v = draw(), draw()
    q = bf16(rng.standard_normal((B, Hq, D)))
    out, _ = m.paged_decode_attention(q.cuda(), m.PagedKVCache(k.cuda(), v.cuda()),
                                      torch.arange(B, dtype=torch.int32, device="cuda")[:, None],
                                      torch.from_numpy(lens.astype(np.int32)).cuda())
    for b, n in enumerate(lens):
        ref, _, mag = ob.attention(f64(q[b]), f64(k[b].float()), f64(v[b].float()), int(n), D ** -0.5)
        close(out[b], ref, mag, 2.0 ** -14, f"b={b}")
