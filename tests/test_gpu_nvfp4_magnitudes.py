"""Paged attention over NVFP4 caches whose tensor scales, queries and softmax scale have magnitudes from one end of
their ranges to the other, with scores of about one, so that keys, values and both scales count.

Tolerance: as in test_gpu_nvfp4_weights (2^-14 of sum p|v|): factors of two move no rounding, and the factor of a
score, a product of four numbers, is within 2^-22 of itself.
"""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.block_util import bf16, f64
from tests.layer_util import ftmoe

pytestmark = pytest.mark.gpu
REL = 2.0 ** -14


def check(D, Hq, Hkv, g, top, q_size, scale_sign=1.0, n=200, seed=0):
    """g: tensor scales of keys and values; top: their magnitudes over g, block scales of top / 6 or so."""
    m = ftmoe()
    rng = np.random.default_rng(seed + D)
    page = 16
    count = -(-n // page)
    perm = rng.permutation(count + 1)[:count]
    pools, seqs = [], []
    for which in range(2):
        x = rng.standard_normal((n, Hkv, D)) * top[which] / 3 * g[which]
        x *= 2.0 ** rng.integers(-2, 1, (n, Hkv, 1))
        stored = ob.nvfp4_rows(x.astype(np.float32), g[which])
        sc = stored[1]
        assert ((sc > 0) & (sc < 0x7E)).mean() > 0.99      # neither nothing nor all of it saturated
        for part in stored:
            flat = np.full((count * page, *part.shape[1:]), 0x7F, np.uint8)
            flat[:n] = part
            pool = np.full((count + 1, page, *part.shape[1:]), 0x7F, np.uint8)
            pool[perm] = flat.reshape(count, page, *part.shape[1:])
            pools.append(torch.from_numpy(pool).cuda())
        seqs.append(ob.nvfp4_values(*stored, 1.0).astype(np.float64) * float(np.float32(g[which])))
    cache = m.NvFP4KVCache(pools[0], pools[2], pools[1], pools[3], *g)
    q = bf16(rng.standard_normal((1, Hq, D)) * q_size)
    assert torch.isfinite(q).all()
    scale = float(np.float32(scale_sign / (np.sqrt(D) * q_size * top[0] / 3 * g[0])))
    assert np.isfinite(scale) and scale != 0
    out, lse = m.paged_decode_attention(q.cuda(), cache, torch.from_numpy(perm.astype(np.int32))[None].cuda(),
                                        torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale)
    assert m.get_error() == 0
    ref, rlse, mag = ob.attention(f64(q[0]), *seqs, n, scale)
    assert 0.1 < np.abs(rlse - np.log(n)).max() < 20       # the scores are of about one
    got = f64(out[0])
    bound = 1.02 * 2.0 ** -8 * np.abs(ref) + REL * mag     # no absolute part: values may be of any size
    assert np.all(np.abs(got - ref) <= bound), np.max(np.abs(got - ref) / bound)
    assert np.all(np.abs(f64(lse[0]) - rlse) <= 2.0 ** -22 * np.abs(rlse) + 4e-5)


SCALES = [(2.0 ** -100, 2.0 ** 100), (2.0 ** 100, 2.0 ** -100), (2.0 ** -60, 2.0 ** 40), (3.0e4, 1.0e-20),
          (1.7e-19, 5.0e29)]


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 32, 2), (256, 16, 1)])
@pytest.mark.parametrize("g", SCALES)
def test_tensor_scales_that_the_softmax_scale_undoes(g, D, Hq, Hkv):
    check(D, Hq, Hkv, g, (400.0, 400.0), 1.0)
    check(D, Hq, Hkv, g, (1.0, 900.0), 1.0, -1.0, seed=1)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 32, 2), (256, 16, 1)])
@pytest.mark.parametrize("g,top,q_size", [
    (2.0 ** -100, 400.0, 2.0 ** 100), (2.0 ** -100, 2000.0, 2.0 ** 124),   # the latter: scale * g under 2^-126
    (2.0 ** 100, 0.1, 2.0 ** -120), (2.0 ** 100, 0.1, 2.0 ** -127)])       # past 2^128
def test_queries_that_the_scales_undo(g, top, q_size, D, Hq, Hkv):
    check(D, Hq, Hkv, (g, 1.0), (top, 400.0), q_size)


FACTORS = [(16, 128, 64.0, 122, -90), (8, 256, 64.0, 110, -10), (8, 64, 2.0 ** -6, -126, 99), (16, 128, 2.0 ** -6, -126, 90)]


@pytest.mark.parametrize("kind,Hq,D,codes,power,k_power", [("nvfp4", *f) for f in FACTORS] + [("e4m3", *f) for f in FACTORS] +
                         [("e4m3", 8, 64, 64.0, 122, -110)])   # a tensor scale of NVFP4 is 2^-100 at least
def test_powers_of_two_cancel(kind, Hq, D, codes, power, k_power):
    """q 2^power, keys 2^k_power and the softmax scale over both: the bits of q, keys and scale themselves."""
    m = ftmoe()
    rng = np.random.default_rng(Hq)
    n, page = 150, 16
    x = np.clip(np.round(8 * rng.standard_normal((2, 10 * page, 1, D))) / 8, -3, 3).astype(np.float32)
    x[0] *= codes
    if kind == "nvfp4":
        (kc, ks), (vc, vs) = (ob.nvfp4_rows(a.reshape(10, page, 1, D), 1.0) for a in x)
        t = [torch.from_numpy(a).cuda() for a in (kc, vc, ks, vs)]
        cache = lambda g: m.NvFP4KVCache(*t, g, 1.0)  # noqa: E731
    else:
        t = [torch.from_numpy(a.reshape(10, page, 1, D)).to(torch.float8_e4m3fn).cuda() for a in x]
        cache = lambda g: m.PagedKVCache(*t, g, 1.0)  # noqa: E731
    q = bf16(np.clip(np.round(4 * rng.standard_normal((1, Hq, D))) / 4, -3, 3))
    table = torch.arange(10, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    scale = float(np.float32(1 / (codes * np.sqrt(D))))
    want = m.paged_decode_attention(q.cuda(), cache(1.0), table, lens, scale=scale)
    far = (q.double() * 2.0 ** power).bfloat16()
    assert torch.equal(far.double(), q.double() * 2.0 ** power)
    got = m.paged_decode_attention(far.cuda(), cache(2.0 ** k_power), table, lens, scale=scale * 2.0 ** (-power - k_power))
    assert torch.isfinite(want[1]).all()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
