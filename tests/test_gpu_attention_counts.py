"""Paged attention at the largest lengths that a call counts: 2^37 / B - 512 keys of a sequence. A cache whose slots all lie
in one place (strides of zero) holds any number of equal keys; the log-sum-exp tells how many of them counted."""
import math

import numpy as np
import pytest
import torch

from tests.block_util import f64
from tests.layer_util import ftmoe

pytestmark = pytest.mark.gpu


def cache_of(m, kind, D, page):
    """One page of `page` slots, all of them the same key and value: ones."""
    same = lambda t: t.cuda()[None, None, None].expand(1, page, 1, len(t))  # noqa: E731
    if kind == "nvfp4":
        codes, scales = torch.full((D // 2,), 0x22, dtype=torch.uint8), torch.full((D // 16,), 0x38, dtype=torch.uint8)
        return m.NvFP4KVCache(same(codes), same(codes), same(scales), same(scales))
    one = torch.ones(D).to(torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
    return m.PagedKVCache(same(one), same(one))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("D", [64, 256])
def test_lengths_are_cut_where_the_units_of_a_call_no_longer_count(kind, D):
    m = ftmoe()
    B, most = 4096, 2 ** 25 - 512
    page = 2 ** 26
    cache = cache_of(m, kind, D, page)
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    q = torch.zeros((B, 1, D), dtype=torch.bfloat16, device="cuda")
    for lens, window, counted, flag in (({5: most, 4000: 3}, 0, {5: most, 4000: 3}, 0),
                                        ({0: page, 4095: 70}, 0, {0: most, 4095: 70}, 6),
                                        ({i: page for i in range(B)}, 100, {0: 100, 77: 100, 4095: 100}, 0),
                                        ({1: page, 9: 2000}, 1000, {1: 1000, 9: 1000}, 0),
                                        ({1: page, 9: 2000}, most + 1, {1: most, 9: 2000}, 6)):
        n = torch.zeros(B, dtype=torch.int32)
        for i, length in lens.items():
            n[i] = length
        out, lse = m.paged_decode_attention(q, cache, table, n.cuda(), window=window)
        assert m.get_error() == flag
        got = f64(lse)[:, 0]
        for i, keys in counted.items():
            # sums of equal weights in float32, some thousands of them at each of their stages: within 2^-10
            assert abs(got[i] - math.log(keys)) <= 2.0 ** -9, (i, keys)
            assert torch.equal(out[i], torch.ones_like(out[i]))
        none = [i for i in range(B) if i not in lens]
        assert np.all(np.isneginf(got[none])) and not out[none].any()
