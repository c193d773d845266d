"""Paged attention and read-back over NVFP4 caches whose keys and values lie differently, and in parts of wider storage:
offsets of their own for each, for every size of head, with windows and with pages outside the pool. Tolerance: as in
test_gpu_nvfp4_weights."""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.block_util import bf16, close, f64
from tests.layer_util import ftmoe

pytestmark = pytest.mark.gpu
REL = 2.0 ** -14
G = (0.0021, 0.0017)


def pools(how, P, page, Hkv, D):
    """Codes and scales of keys and of values [P, page, Hkv, ..], views of storage that is NaN around them."""
    full = lambda byte, *s: torch.full(s, byte, dtype=torch.uint8, device="cuda")  # noqa: E731
    turned = lambda t: t.permute(0, 2, 1, 3)  # noqa: E731
    c, s = D // 2, D // 16
    if how == "values head by head":
        return (full(0xA5, P, page, Hkv + 1, D)[:, :, 1:, :c], turned(full(0xA5, P, Hkv, page, c)),
                full(0x7F, P, page, Hkv, 2 * s)[..., s:], turned(full(0x7F, P, Hkv, page + 3, s)[:, :, 3:]))
    if how == "keys head by head":
        return (turned(full(0xA5, P, Hkv, page, c)), full(0xA5, P, page, Hkv, c),
                turned(full(0x7F, P, Hkv, page, s)), full(0x7F, P, page, Hkv, s))
    if how == "scales apart":                                # codes alike, scales not
        return (full(0xA5, P, page, Hkv, c), full(0xA5, P, page, Hkv, c),
                full(0x7F, P, page, Hkv, s), turned(full(0x7F, P, Hkv, page, s)))
    kv = full(0xA5, P, 2, page, Hkv, c)                      # keys and values of a page side by side: alike
    sc = full(0x7F, P, 2, page, Hkv, s)
    return kv[:, 0], kv[:, 1], sc[:, 0], sc[:, 1]


@pytest.mark.parametrize("how", ["values head by head", "keys head by head", "scales apart", "side by side"])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 16, 2), (64, 48, 3), (128, 24, 3), (128, 32, 2), (256, 8, 1), (256, 48, 3)])
@pytest.mark.parametrize("window", [0, 77])
def test_keys_and_values_that_lie_otherwise(how, D, Hq, Hkv, window):
    m = ftmoe()
    rng = np.random.default_rng(D + Hq)
    lens, page = [131, 0, 16, 1, 700, 65], 24
    counts = [-(-n // page) for n in lens]
    P = sum(counts) + 2
    table = np.full((len(lens), max(counts)), -1, np.int32)
    perm, at = rng.permutation(P), 0
    for b, n in enumerate(counts):
        table[b, :n] = perm[at:at + n]
        at += n
    k, v, ks, vs = pools(how, P, page, Hkv, D)
    seqs = [[], []]
    for b, n in enumerate(lens):
        where = np.arange(n)
        p, s = torch.from_numpy(table[b][where // page]).long().cuda(), torch.from_numpy(where % page).cuda()
        for which, (codes, scales) in enumerate(((k, ks), (v, vs))):
            new = ob.nvfp4_rows(rng.standard_normal((n, Hkv, D)).astype(np.float32), G[which])
            codes[p, s], scales[p, s] = (torch.from_numpy(a).cuda() for a in new)
            seqs[which].append(ob.nvfp4_values(*new, 1.0).astype(np.float64) * float(np.float32(G[which])))
    cache = m.NvFP4KVCache(k, v, ks, vs, *G)
    on_gpu, n = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = bf16(rng.standard_normal((len(lens), Hq, D)))
    qd = q.cuda()

    def check(out, keys, values):
        for b, length in enumerate(lens):
            ref, _, mag = ob.attention(f64(q[b]), keys[b], values[b], length, D ** -0.5, window)
            close(out[b], ref, mag, REL, f"b={b}")

    out, _ = m.paged_decode_attention(qd, cache, on_gpu, n, window=window)
    assert m.get_error() == 0
    check(out, *seqs)
    # one page of the longest sequence outside the pool, inside the window if there is one: zeros, and a flag
    gone = lens[4] // page - 1
    for page_id in (P, -1):
        on_gpu[4, gone] = page_id
        out, _ = m.paged_decode_attention(qd, cache, on_gpu, n, window=window)
        assert m.get_error() == 6
        zeroed = [[x.copy() for x in which] for which in seqs]
        for which in zeroed:
            which[4][gone * page:(gone + 1) * page] = 0
        check(out, *zeroed)
    # read back through the same offsets
    pos = torch.arange(lens[0], dtype=torch.int32, device="cuda")
    got = m.kv_gather(cache, on_gpu, pos, seq_ids=torch.zeros_like(pos))
    for g, which in zip(got, seqs):
        close(g, which[0], np.zeros(which[0].shape), 0)
