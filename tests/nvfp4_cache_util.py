"""Helpers of the NVFP4 cache tests: pages of codes and scales whose unused slots read as NaN."""
import numpy as np
import torch

from oracle import block as ob


def pool(P, page, Hkv, D, order, fill=True):
    """(codes, scales) u8 views [P,page,Hkv,..] of storage in `order` ("slot" or "head"), on the CPU. fill: NaN."""
    got = []
    for width, byte in ((D // 2, 0xA5), (D // 16, 0x7F)):
        shape = (P, page, Hkv, width) if order == "slot" else (P, Hkv, page, width)
        t = torch.full(shape, byte if fill else 0, dtype=torch.uint8)
        got.append(t if order == "slot" else t.permute(0, 2, 1, 3))
    return got


def to_gpu(t, order):
    """On the GPU in the storage order of the view."""
    if order == "slot":
        return t.cuda()
    return t.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)


def paged(rng, lens, page, Hkv, D, order="slot", spare=3, gscale=(0.0021, 0.0017), sigma=1.0):
    """(cache, table, keys, values): sequences of normal keys and values as stored (float64), their pages in
    random order in a pool whose other slots are NaN."""
    from tests.layer_util import ftmoe
    counts = [-(-n // page) for n in lens]
    P = sum(counts) + spare
    perm = rng.permutation(P)
    table = np.full((len(lens), max(max(counts), 1)), -7, np.int32)
    pools, seqs = [], [[], []]
    for which in range(2):
        codes, scales = pool(P, page, Hkv, D, order)
        at = 0
        for b, n in enumerate(lens):
            c, s = ob.nvfp4_rows((sigma * rng.standard_normal((n, Hkv, D))).astype(np.float32), gscale[which])
            for i in range(counts[b]):
                part = slice(i * page, (i + 1) * page)
                m = len(c[part])
                codes[int(perm[at])][:m] = torch.from_numpy(c[part])
                scales[int(perm[at])][:m] = torch.from_numpy(s[part])
                table[b, i] = perm[at]
                at += 1
            # in 64 bits: the product with the tensor's scale is not rounded
            seqs[which].append(ob.nvfp4_values(c, s, 1.0).astype(np.float64) * float(np.float32(gscale[which])))
        pools.append((to_gpu(codes, order), to_gpu(scales, order)))
    (kc, ks), (vc, vs) = pools
    cache = ftmoe().NvFP4KVCache(kc, vc, ks, vs, *gscale)
    return cache, torch.from_numpy(table).cuda(), seqs[0], seqs[1]
