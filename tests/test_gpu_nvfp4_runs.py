"""Paged attention over an NVFP4 cache where the work fills every run: segments that runs cut, that are charged for, that
are left whole, with and without windows; against float64 on the GPU. Random codes under random scales stand for keys
and values (all codes occur). Tolerance: as in test_gpu_nvfp4_attention.
"""
import numpy as np
import pytest
import torch

from oracle.nvfp4 import E2M1_VALUES, E4M3_VALUES
from tests.block_util import close
from tests.layer_util import ftmoe

pytestmark = pytest.mark.gpu
REL = 2.0 ** -10
E2M1 = torch.from_numpy(E2M1_VALUES).double()
E4M3 = torch.from_numpy(E4M3_VALUES).double()


def values(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    return E2M1.cuda()[c] * E4M3.cuda()[scales.long()].repeat_interleave(16, -1)


def check(lens, Hq, Hkv, D, window=0, page=32, order="slot", seed=0):
    m = ftmoe()
    g = torch.Generator(device="cuda").manual_seed(seed)
    byte = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    counts = [-(-n // page) for n in lens]
    P = sum(counts) + 3
    perm = torch.randperm(P, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(lens), max(counts)), -7, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = perm[at:at + n]
        at += n
    turned = lambda t: t if order == "slot" else t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)  # noqa: E731
    # scales between 2^-4 and 2: elements of about 1
    pools = [turned(t) for t in (byte(0, 256, P, page, Hkv, D // 2), byte(0, 256, P, page, Hkv, D // 2),
                                 byte(0x18, 0x40, P, page, Hkv, D // 16), byte(0x18, 0x40, P, page, Hkv, D // 16))]
    cache = m.NvFP4KVCache(*pools, 0.5, 0.25)
    q = torch.randn((len(lens), Hq, D), device="cuda", generator=g).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = m.paged_decode_attention(q, cache, table, n, window=window)
    again, lse2 = m.paged_decode_attention(q, cache, table, n, window=window)
    assert m.get_error() == 0
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    G = Hq // Hkv
    for b, length in enumerate(lens):
        if length == 0:
            assert not out[b].any() and torch.isneginf(lse[b]).all()
            continue
        lo = max(0, length - window) if window else 0
        where = torch.arange(lo, length, device="cuda")
        p, s = table[b].long()[where // page], where % page
        k = values(cache.k[p, s], cache.k_scales[p, s]) * 0.5
        v = values(cache.v[p, s], cache.v_scales[p, s]) * 0.25
        a = torch.einsum("hgd,nhd->hgn", q[b].double().view(Hkv, G, D), k) * D ** -0.5
        w = torch.softmax(a, -1)
        ref = torch.einsum("hgn,nhd->hgd", w, v).reshape(Hq, D)
        mag = torch.einsum("hgn,nhd->hgd", w, v.abs()).reshape(Hq, D)
        close(out[b], ref.cpu().numpy(), mag.cpu().numpy(), REL, f"b={b} len={length}")
        rlse = torch.logsumexp(a, -1).reshape(Hq)
        assert ((lse[b].double() - rlse).abs() <= 2.0 ** -22 * rlse.abs() + 4e-5).all()


def lengths(count, most, seed):
    rng = np.random.default_rng(seed)
    return [0 if rng.random() < 0.1 else int(rng.integers(1, most)) for _ in range(count)]


@pytest.mark.parametrize("D,Hq,Hkv,lens", [
    (128, 32, 8, [9000, 17000, 3, 0, 12001, 6600]),       # few sequences, long runs
    (128, 64, 8, lengths(60, 3000, 1)),                   # past 32 sequences
    (128, 36, 4, lengths(40, 9000, 2)),                   # nine heads a key head
    (128, 14, 2, [60001, 0, 130, 70000, 44444]),
    (64, 28, 4, lengths(50, 12000, 3)),
    (64, 16, 8, [30000, 20001, 0, 64]),
    (64, 32, 2, lengths(33, 30000, 4)),
    (256, 8, 4, [9000, 0, 12001, 6500, 255]),
    (256, 32, 2, lengths(40, 4000, 5))])
def test_runs_that_cut_segments_and_are_charged_for_them(D, Hq, Hkv, lens):
    check(lens, Hq, Hkv, D, order="head" if Hkv == 4 else "slot")


@pytest.mark.parametrize("D,Hq,Hkv,B,L,window", [
    (128, 32, 8, 32, 4000, 512), (128, 8, 8, 60, 300, 0), (64, 16, 2, 60, 300, 0), (256, 16, 2, 90, 200, 0),
    (128, 64, 8, 33, 700, 600), (64, 28, 4, 200, 1700, 1023), (128, 16, 4, 500, 150, 100)])
def test_segments_about_as_long_as_a_run(D, Hq, Hkv, B, L, window):
    check([L] * B, Hq, Hkv, D, window)
    check(lengths(B, L, B), Hq, Hkv, D, window, page=24)
