"""Cached tokens read back: bit-exact against the value an element stands for, rounded to bf16."""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.block_util import bf16
from tests.layer_util import ftmoe
from tests.nvfp4_cache_util import pool, to_gpu
from tests.test_gpu_block_attention import F8, bits
from tests.test_gpu_nvfp4_append import i32

pytestmark = pytest.mark.gpu


def cache_of(rng, kind, P, page, Hkv, D, order, gs):
    """A pool full of random values, and what they stand for in float32, [P,page,Hkv,D]."""
    m = ftmoe()
    tensors, values = [], []
    for g in gs:
        x = (rng.standard_normal((P, page, Hkv, D)) * 2.0 ** rng.integers(-6, 6, (P, page, Hkv, 1))).astype(np.float32)
        if kind == "nvfp4":
            c, s = ob.nvfp4_rows(x, g)
            s[0, 0, 0, 0] = 0x7F                          # a block that reads as NaN
            v = ob.nvfp4_values(c, s, g)
            store = [torch.from_numpy(c), torch.from_numpy(s)]
        else:
            t = torch.from_numpy(x).to(F8 if kind == "e4m3" else torch.bfloat16)
            v = t.float().numpy() * np.float32(g)
            store = [t]
        if order == "head":
            store = [t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in store]
        tensors.append([to_gpu(t, order) for t in store])
        values.append(torch.from_numpy(v).bfloat16())
    if kind == "nvfp4":
        return m.NvFP4KVCache(tensors[0][0], tensors[1][0], tensors[0][1], tensors[1][1], *gs), values
    return m.PagedKVCache(tensors[0][0], tensors[1][0], *gs), values


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("D,Hkv,page,order", [(64, 1, 16, "slot"), (128, 8, 24, "head"), (256, 3, 7, "slot"),
                                              (128, 5, 1, "slot"), (64, 2, 128, "head")])
@pytest.mark.parametrize("T", [1, 3, 77, 500])
def test_gather_is_exact(kind, D, Hkv, page, order, T):
    m = ftmoe()
    rng = np.random.default_rng(T + D)
    P = 12
    cache, values = cache_of(rng, kind, P, page, Hkv, D, order, (0.13, 0.0021) if kind != "bf16" else (1.0, 0.3))
    table = rng.permutation(P)[:8].reshape(2, 4).astype(np.int32)
    seq, pos = rng.integers(0, 2, T), rng.integers(0, 4 * page, T)   # any order, some twice
    if T > 3:
        pos[[0, T - 1]] = -1
    out = [torch.full((T, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    m.kv_gather(cache, i32(table), i32(pos), seq_ids=i32(seq), k_out=out[0], v_out=out[1])
    assert m.get_error() == 0
    p, s = table[seq, np.maximum(pos, 0) // page], np.maximum(pos, 0) % page
    for got, v in zip(out, values):
        want = v[p, s]
        want[torch.from_numpy(pos < 0)] = 0
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got.cpu()), nan)
        assert np.array_equal(bits(got.cpu().masked_fill(nan, 0)), bits(want.masked_fill(nan, 0)))
    # the next tokens of a batch: a row of the table each
    n = 2
    k, v = m.kv_gather(cache, i32(table), i32(pos[:n].clip(0)) if T >= n else i32([0, 1]))
    p2 = pos[:n].clip(0) if T >= n else np.array([0, 1])
    want = values[0][table[np.arange(n), p2 // page], p2 % page]
    assert torch.equal(torch.nan_to_num(k.cpu()), torch.nan_to_num(want))


def test_what_was_appended_comes_back():
    """An E4M3 or bf16 cache gives back what was stored, an NVFP4 one within its rounding: half a code's step of
    at most a sixth of the block's largest magnitude, and a scale within 2^-4."""
    m = ftmoe()
    rng = np.random.default_rng(3)
    T, Hkv, D, page = 333, 4, 128, 16
    x = bf16(rng.standard_normal((T, 2 * Hkv, D))).cuda()
    table, pos = i32(rng.permutation(25)[None]), torch.arange(T, dtype=torch.int32, device="cuda")
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    zero = lambda w: torch.zeros((25, page, Hkv, w), dtype=torch.uint8, device="cuda")  # noqa: E731
    four = m.NvFP4KVCache(zero(D // 2), zero(D // 2), zero(D // 16), zero(D // 16), 0.0021, 0.0021)
    eight = m.PagedKVCache(zero(D).view(F8), zero(D).view(F8))
    whole = m.PagedKVCache(*(torch.zeros((25, page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    for cache in (four, eight, whole):
        m.kv_append(x[:, :Hkv], x[:, Hkv:], cache, table, pos, seq_ids=seq)
        k, v = m.kv_gather(cache, table, pos, seq_ids=seq)
        for got, want in ((k, x[:, :Hkv]), (v, x[:, Hkv:])):
            if cache is whole:
                assert torch.equal(got, want)
            elif cache is eight:
                assert torch.equal(got, want.to(F8).bfloat16())
            else:
                top = want.float().unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True)
                off = (got.float() - want.float()).unflatten(-1, (-1, 16)).abs()
                assert (off <= top * (1 / 6 + 1 / 16 + 1 / 128)).all()


def test_offsets_past_32_bits():
    """Pages beyond 2^32 bytes of codes, and results beyond 2^32 bytes."""
    m = ftmoe()
    rng = np.random.default_rng(10)
    P, page, Hkv, D = 140000, 64, 4, 256                  # 4.6e9 bytes of codes
    zero = lambda w: torch.empty((P, page, Hkv, w), dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = m.NvFP4KVCache(zero(D // 2), zero(D // 2), zero(D // 16), zero(D // 16), 0.0021, 0.0017)
    table = torch.tensor([[139999, 133333, 2]], dtype=torch.int32, device="cuda")
    k, v = (bf16(rng.standard_normal((150, Hkv, D))) for _ in range(2))
    pos, seq = torch.arange(150, dtype=torch.int32, device="cuda"), torch.zeros(150, dtype=torch.int32, device="cuda")
    m.kv_append(k.cuda(), v.cuda(), cache, table, pos, seq_ids=seq)
    want = [torch.from_numpy(ob.nvfp4_values(*ob.nvfp4_rows(x.float().numpy(), g), g)).bfloat16()
            for x, g in ((k, 0.0021), (v, 0.0017))]
    got = m.kv_gather(cache, table, pos, seq_ids=seq)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
    T = 2_200_000                                         # 4.5e9 bytes of keys
    where = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    where[-150:] = pos
    out = [torch.full((T, Hkv, D), 1.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    m.kv_gather(cache, table, where, seq_ids=torch.zeros_like(where), k_out=out[0], v_out=out[1])
    for o, w in zip(out, want):
        assert torch.equal(o[-150:].cpu(), w) and not o[:-150].any()
