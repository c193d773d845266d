"""Cache appends of more tokens than the device's blocks take in one round: the same bits as the same tokens in chunks
that each fit one (whose values test_gpu_nvfp4_append and test_gpu_block_append hold against float32 arithmetic)."""
import pytest
import torch

from tests.layer_util import ftmoe

pytestmark = pytest.mark.gpu
I32 = torch.int32


def cache_of(m, kind, P, page, Hkv, D):
    zeros = lambda w, t: torch.zeros((P, page, Hkv, w), dtype=t, device="cuda")  # noqa: E731
    if kind == "nvfp4":
        return m.NvFP4KVCache(*(zeros(w, torch.uint8) for w in (D // 2, D // 2, D // 16, D // 16)), 0.002, 0.003)
    t = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    return m.PagedKVCache(zeros(D, t), zeros(D, t), 0.5, 0.25)


def held(cache):
    return [getattr(cache, n).view(torch.uint8) for n in ("k", "v", "k_scales", "v_scales") if hasattr(cache, n)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("T,D,R,Hq,Hkv,axes", [
    (14592, 128, 128, 32, 8, False), (14593, 128, 128, 32, 8, False), (16001, 128, 64, 32, 8, False),
    (29999, 128, 96, 32, 8, True), (15003, 256, 256, 20, 2, True), (17003, 256, 64, 36, 2, False),
    (90001, 64, 64, 1, 1, True)])
def test_prompts_of_several_rounds(kind, T, D, R, Hq, Hkv, axes):
    m = ftmoe()
    g = torch.Generator(device="cuda").manual_seed(T)
    page = 32
    P = -(-T // page)
    wide = torch.randn((T, Hq + 2 * Hkv, D), device="cuda", generator=g).bfloat16()
    q, k, v = wide.split([Hq, Hkv, Hkv], 1)
    angles = torch.rand((T, R // 2), device="cuda", generator=g) * 6.28
    rope = torch.cat([angles.cos(), angles.sin()], 1)
    table = torch.randperm(P, device="cuda", generator=g).to(I32)[None]
    pos, seq = torch.arange(T, dtype=I32, device="cuda"), torch.zeros(T, dtype=I32, device="cuda")
    pos[T // 2] = -1
    turn = torch.randint(0, T, (3, T), dtype=I32, device="cuda", generator=g) if axes else None
    of = m.RopeAxes(tuple(i % 3 for i in range(R // 2))) if axes else None
    one, many = cache_of(m, kind, P, page, Hkv, D), cache_of(m, kind, P, page, Hkv, D)
    got = m.kv_append(k, v, one, table, pos, seq_ids=seq, q=q, rope=rope, rope_positions=turn, rope_axes=of)
    for part in torch.arange(T, device="cuda").split(3500):
        s = slice(int(part[0]), int(part[-1]) + 1)
        want = m.kv_append(k[s], v[s], many, table, pos[s], seq_ids=seq[s], q=q[s], rope=rope, rope_axes=of,
                           rope_positions=turn[:, s].contiguous() if axes else None)
        assert torch.equal(got[s].view(torch.int16), want.view(torch.int16)), s
    assert m.get_error() == 0 and not got[T // 2].any() and got[T - 1].any()
    for a, b in zip(held(one), held(many)):
        assert torch.equal(a, b) and a.any()
