"""Sizes past 32 bits are refused by the binding of the decode block's calls: the C ABI's are 32-bit integers, and
ctypes would pass their lower bits on. Tensors without storage stand for large ones."""
import pytest
import torch

BIG = 2 ** 32 + 8   # its lower 32 bits are a size that the library takes
BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


@pytest.fixture
def m(monkeypatch):
    from nvfp4_mixture_experts_02_gb300 import ftmoe
    monkeypatch.setattr(ftmoe, "_device_of", lambda t, what: t.get_device())
    monkeypatch.setattr(ftmoe, "_stream", lambda s, dev=None: pytest.fail("the call was not refused"))
    monkeypatch.setattr(ftmoe, "_scratch", lambda *a: pytest.fail("the call was not refused"))
    return ftmoe


def empty(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_matrix(m):
    with pytest.raises(ValueError, match="too large"):
        m.NvFP4Linear(empty(BIG, 16, dtype=U8), empty(BIG, 2, dtype=U8), torch.zeros(1))


def test_cache(m):
    with pytest.raises(ValueError, match="too large"):
        m.PagedKVCache(empty(BIG, 16, 2, 64), empty(BIG, 16, 2, 64))


def test_append_and_attention(m):
    cache = m.PagedKVCache(torch.zeros(4, 16, 2, 64, dtype=BF), torch.zeros(4, 16, 2, 64, dtype=BF))
    k, q, one = torch.zeros(1, 2, 64, dtype=BF), torch.zeros(1, 4, 64, dtype=BF), torch.zeros(1, dtype=I32)
    table = torch.zeros(1, 2, dtype=I32)
    for wrong in (empty(BIG, 1, dtype=I32), empty(1, BIG, dtype=I32)):
        with pytest.raises(ValueError, match="too large"):
            m.kv_append(k, k, cache, wrong, one)
    with pytest.raises(ValueError, match="too many"):
        m.kv_append(k, k, cache, table, one, rope=empty(BIG, 16, dtype=torch.float32))
    with pytest.raises(ValueError, match="out of range"):
        m.paged_decode_attention(q, cache, empty(1, BIG, dtype=I32), one)
    for window in (2 ** 32 + 100, 2 ** 31):
        with pytest.raises(ValueError, match="out of range"):
            m.paged_decode_attention(q, cache, table, one, window=window)


def test_norm(m):
    y = empty(BIG, 8)
    with pytest.raises(ValueError, match="too many"):
        m.residual_norm(y, y)
    with pytest.raises(ValueError, match="too many"):
        m.residual_norm_backward(y, y, y)
