"""What the calls on an NVFP4 cache, the read-back and several rotary axes refuse, on the CPU: the library's
status for each argument (the fake pointers are never dereferenced: every call fails its checks first, or has no
tokens), and the binding's errors."""
import ctypes

import pytest
import torch

from tests.test_block_refusals_cpu import CACHE, _cache, m, on_cpu  # noqa: F401

NAN, INF = float("nan"), float("inf")
BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


def _cache4(m, over):  # noqa: F811
    a = dict(k=0x10000, v=0x20000, ksc=0x11000, vsc=0x21000, P=4, ps=16, Hkv=2, D=64, kp=1024, ks=64, kh=32,
             vp=1024, vs=64, vh=32, ksp=128, kss=8, ksh=4, vsp=128, vss=8, vsh=4, kg=1.0, vg=1.0)
    a |= {n: over.pop(n) for n in list(over) if n in a}
    return m._NvFP4KV(*a.values())


CACHE4 = [(dict(P=0), 1), (dict(ps=0), 1), (dict(Hkv=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(ksc=0), 1),
          (dict(vsc=0), 1), (dict(kg=0.0), 1), (dict(vg=NAN), 1), (dict(kg=INF), 1), (dict(vg=-1.0), 1),
          (dict(kg=2.0 ** -101), 1), (dict(vg=2.0 ** 101), 1), (dict(D=96), 2), (dict(Hkv=1025), 2),
          (dict(ks=-64), 1), (dict(vss=-8), 1), (dict(kp=1032), 3), (dict(vh=40), 3), (dict(ksh=2), 3),
          (dict(D=128, vsp=132), 3), (dict(k=0x10008), 3), (dict(ksc=0x11002), 3), (dict(D=256, vsc=0x21008), 3)]
APPEND = [(dict(T=-1), 1), (dict(T=(1 << 20) + 1), 2), (dict(Hq=-1), 1), (dict(B=-1), 1), (dict(width=-1), 1),
          (dict(rope_dim=8), 2), (dict(rope_dim=96), 2), (dict(T=0, kn=0), 0), (dict(kn=0), 1), (dict(vn=0), 1),
          (dict(table=0), 1), (dict(pos=0), 1), (dict(q=0), 1), (dict(q_out=0), 1), (dict(rope=0), 1),
          (dict(T=9), 1), (dict(kn=0x30008), 3), (dict(k_stride=130), 3), (dict(q_stride=260), 3),
          (dict(q_out=0x60008), 3), (dict(rope=0x90004), 3), (dict(table=0x70002), 3), (dict(ws=0xa0010), 3),
          (dict(axes=0), 1), (dict(axes=5), 1), (dict(axis=(0,) * 31 + (3,)), 1), (dict(stride=-1), 1),
          (dict(turn=0), 1), (dict(turn=0xb0002), 3), (dict(T=0, turn=0), 0)]


def _append(m, fn, c, over):  # noqa: F811
    a = dict(kn=0x30000, k_stride=128, vn=0x40000, v_stride=128, q=0x50000, q_stride=256, q_out=0x60000,
             T=3, Hq=4, table=0x70000, B=8, width=2, seq=0, pos=0x80000, rope=0x90000, rows=10, rope_dim=64,
             ws=0xa0000, turn=0xb0000, stride=3, axes=3, axis=(0, 1, 2) * 10 + (0, 1)) | over
    x = m._RopeAxes(a["turn"], a["stride"], a["axes"], (ctypes.c_uint8 * 128)(*a["axis"]))
    return fn(a["kn"], a["k_stride"], a["vn"], a["v_stride"], a["q"], a["q_stride"], a["q_out"], a["T"], a["Hq"],
              ctypes.byref(c), a["table"], a["B"], a["width"], a["seq"], a["pos"], a["rope"], a["rows"],
              a["rope_dim"], ctypes.byref(x), a["ws"], None)


@pytest.mark.parametrize("over,expect", CACHE4 + APPEND + [(dict(rope_dim=16), 2), (dict(rope_dim=48), 2)])
def test_nvfp4_append(m, over, expect):  # noqa: F811
    over = dict(over)
    c = _cache4(m, over)
    assert _append(m, m.lib().ft_nvfp4_kv_append, c, over) == expect


@pytest.mark.parametrize("over,expect", CACHE + APPEND)
def test_append_with_axes(m, over, expect):  # noqa: F811
    over = dict(over)
    c = _cache(m, over)
    assert _append(m, m.lib().ft_kv_append_axes, c, over) == expect


GATHER = [(dict(T=-1), 1), (dict(T=(1 << 26) + 1), 2), (dict(B=-1), 1), (dict(width=-1), 1), (dict(table=0), 1),
          (dict(pos=0), 1), (dict(k_out=0), 1), (dict(v_out=0), 1), (dict(T=9), 1), (dict(T=9, seq=0x80002), 3),
          (dict(k_out=0x50010), 3), (dict(v_out=0x60008), 3), (dict(pos=0x70001), 3), (dict(ws=0xa0080), 3),
          (dict(T=0, table=0, pos=0, k_out=0, v_out=0), 0)]


@pytest.mark.parametrize("four,over,expect", [(True, *x) for x in CACHE4 + GATHER] + [(False, *x) for x in CACHE + GATHER])
def test_gather(m, four, over, expect):  # noqa: F811
    over = dict(over)
    c = (_cache4 if four else _cache)(m, over)
    a = dict(table=0x40000, B=8, width=2, seq=0, pos=0x70000, T=3, k_out=0x50000, v_out=0x60000, ws=0xa0000) | over
    fn = m.lib().ft_nvfp4_kv_gather if four else m.lib().ft_kv_gather
    assert fn(ctypes.byref(c), a["table"], a["B"], a["width"], a["seq"], a["pos"], a["T"], a["k_out"], a["v_out"],
              a["ws"], None) == expect


@pytest.mark.parametrize("over,expect", CACHE4 + [
    (dict(B=-1), 1), (dict(B=4097), 2), (dict(Hq=0), 1), (dict(Hq=5), 1), (dict(Hq=2048), 2),
    (dict(window=-1), 1), (dict(scale=NAN), 1), (dict(width=-1), 1), (dict(B=0, q=0), 0), (dict(q=0), 1),
    (dict(table=0), 1), (dict(lens=0), 1), (dict(out=0), 1), (dict(ws=0), 1), (dict(q=0x30008), 3),
    (dict(q_stride=260), 3), (dict(lse=0x60002), 3), (dict(ws=0x90010), 3), (dict(bytes=4096), 4),
    (dict(kp=1 << 35), 2), (dict(vs=1 << 33), 2), (dict(ksp=1 << 33), 2), (dict(vsh=1 << 34), 2)])
def test_attention(m, over, expect):  # noqa: F811
    over = dict(over)
    c = _cache4(m, over)
    a = dict(q=0x30000, q_stride=256, B=3, Hq=4, table=0x40000, width=2, lens=0x50000, scale=0.1, window=0,
             out=0x70000, lse=0x60000, ws=0x90000, bytes=1 << 30) | over
    st = m.lib().ft_nvfp4_paged_decode_attention(
        a["q"], a["q_stride"], a["B"], a["Hq"], ctypes.byref(c), a["table"], a["width"], a["lens"],
        a["scale"], a["window"], a["out"], a["lse"], a["ws"], a["bytes"], None)
    assert st == expect


# ---------------------------------------------------------------- the binding
def zeros(*shape, dtype=U8):
    return torch.zeros(shape, dtype=dtype)


def cache4(m, **over):  # noqa: F811
    a = dict(k=zeros(4, 16, 2, 32), v=zeros(4, 16, 2, 32), k_scales=zeros(4, 16, 2, 4),
             v_scales=zeros(4, 16, 2, 4)) | over
    return m.NvFP4KVCache(**a)


@pytest.mark.parametrize("over,error", [
    (dict(k=zeros(4, 16, 64)), ValueError), (dict(v=zeros(4, 16, 2, 64)), ValueError),
    (dict(k_scales=zeros(4, 16, 2, 8)), ValueError), (dict(v_scales=zeros(4, 16, 4)), ValueError),
    (dict(k=zeros(4, 16, 2, 32, dtype=BF)), TypeError), (dict(v_scales=zeros(4, 16, 2, 4, dtype=F32)), TypeError),
    (dict(k=zeros(4, 16, 2, 64)[..., ::2]), ValueError), (dict(k_scales=zeros(4, 16, 2, 8)[..., ::2]), ValueError)])
def test_cache_objects(on_cpu, over, error):  # noqa: F811
    with pytest.raises(error):
        cache4(on_cpu, **over)


def test_sizes_past_32_bits(on_cpu):  # noqa: F811
    big = 1 << 31
    e = lambda w: zeros(1, 1, 1, w).expand(big, 1, 1, w)  # noqa: E731
    with pytest.raises(ValueError, match="too large"):
        on_cpu.NvFP4KVCache(e(32), e(32), e(4), e(4))
    c = cache4(on_cpu)
    many = zeros(1, dtype=I32).expand(big)
    for call in (lambda: on_cpu.kv_gather(c, zeros(1, 2, dtype=I32), many),
                 lambda: on_cpu.kv_gather(c, zeros(1, 1, dtype=I32).expand(1, big), zeros(1, dtype=I32))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("axes", [(), (0,) * 129, (0, -1), (0, 4)])
def test_axes_out_of_range(m, axes):  # noqa: F811
    with pytest.raises(ValueError):
        m.RopeAxes(axes)


def test_sections(m):  # noqa: F811
    assert m.RopeAxes.of_sections((2, 1, 3)).axes == (0, 0, 1, 2, 2, 2)
    assert m.RopeAxes.of_sections((3, 1, 2), interleaved=True).axes == (0, 1, 2, 0, 0, 2)
    assert m.RopeAxes([0, 1]).count == 2
    for bad in ((), (1, -1), (0, 0)):
        with pytest.raises(ValueError):
            m.RopeAxes.of_sections(bad)


def _place(T=2):
    return zeros(4, 2, dtype=I32), zeros(T, dtype=I32)


@pytest.mark.parametrize("over", [
    dict(rope_axes=None), dict(rope=None), dict(rope_positions=None), dict(rope=zeros(9, 32, dtype=F32)),
    dict(rope_positions=zeros(2, 2, dtype=I32)), dict(rope_positions=zeros(3, 3, dtype=I32)),
    dict(rope_positions=zeros(6, dtype=I32)), dict(rope_positions=zeros(2, 3, dtype=I32).T)])
@pytest.mark.parametrize("four", [True, False])
def test_axes_of_a_call(on_cpu, over, four):  # noqa: F811
    c = cache4(on_cpu) if four else on_cpu.PagedKVCache(zeros(4, 16, 2, 64, dtype=BF), zeros(4, 16, 2, 64, dtype=BF))
    a = dict(rope=zeros(9, 64, dtype=F32), rope_positions=zeros(3, 2, dtype=I32),
             rope_axes=on_cpu.RopeAxes.of_sections((8, 12, 12))) | over
    k = zeros(2, 2, 64, dtype=BF)
    with pytest.raises(ValueError):
        on_cpu.kv_append(k, k, c, *_place(), **a)
    with pytest.raises(TypeError):
        on_cpu.kv_append(k, k, c, *_place(), **(a | dict(rope=zeros(9, 64, dtype=F32), rope_axes=on_cpu.RopeAxes((0, 1) * 16),
                                                         rope_positions=zeros(3, 2, dtype=torch.int64))))


@pytest.mark.parametrize("over,error", [
    (dict(positions=zeros(2, 1, dtype=I32)), ValueError), (dict(positions=zeros(2, dtype=torch.int64)), TypeError),
    (dict(seq_ids=zeros(3, dtype=I32)), ValueError), (dict(positions=zeros(5, dtype=I32)), ValueError),
    (dict(k_out=zeros(2, 2, 32, dtype=BF)), ValueError), (dict(v_out=zeros(2, 2, 64, dtype=F32)), TypeError),
    (dict(k_out=zeros(2, 64, 2, dtype=BF).transpose(1, 2)), ValueError),
    (dict(workspace=zeros(100)), ValueError), (dict(block_table=zeros(8, dtype=I32)), ValueError),
    (dict(block_table=zeros(2, 4, dtype=I32).T), ValueError)])
def test_gather_tensors(on_cpu, over, error):  # noqa: F811
    table, pos = _place()
    a = dict(block_table=table, positions=pos) | over
    with pytest.raises(error):
        on_cpu.kv_gather(cache4(on_cpu), **a)
