"""What the decode block's calls refuse, on the CPU: the library's status for each argument (the fake
pointers are never dereferenced: every call fails its checks first), and the binding's errors."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    from nvfp4_mixture_experts_02_gb300 import ftmoe
    return ftmoe


@pytest.fixture
def on_cpu(m, monkeypatch):
    """CPU tensors stand for one device (index -1); a call that reaches the library fails the test."""
    monkeypatch.setattr(m, "_device_of", lambda t, what: t.get_device())
    monkeypatch.setattr(m, "_stream", lambda s, dev=None: pytest.fail("the call was not refused"))
    monkeypatch.setattr(m, "_scratch", lambda *a: pytest.fail("the call was not refused"))
    return m


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("over,expect", [
    (dict(T=-1), 1), (dict(T=65), 2), (dict(N=0), 1), (dict(K=0), 1), (dict(K=48), 2),
    (dict(K=32800), 2), (dict(N=(1 << 30) + 1), 2), (dict(codes=0), 1), (dict(gscale=0), 1), (dict(codes=0x10008), 3),
    (dict(scales=0x20001), 3), (dict(gscale=0x30002), 3), (dict(x=0), 1), (dict(out=0), 1),
    (dict(T=2, stride=56), 1), (dict(stride=68), 3), (dict(x=0x40008), 3), (dict(out=0x50001), 3),
    (dict(out=0x50002, f32=1), 3), (dict(T=0, x=0, out=0), 0), (dict(T=9, ws=0), 1),
    (dict(T=9, ws=0x60010), 3), (dict(T=9, bytes=4096), 4)])
def test_linear(m, over, expect):
    a = dict(T=1, N=8, K=64, codes=0x10000, scales=0x20000, gscale=0x30000, x=0x40000, out=0x50000,
             stride=64, f32=0, ws=0x60000, bytes=1 << 30) | over
    w = m._Matrix(a["N"], a["K"], a["codes"], a["scales"], a["gscale"])
    assert m.lib().ft_nvfp4_linear(a["x"], a["T"], a["stride"], ctypes.byref(w), a["out"], a["f32"],
                                   a["ws"], a["bytes"], None) == expect


def _cache(m, over):
    a = dict(k=0x10000, v=0x20000, P=4, ps=16, Hkv=2, D=64, kp=2048, ks=128, kh=64, vp=2048, vs=128,
             vh=64, dtype=0, k_scale=1.0, v_scale=1.0)
    a |= {n: over.pop(n) for n in list(over) if n in a}
    return m._PagedKV(*a.values())


CACHE = [(dict(P=0), 1), (dict(ps=0), 1), (dict(Hkv=0), 1), (dict(k=0), 1), (dict(dtype=2), 1),
         (dict(k_scale=0.0), 1), (dict(v_scale=NAN), 1), (dict(k_scale=INF), 1), (dict(v_scale=1e-40), 1),
         (dict(D=96), 2), (dict(ks=-128), 1), (dict(vh=68), 3), (dict(dtype=1, kp=2056), 3),
         (dict(v=0x20008), 3)]


@pytest.mark.parametrize("over,expect", CACHE + [
    (dict(T=-1), 1), (dict(T=(1 << 20) + 1), 2), (dict(Hq=-1), 1), (dict(B=-1), 1), (dict(width=-1), 1),
    (dict(rope_dim=8), 2), (dict(rope_dim=80), 2), (dict(T=0, kn=0), 0), (dict(kn=0), 1), (dict(vn=0), 1),
    (dict(table=0), 1), (dict(pos=0), 1), (dict(q=0), 1), (dict(q_out=0), 1), (dict(rope=0), 1),
    (dict(T=9), 1), (dict(kn=0x30008), 3), (dict(k_stride=130), 3), (dict(q_stride=260), 3),
    (dict(q_out=0x60008), 3), (dict(rope=0x90004), 3), (dict(table=0x70002), 3), (dict(ws=0xa0010), 3)])
def test_append(m, over, expect):
    over = dict(over)
    c = _cache(m, over)
    a = dict(kn=0x30000, k_stride=128, vn=0x40000, v_stride=128, q=0x50000, q_stride=256, q_out=0x60000,
             T=3, Hq=4, table=0x70000, B=8, width=2, seq=0, pos=0x80000, rope=0x90000, rows=10, rope_dim=64,
             ws=0xa0000) | over
    st = m.lib().ft_kv_append(a["kn"], a["k_stride"], a["vn"], a["v_stride"], a["q"], a["q_stride"],
                              a["q_out"], a["T"], a["Hq"], ctypes.byref(c), a["table"], a["B"], a["width"],
                              a["seq"], a["pos"], a["rope"], a["rows"], a["rope_dim"], a["ws"], None)
    assert st == expect


@pytest.mark.parametrize("over,expect", CACHE + [
    (dict(B=-1), 1), (dict(B=4097), 2), (dict(Hq=0), 1), (dict(Hq=5), 1), (dict(Hq=2048), 2),
    (dict(window=-1), 1), (dict(scale=NAN), 1), (dict(width=-1), 1), (dict(B=0, q=0), 0), (dict(q=0), 1),
    (dict(table=0), 1), (dict(lens=0), 1), (dict(out=0), 1), (dict(ws=0), 1), (dict(q=0x30008), 3),
    (dict(q_stride=260), 3), (dict(lse=0x60002), 3), (dict(ws=0x90010), 3), (dict(bytes=4096), 4)])
def test_attention(m, over, expect):
    over = dict(over)
    c = _cache(m, over)
    a = dict(q=0x30000, q_stride=256, B=3, Hq=4, table=0x40000, width=2, lens=0x50000, scale=0.1, window=0,
             out=0x70000, lse=0x60000, ws=0x90000, bytes=1 << 30) | over
    st = m.lib().ft_paged_decode_attention(
        a["q"], a["q_stride"], a["B"], a["Hq"], ctypes.byref(c), a["table"], a["width"], a["lens"],
        a["scale"], a["window"], a["out"], a["lse"], a["ws"], a["bytes"], None)
    assert st == expect


NORM = [(dict(T=-1), 1), (dict(H=12), 2), (dict(H=16392), 2), (dict(kind=4), 1), (dict(eps=-1.0), 1),
        (dict(eps=NAN), 1), (dict(scale=INF), 1), (dict(y=0), 1), (dict(gate=0), 1), (dict(y=0x10008), 3),
        (dict(r=0x20008), 3), (dict(w_post=0x30002), 3), (dict(kind=3, gate=0x50002), 3),
        (dict(gate=0x50001), 3)]


def _norm(over):
    return dict(y=0x10000, r=0x20000, w_post=0x30000, w_pre=0x40000, gate=0x50002, kind=2, T=2, H=64,
                scale=1.0, eps=1e-6) | over


@pytest.mark.parametrize("over,expect", NORM + [
    (dict(T=0, y=0, gate=0, x_out=0, r_out=0), 0), (dict(x_out=0), 1), (dict(w_pre=0, r_out=0), 1),
    (dict(r_out=0x60004), 3), (dict(x_out=0x70002), 3)])
def test_norm(m, over, expect):
    a = dict(r_out=0x60000, x_out=0x70000) | _norm(over)
    assert m.lib().ft_residual_norm(a["y"], a["r"], a["w_post"], a["w_pre"], a["gate"], a["kind"], a["T"],
                                    a["H"], 0, a["scale"], a["eps"], a["r_out"], a["x_out"], None) == expect


@pytest.mark.parametrize("over,expect", NORM + [
    (dict(dw_post=0), 1), (dict(dw_pre=0), 1), (dict(dgate=0), 1), (dict(dx=0), 1), (dict(dy=0), 1),
    (dict(dres=0), 1), (dict(dw_pre=0x90004), 3), (dict(dgate=0xa0002), 3), (dict(kind=1, gate=0x50000, dgate=0xa0004), 3),
    (dict(dy=0xb0004), 3), (dict(dr=0xc0002), 3), (dict(ws=0), 1), (dict(ws=0xf0010), 3),
    (dict(bytes=512), 4)])
def test_norm_backward(m, over, expect):
    a = dict(dr=0xc0000, dx=0xd0000, dy=0xb0000, dres=0xe0000, dw_post=0x80000, dw_pre=0x90000, dgate=0xa0000,
             ws=0xf0000, bytes=1 << 30) | _norm(over)
    st = m.lib().ft_residual_norm_backward(
        a["y"], a["r"], a["w_post"], a["w_pre"], a["gate"], a["kind"], a["dr"], a["dx"], a["T"], a["H"], 0,
        a["scale"], a["eps"], a["dy"], a["dres"], a["dw_post"], a["dw_pre"], a["dgate"], a["ws"], a["bytes"],
        None)
    assert st == expect


# ---------------------------------------------------------------- the binding
B16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def test_linear_binding(on_cpu):
    m = on_cpu
    z = torch.zeros
    with pytest.raises(ValueError, match="multiple of 32"):
        m.NvFP4Linear(z(4, 24, dtype=U8), z(4, 3, dtype=U8), z(1))
    with pytest.raises(ValueError, match="scales"):
        m.NvFP4Linear(z(4, 32, dtype=U8), z(4, 3, dtype=U8), z(1))
    with pytest.raises(TypeError):
        m.NvFP4Linear(z(4, 32, dtype=I32), z(4, 4, dtype=U8), z(1))
    w = m.NvFP4Linear(z(4, 32, dtype=U8), z(4, 4, dtype=U8), z(1))
    for x, err in ((z(2, 60, dtype=B16), ValueError), (z(2, 64), TypeError), (z(64, dtype=B16), ValueError),
                   (z(64, 2, dtype=B16).T, ValueError), (z(1, 64, dtype=B16).expand(3, 64), ValueError)):
        with pytest.raises(err):
            m.nvfp4_linear(x, w)
    with pytest.raises(TypeError):
        m.nvfp4_linear(z(2, 64, dtype=B16), w, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out"):
        m.nvfp4_linear(z(2, 64, dtype=B16), w, out=z(2, 5, dtype=B16))


def test_cache_binding(on_cpu):
    m = on_cpu
    k = torch.zeros(4, 16, 2, 64, dtype=B16)
    with pytest.raises(ValueError):
        m.PagedKVCache(k, k[:3])
    with pytest.raises(TypeError):
        m.PagedKVCache(k, k.to(torch.float8_e4m3fn))
    with pytest.raises(TypeError):
        m.PagedKVCache(k.float(), k.float())
    with pytest.raises(ValueError, match="contiguous"):
        m.PagedKVCache(k.transpose(1, 3), k.transpose(1, 3))
    c = m.PagedKVCache(k, k.clone())
    assert (c.page_size, c.Hkv, c.D) == (16, 2, 64)
    i = lambda *s: torch.zeros(s, dtype=I32)
    new, q = torch.zeros(3, 2, 64, dtype=B16), torch.zeros(3, 4, 64, dtype=B16)
    for args, kw, err in (((new, new[:2], c, i(3, 2), i(3)), {}, ValueError),
                          ((new, new, c, i(3, 2), i(4)), {}, ValueError),
                          ((new, new, c, i(2, 2), i(3)), {}, ValueError),
                          ((new, new, c, i(3, 2).long(), i(3)), {}, TypeError),
                          ((new.float(), new, c, i(3, 2), i(3)), {}, TypeError),
                          ((new[:, :1], new, c, i(3, 2), i(3)), {}, ValueError),
                          ((new, new, c, i(3, 2), i(3)), dict(q=q[:2]), ValueError),
                          ((new, new, c, i(3, 2), i(3)), dict(q=q, q_out=q[:, :2]), ValueError),
                          ((new, new, c, i(3, 2), i(3)), dict(rope=torch.zeros(4, 64, dtype=B16)), TypeError),
                          ((new, new, c, i(3, 2), i(3)), dict(seq_ids=i(2)), ValueError),
                          ((new, new, c, i(3, 2), i(3)), dict(workspace=torch.zeros(64, dtype=U8)), ValueError)):
        with pytest.raises(err):
            m.kv_append(*args, **kw)
    for args, kw, err in (((q, c, i(2, 2), i(3)), {}, ValueError), ((q, c, i(3, 2), i(2)), {}, ValueError),
                          ((q[..., :32], c, i(3, 2), i(3)), {}, ValueError),
                          ((q, c, i(3, 2), i(3).float()), {}, TypeError),
                          ((q, c, i(3, 2), i(3)), dict(out=q.float()), TypeError),
                          ((q, c, i(3, 2), i(3)), dict(lse=torch.zeros(3, 3)), ValueError)):
        with pytest.raises(err):
            m.paged_decode_attention(*args, **kw)


def test_norm_binding(on_cpu):
    m = on_cpu
    z = torch.zeros
    y, w = z(3, 64, dtype=B16), z(64, dtype=B16)
    for args, kw, err in (((y[0],), {}, ValueError), ((y.float(),), {}, TypeError),
                          ((y, z(3, 32, dtype=B16)), {}, ValueError), ((y, z(3, 64, dtype=torch.float64)), {}, TypeError),
                          ((y, y), dict(w_post=w[:8]), ValueError), ((y, y), dict(w_pre=w.float()), TypeError),
                          ((y, y), dict(gate=z(3, dtype=B16)), ValueError), ((y, y), dict(gate=z(3, 1)), TypeError),
                          ((y, y), dict(res_out=z(3, 64)), TypeError), ((y.T.contiguous().T, y), {}, ValueError),
                          ((y, y), dict(w_pre=w, x_out=z(3, 64)), TypeError)):
        with pytest.raises(err):
            m.residual_norm(*args, **kw)
    for args, kw, err in (((y, y, y[:2]), {}, ValueError), ((y, y, y.float()), {}, TypeError),
                          ((y, y, y), dict(w_pre=w), ValueError), ((y, y, y, y.float()), dict(w_pre=w), TypeError)):
        with pytest.raises(err):
            m.residual_norm_backward(*args, **kw)
