"""GPU parity of the dense NVFP4 product against float64.

Tolerance: bf16 x and dequantised weights are exact in the products; float32 accumulation of K/16
partial products and the joins, each within 2^-23 of the sum of magnitudes, then one rounding to
the output's type: rel = (K/16 + 32) 2^-23.
"""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.block_util import bf16, close, f64
from tests.layer_util import ftmoe

pytestmark = pytest.mark.gpu


def matrix(rng, N, K):
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = rng.integers(0x18, 0x50, (N, K // 16), dtype=np.uint8)    # 2^-4 .. 2^2.9
    return codes, scales, np.array([0.0123], np.float32)


def on_gpu(m, codes, scales, g):
    return m.NvFP4Linear(*(torch.from_numpy(a).cuda() for a in (codes, scales, g)))


def check(T, N, K, dtype, seed, spread=0):
    m = ftmoe()
    rng = np.random.default_rng(seed)
    w = matrix(rng, N, K)
    x = rng.standard_normal((T, K)) * np.exp2(rng.integers(-spread, spread + 1, (T, 1)))
    x = bf16(x)
    got = m.nvfp4_linear(x.cuda(), on_gpu(m, *w), out_dtype=dtype)
    ref, mag = ob.linear(f64(x), *w)
    close(got, ref, mag, (K / 16 + 32) * 2.0 ** -23, f"T={T} N={N} K={K}")


@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 47, 63, 64])
def test_token_counts(T):
    check(T, 200, 1024, torch.bfloat16, T)


@pytest.mark.parametrize("T", [1, 5, 12, 40])
@pytest.mark.parametrize("N,K", [(1, 32), (15, 64), (16, 96), (17, 128), (33, 160), (1003, 416),
                                 (64, 2080), (130, 4096), (7, 16384), (40, 32768), (2500, 1056)])
def test_odd_sizes(T, N, K):
    check(T, N, K, torch.float32, N + K)


@pytest.mark.parametrize("T", [17, 32, 33, 40, 49, 64])
@pytest.mark.parametrize("N", [2333, 4777, 5003])
def test_token_groups(T, N):
    check(T, N, 608, torch.bfloat16, T + N)


@pytest.mark.parametrize("T", [1, 8, 32])
def test_many_rows(T):
    check(T, 20011, 512, torch.bfloat16, 3)


@pytest.mark.parametrize("T", [2, 20])
def test_magnitudes_differ_by_token(T):
    check(T, 65, 512, torch.float32, 4, spread=90)


@pytest.mark.parametrize("T", [1, 20])
def test_rows_of_a_wider_tensor_and_repeatable(T):
    m = ftmoe()
    rng = np.random.default_rng(5)
    w = matrix(rng, 100, 512)
    wide = bf16(rng.standard_normal((T, 800))).cuda()
    x = wide[:, 64:576]
    lin = on_gpu(m, *w)
    a = m.nvfp4_linear(x, lin)
    out = torch.full((T, 100), float("nan"), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert m.nvfp4_linear(x, lin, out=out) is out
    s.synchronize()
    assert torch.equal(a, out)
    assert torch.equal(a, m.nvfp4_linear(x.contiguous(), lin))


@pytest.mark.parametrize("T", [1, 8, 20])
def test_special_values(T):
    """A NaN block scale, and NaN or infinity in one token, reach their outputs and no others; a
    token of zeros, and one of subnormals, are exact."""
    m = ftmoe()
    rng = np.random.default_rng(6)
    codes, scales, g = matrix(rng, 48, 256)
    codes |= 0x11                    # no zero weight: infinity times it is infinity
    scales[5, 3] = 0x7F
    x = bf16(rng.standard_normal((T, 256)))
    if T > 4:
        x[1, 7], x[2, 9] = float("nan"), float("inf")
        x[3] = 0
        x[4] = bf16(rng.integers(-100, 100, 256) * 2.0 ** -133)
    got = f64(m.nvfp4_linear(x.cuda(), on_gpu(m, codes, scales, g), out_dtype=torch.float32))
    rows = np.arange(48) != 5
    assert np.isnan(got[:, 5]).all()
    fine = [t for t in range(T) if t not in (1, 2)] if T > 4 else range(T)
    assert np.isfinite(got[np.ix_(fine, rows)]).all()
    if T > 4:
        assert np.isnan(got[1]).all() and np.isinf(got[2, rows]).all()
        assert not got[3, rows].any()
        ref, mag = ob.linear(f64(x[4:5]), codes[rows], scales[rows], g)
        # float32 subnormal sums: half of 2^-149 each for the products' sum and the last scale
        assert np.all(np.abs(got[4, rows] - ref[0]) <= 48 * 2.0 ** -23 * mag[0] + 2.0 ** -148)


def test_no_tokens_and_graph_capture():
    m = ftmoe()
    rng = np.random.default_rng(7)
    lin = on_gpu(m, *matrix(rng, 96, 256))
    assert m.nvfp4_linear(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), lin).shape == (0, 96)
    x = bf16(rng.standard_normal((3, 256))).cuda()
    out = torch.empty((3, 96), dtype=torch.bfloat16, device="cuda")
    want = m.nvfp4_linear(x, lin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.nvfp4_linear(x, lin, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
