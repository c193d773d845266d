"""GPU parity of the norms around the gated residual sum, and of their gradient, against float64.

Tolerance: sums of squares and means of H float32 terms (each lane at most 32 in a row, then trees)
are within 2^-19 of their magnitudes, the reciprocal root halves that; the few products after them
add 2^-22: rel = 2^-18 of the sum of magnitudes, for column sums over T rows 2^-17, then one rounding
to the output's type.
"""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.block_util import bf16, close, f64
from tests.layer_util import ftmoe

pytestmark = pytest.mark.gpu
REL, EPS = 2.0 ** -18, 1e-5


def inputs(rng, T, H, res, post, pre, gate):
    shape = {"none": None, "channel": (H,), "token": (T, 1), "element": (T, H)}[gate]
    rt = (lambda a: bf16(a)) if res == torch.bfloat16 else (lambda a: torch.from_numpy(a.astype(np.float32)))
    n = rng.standard_normal
    return dict(y=bf16(n((T, H))), r=rt(2 * n((T, H))), w_post=bf16(1 + 0.2 * n(H)) if post else None,
                w_pre=bf16(1 + 0.2 * n(H)) if pre else None, gate=bf16(n(shape)) if shape else None,
                dr=rt(n((T, H))), dx=bf16(n((T, H))))


def cuda(t):
    return None if t is None else t.cuda()


def forward_close(got, x, a, scale):
    ref, rx = ob.residual_norm(f64(a["y"]), f64(a["r"]), f64(a["w_post"]), f64(a["w_pre"]), f64(a["gate"]),
                               scale, EPS)
    mag = np.abs(ref) + (2 * np.abs(f64(a["r"])) if a["r"] is not None else 0)
    close(got, ref, mag, REL, "r'")
    if a["w_pre"] is None:
        assert x is None
    else:
        s2 = 1 / np.sqrt((ref ** 2).mean(1, keepdims=True) + EPS)
        close(x, rx, mag * s2 * np.abs(f64(a["w_pre"])), REL, "x'")


def check(T, H, res, post, pre, gate, seed, scale=0.7):
    m = ftmoe()
    a = inputs(np.random.default_rng(seed), T, H, res, post, pre, gate)
    d = {n: cuda(t) for n, t in a.items()}
    kw = dict(w_post=d["w_post"], w_pre=d["w_pre"], gate=d["gate"], scale=scale, eps=EPS)
    r, x = m.residual_norm(d["y"], d["r"], **kw)
    assert r.dtype == res
    forward_close(r, x, a, scale)
    g = m.residual_norm_backward(d["y"], d["r"], d["dr"], d["dx"] if pre else None, **kw)
    ref, mag = ob.residual_norm_backward(f64(a["y"]), f64(a["r"]), f64(a["dr"]), f64(a["dx"]),
                                         f64(a["w_post"]), f64(a["w_pre"]), f64(a["gate"]), scale, EPS)
    if gate in ("channel", "token"):
        axis = dict(axis=0) if gate == "channel" else dict(axis=1, keepdims=True)
        ref["dgate"], mag["dgate"] = ref["dgate"].sum(**axis), mag["dgate"].sum(**axis)
    for name in ("dy", "dresidual", "dw_post", "dw_pre", "dgate"):
        t = getattr(g, name)
        if {"dw_post": not post, "dw_pre": not pre, "dgate": gate == "none"}.get(name, False):
            assert t is None
            continue
        close(t, ref[name], mag[name], 2 * REL if name.startswith(("dw", "dg")) else REL, name)
    again = m.residual_norm_backward(d["y"], d["r"], d["dr"], d["dx"] if pre else None, **kw)
    for p, q in zip(g, again):
        assert (p is None) == (q is None) and (p is None or torch.equal(p, q))


KINDS = [(True, True), (True, False), (False, True), (False, False)]


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("post,pre", KINDS)
@pytest.mark.parametrize("H", [136, 1032])
def test_kinds(res, gate, post, pre, H):
    check(19, H, res, post, pre, gate, H)


@pytest.mark.parametrize("H", [8, 64, 248, 256, 264, 504, 512, 520, 2048, 4096, 8184, 8192, 8200, 16384])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_widths(H, res):
    check(5, H, res, True, True, "element", H)


@pytest.mark.parametrize("H,gate", [(8, "token"), (40, "channel"), (64, "element"), (72, "none"), (128, "token"),
                                    (128, "channel"), (200, "element"), (256, "channel")])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [33, 10037])
def test_narrow_rows(T, H, res, gate):
    """Several rows a warp, and several rounds of them a block."""
    check(T, H, res, True, True, gate, T + H)
    check(T, H, res, H % 16 == 0, H % 16 != 0, gate, T + H + 1)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 303, 305, 1000, 5003])
@pytest.mark.parametrize("H", [64, 768])
def test_row_counts(T, H):
    check(T, H, torch.bfloat16, True, True, "channel", T)
    check(T, H, torch.float32, True, True, "token", T)


@pytest.mark.parametrize("T,H,res,gate", [(1500, 4096, torch.float32, "token"), (700, 8192, torch.bfloat16, "element"),
                                          (2000, 1032, torch.float32, "element"), (400, 16384, torch.bfloat16, "none"),
                                          (500, 8192, torch.bfloat16, "channel")])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_several_rows_per_block(T, H, res, gate, post, pre):
    """One, two and three rows in flight per row group."""
    check(T, H, res, post, pre, gate, T)


@pytest.mark.parametrize("T,H,res,gate", [(19500, 72, torch.bfloat16, "channel"), (10001, 776, torch.float32, "element"),
                                          (5003, 2048, torch.bfloat16, "token"), (2600, 4096, torch.float32, "element"),
                                          (1300, 8192, torch.bfloat16, "channel"), (1250, 8200, torch.float32, "none"),
                                          (700, 16384, torch.float32, "element"), (650, 16384, torch.bfloat16, "none")])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_many_rows(T, H, res, gate, post, pre):
    """Several rows per block in the forward pass, in place as well."""
    m = ftmoe()
    a = inputs(np.random.default_rng(T), T, H, res, post, pre, gate)
    d = {n: cuda(t) for n, t in a.items()}
    kw = dict(w_post=d["w_post"], w_pre=d["w_pre"], gate=d["gate"], scale=0.7, eps=EPS)
    r, x = m.residual_norm(d["y"], d["r"], **kw)
    forward_close(r, x, a, 0.7)
    again, _ = m.residual_norm(d["y"], d["r"], res_out=d["r"], x_out=d["y"] if pre else None, **kw)
    assert torch.equal(again, r) and (x is None or torch.equal(d["y"], x))


def test_no_residual_in_place_and_no_gradient_of_r():
    m = ftmoe()
    rng = np.random.default_rng(1)
    a = inputs(rng, 6, 640, torch.bfloat16, True, True, "token")
    d = {n: cuda(t) for n, t in a.items()}
    kw = dict(w_post=d["w_post"], w_pre=d["w_pre"], gate=d["gate"], scale=-1.5, eps=EPS)
    r, x = m.residual_norm(d["y"], None, **kw)
    forward_close(r, x, {**a, "r": None}, -1.5)
    # in place: the sum over the residual, x' over y
    want = m.residual_norm(d["y"], d["r"], **kw)
    y, res = d["y"].clone(), d["r"].clone()
    got = m.residual_norm(y, res, res_out=res, x_out=y, **kw)
    assert got[0] is res and got[1] is y
    assert torch.equal(res, want[0]) and torch.equal(y, want[1])
    g = m.residual_norm_backward(d["y"], d["r"], None, d["dx"], **kw)
    h = m.residual_norm_backward(d["y"], d["r"], torch.zeros_like(d["r"]), d["dx"], **kw)
    for p, q in zip(g, h):
        assert torch.equal(p, q)
    # a plain norm: no residual, no weight after the block
    r, x = m.residual_norm(d["y"], w_pre=d["w_pre"], eps=EPS)
    assert torch.equal(r, d["y"])
    ref = f64(a["y"])
    ref = ref / np.sqrt((ref ** 2).mean(1, keepdims=True) + EPS) * f64(a["w_pre"])
    close(x, ref, np.abs(ref), REL)


def test_rows_of_zeros_and_special_values():
    """A zero row is finite through eps; NaN and infinity stay in their row."""
    m = ftmoe()
    rng = np.random.default_rng(2)
    for H in (64, 1024):
        a = inputs(rng, 12, H, torch.float32, True, True, "channel")
        a["y"][3] = 0
        a["r"][3] = 0
        a["y"][5, 7] = float("nan")
        a["y"][6, 1] = float("inf")
        d = {n: cuda(t) for n, t in a.items()}
        kw = dict(w_post=d["w_post"], w_pre=d["w_pre"], gate=d["gate"], eps=EPS)
        r, x = m.residual_norm(d["y"], d["r"], **kw)
        assert not f64(r[3]).any() and not f64(x[3]).any()
        rows = torch.tensor([i for i in range(12) if i not in (5, 6)])
        assert torch.isfinite(r[rows]).all() and torch.isfinite(x[rows]).all()
        assert torch.isnan(x[5]).all() and torch.isnan(r[6]).any()
        g = m.residual_norm_backward(d["y"], d["r"], d["dr"], d["dx"], **kw)
        assert torch.isfinite(g.dy[rows]).all() and torch.isfinite(g.dresidual[rows]).all()


def test_empty_batch_and_side_stream():
    m = ftmoe()
    y = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    r, x = m.residual_norm(y, y, w_post=w, w_pre=w, gate=w)
    assert r.shape == x.shape == (0, 64)
    g = m.residual_norm_backward(y, y, y, y, w_post=w, w_pre=w, gate=w)
    assert not g.dw_post.any() and not g.dw_pre.any() and not g.dgate.any()
    rng = np.random.default_rng(3)
    a = {n: cuda(t) for n, t in inputs(rng, 50, 256, torch.bfloat16, True, True, "channel").items()}
    args = (a["y"], a["r"], a["dr"], a["dx"])
    kw = dict(w_post=a["w_post"], w_pre=a["w_pre"], gate=a["gate"])
    want = m.residual_norm_backward(*args, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = m.residual_norm_backward(*args, **kw)
    s.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)
