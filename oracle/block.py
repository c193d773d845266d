"""Oracle: the decode block's operators in float64, written from their definitions.

TEST INFRASTRUCTURE — see the package docstring for who may import this.

* linear: y_t = W x_t with W dequantised (oracle.nvfp4).
* rotary: element i and i + R/2 of a head turn by the position's angle i.
* rotary with several axes: pair i turns by the position on its own axis.
* NVFP4 rows: blocks of 16 elements, s = e4m3(max|x| / (6 g)), code = e2m1(x / (s g)), in the float32
  steps that the cache append is defined by.
* attention: softmax(scale q K^T) V over the last `window` of a sequence's first `len` slots.
* norms: r' = r + scale gate norm(y), x' = norm(r'), norm(v) = v / sqrt(mean v^2 + eps) * w, and
  the gradient by the chain rule over each row.

Every function also returns (or takes) plain float64 arrays; `mags` are the sums of magnitudes
behind a result, from which a test derives what rounding may do to it.
"""
from __future__ import annotations

import numpy as np

from .nvfp4 import E2M1_VALUES, E4M3_VALUES, dequantize


def linear(x, codes, scales, gscale):
    """x [T,K] float64 -> (y [T,N], sums of |w x|)."""
    w = dequantize(codes, scales, 1.0).astype(np.float64) * float(np.asarray(gscale).reshape(()))
    return x @ w.T, np.abs(x) @ np.abs(w).T


def rotate(v, rope, positions):
    """v [T,heads,D]; rope [rows,R] = cos | sin."""
    v = np.array(v, np.float64)
    if rope is None or rope.shape[1] == 0:
        return v
    h = rope.shape[1] // 2
    out = v.copy()
    for t, p in enumerate(positions):
        c, s = rope[p, :h].astype(np.float64), rope[p, h:].astype(np.float64)
        a, b = v[t, :, :h], v[t, :, h:2 * h]
        out[t, :, :h] = a * c - b * s
        out[t, :, h:2 * h] = b * c + a * s
    return out


def rotate_axes(v, rope, positions, axis):
    """v [T,heads,D]; positions [axes,T]; axis: one number for each of the R/2 pairs."""
    v = np.array(v, np.float64)
    h, axis = rope.shape[1] // 2, np.asarray(axis)
    at = np.asarray(positions)[axis].T                  # [T, pairs]
    c = rope[at, np.arange(h)].astype(np.float64)[:, None]
    s = rope[at, h + np.arange(h)].astype(np.float64)[:, None]
    out = v.copy()
    out[..., :h] = v[..., :h] * c - v[..., h:2 * h] * s
    out[..., h:2 * h] = v[..., h:2 * h] * c + v[..., :h] * s
    return out


def _nearest(v, values):
    """Index of the value nearest to v >= 0 among `values` (ascending from 0), ties to the even index,
    past the largest: the largest."""
    v = np.asarray(v, np.float64)
    middle = (values[:-1].astype(np.float64) + values[1:]) / 2
    i = np.searchsorted(middle, v, side="left")         # a tie: the lower one
    tie = (i < len(middle)) & (v == middle[np.minimum(i, len(middle) - 1)])
    return (i + (tie & (i % 2 == 1))).astype(np.uint8)


def nvfp4_rows(x, g):
    """float32 [..., D] -> (codes u8 [..., D/2], scales u8 [..., D/16]) under the tensor scale g."""
    g, x = np.float32(g), np.asarray(x, np.float32)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    nan = np.isnan(b).any(-1)
    top = np.where(np.isnan(b), 0, np.abs(b)).max(-1)
    with np.errstate(all="ignore"):
        s = _nearest(top * (np.float32(1) / (np.float32(6) * g)), E4M3_VALUES[:127])
        d = E4M3_VALUES[s] * g
        r = np.where(d > 0, np.float32(1) / np.where(d > 0, d, np.float32(1)), np.float32(0))
        y = b * r[..., None]
    code = _nearest(np.abs(np.where(np.isnan(y), 0, y)), E2M1_VALUES[:8]) | (np.signbit(y).astype(np.uint8) << 3)
    s = np.where(nan, np.uint8(0x7F), s)
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def nvfp4_values(codes, scales, g):
    """What codes u8 [..., D/2] under scales u8 [..., D/16] stand for, float32."""
    return dequantize(codes, scales, g)


def attention(q, keys, values, length, scale, window=0):
    """One sequence: q [Hq,D], keys/values [slots,Hkv,D] -> (out [Hq,D], lse [Hq], sums of p|v|)."""
    Hq, D = q.shape
    G = Hq // keys.shape[1]
    lo = max(0, length - window) if window > 0 else 0
    out, mag, lse = np.zeros((Hq, D)), np.zeros((Hq, D)), np.full(Hq, -np.inf)
    if length <= 0:
        return out, lse, mag
    for h in range(Hq):
        s = scale * (keys[lo:length, h // G] @ q[h])
        m = s.max()
        p = np.exp(s - m)
        lse[h] = m + np.log(p.sum())
        p /= p.sum()
        out[h] = p @ values[lo:length, h // G]
        mag[h] = p @ np.abs(values[lo:length, h // G])
    return out, lse, mag


def _gate(gate, shape):
    return np.ones(shape) if gate is None else np.broadcast_to(np.asarray(gate, np.float64), shape)


def residual_norm(y, r, w_post, w_pre, gate, scale, eps):
    """-> (r', x' or None)."""
    z = y
    if w_post is not None:
        z = y / np.sqrt((y * y).mean(1, keepdims=True) + eps) * w_post
    out = scale * _gate(gate, y.shape) * z + (0.0 if r is None else r)
    x = None
    if w_pre is not None:
        x = out / np.sqrt((out * out).mean(1, keepdims=True) + eps) * w_pre
    return out, x


def residual_norm_backward(y, r, dr, dx, w_post, w_pre, gate, scale, eps):
    """-> dict of the gradients (dgate elementwise, before any sum) and of their magnitudes."""
    g = _gate(gate, y.shape)
    s1 = 1.0 / np.sqrt((y * y).mean(1, keepdims=True) + eps) if w_post is not None else 1.0
    wp = w_post if w_post is not None else 1.0
    z = y * s1 * wp
    out = scale * g * z + (0.0 if r is None else r)
    d_out = np.zeros_like(y) if dr is None else dr.copy()
    got, mag = {}, {}
    m_out = np.abs(d_out)
    if w_pre is not None:
        s2 = 1.0 / np.sqrt((out * out).mean(1, keepdims=True) + eps)
        d = dx * w_pre
        d_out = d_out + s2 * (d - out * s2 ** 2 * (d * out).mean(1, keepdims=True))
        m_out = m_out + s2 * (np.abs(d) + np.abs(out) * s2 ** 2 *
                              np.abs(d * out).mean(1, keepdims=True))
        got["dw_pre"], mag["dw_pre"] = (dx * out * s2).sum(0), np.abs(dx * out * s2).sum(0)
    got["dresidual"], mag["dresidual"] = d_out, m_out
    dz, m_z = scale * g * d_out, np.abs(scale * g) * m_out
    got["dgate"], mag["dgate"] = scale * z * d_out, np.abs(scale * z) * m_out
    got["dy"], mag["dy"] = dz, m_z
    if w_post is not None:
        got["dw_post"], mag["dw_post"] = (dz * y * s1).sum(0), (m_z * np.abs(y) * s1).sum(0)
        h, m_h = dz * w_post, m_z * np.abs(w_post)
        got["dy"] = s1 * (h - y * s1 ** 2 * (h * y).mean(1, keepdims=True))
        mag["dy"] = s1 * (m_h + np.abs(y) * s1 ** 2 * (m_h * np.abs(y)).mean(1, keepdims=True))
    return got, mag
