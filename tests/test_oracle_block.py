"""The decode block's float64 oracle against closed forms, brute force and differences."""
import numpy as np
import pytest

from oracle import block as ob


def test_linear_is_the_sum_of_weights_times_x():
    codes = np.array([[0x21, 0xF7] + [0] * 14], np.uint8)     # 0.5, 1, 6, -6, 0 ...
    scales = np.array([[0x40, 0x38]], np.uint8)               # 2, 1
    x = np.zeros((1, 32))
    x[0, :4] = [3.0, 5.0, 7.0, 11.0]
    y, mag = ob.linear(x, codes, scales, 0.5)
    assert y[0, 0] == 0.5 * 2 * (0.5 * 3 + 5 + 6 * 7 - 6 * 11)
    assert mag[0, 0] == 0.5 * 2 * (0.5 * 3 + 5 + 6 * 7 + 6 * 11)


def test_rotation_keeps_lengths_and_depends_on_the_distance_alone():
    rng = np.random.default_rng(0)
    R, D = 32, 48
    ang = np.arange(50)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    q, k = rng.standard_normal((2, 1, 1, D))
    at = lambda v, p: ob.rotate(v, rope, [p])[0, 0]
    np.testing.assert_allclose(np.linalg.norm(at(q, 17)), np.linalg.norm(q), rtol=1e-13)
    np.testing.assert_allclose(at(q, 20) @ at(k, 9), at(q, 31) @ at(k, 20), rtol=1e-12)
    assert np.array_equal(at(q, 13)[R:], q[0, 0, R:])
    assert np.array_equal(at(q, 0), q[0, 0])


def test_attention_limits():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((4, 8))
    k, v = rng.standard_normal((2, 30, 2, 8))
    out, lse, _ = ob.attention(q, k, v, 0, 0.3)
    assert not out.any() and np.all(lse == -np.inf)
    out, lse, _ = ob.attention(q, k, v, 1, 0.3)                 # one key: its value
    np.testing.assert_allclose(out, v[0, [0, 0, 1, 1]])
    out, lse, _ = ob.attention(q, k, v, 30, 0.0)                # no scores: the mean
    np.testing.assert_allclose(out[0], v[:, 0].mean(0))
    np.testing.assert_allclose(lse, np.log(30.0))
    a, la, _ = ob.attention(q, k, v, 20, 0.7, window=5)
    b, lb, _ = ob.attention(q, k[15:], v[15:], 5, 0.7)
    assert np.array_equal(a, b) and np.array_equal(la, lb)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
def test_norm_gradient_against_differences(post, pre, gate):
    rng = np.random.default_rng(2)
    T, H, eps, scale, h = 3, 8, 1e-3, 0.6, 1e-6
    shape = {"none": None, "channel": (H,), "token": (T, 1), "element": (T, H)}[gate]
    a = {"y": rng.standard_normal((T, H)), "r": rng.standard_normal((T, H)),
         "w_post": rng.standard_normal(H) if post else None,
         "w_pre": rng.standard_normal(H) if pre else None,
         "gate": rng.standard_normal(shape) if shape else None}
    dr, dx = rng.standard_normal((2, T, H))

    def loss(b):
        out, x = ob.residual_norm(b["y"], b["r"], b["w_post"], b["w_pre"], b["gate"], scale, eps)
        return (out * dr).sum() + ((x * dx).sum() if pre else 0.0)

    got, mag = ob.residual_norm_backward(a["y"], a["r"], dr, dx, a["w_post"], a["w_pre"],
                                         a["gate"], scale, eps)
    if gate == "channel":
        got["dgate"] = got["dgate"].sum(0)
    if gate == "token":
        got["dgate"] = got["dgate"].sum(1, keepdims=True)
    for name, d in (("y", "dy"), ("r", "dresidual"), ("w_post", "dw_post"), ("w_pre", "dw_pre"),
                    ("gate", "dgate")):
        if a[name] is None:
            continue
        assert got[d].shape == a[name].shape
        for at in np.ndindex(a[name].shape):
            up, dn = dict(a), dict(a)
            up[name], dn[name] = a[name].copy(), a[name].copy()
            up[name][at] += h
            dn[name][at] -= h
            # central differences: h^2 of the third derivative, and 1e-16 / h of rounding
            np.testing.assert_allclose(got[d][at], (loss(up) - loss(dn)) / (2 * h), rtol=1e-6,
                                       atol=2e-8)
    for d in mag:
        assert d == "dgate" or np.all(np.abs(got[d]) <= mag[d] * (1 + 1e-12))
