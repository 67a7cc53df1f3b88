"""Pins of the fp64 definitions in oracle/block_oracle.py (CPU): closed forms,
worked values, gradients against central differences."""
import numpy as np
import pytest

from oracle import block_oracle as K


def rng():
    return np.random.default_rng(11)


def test_scan_worked():
    # a = 1/2 at A_P = 0: h = 1, 1/2 + 2, ...; beta 1 | 1/2 | sqrt(3)/2; g = 1/2 at I_P = 0
    x = np.array([[1.0], [2.0], [-4.0]])
    A = np.zeros((3, 1))
    np.testing.assert_allclose(K.scan(x, A, None, None, K.PLAIN)[:, 0], [1, 2.5, -2.75])
    np.testing.assert_allclose(K.scan(x, A, None, None, K.CONVEX)[:, 0], [0.5, 1.25, -1.375])
    np.testing.assert_allclose(K.scan(x, A, A, np.array([8.0]), K.PLAIN)[:, 0], [4.5, 3.25, -0.375])
    np.testing.assert_allclose(K.scan(x, A, None, None, K.UNIT)[:, 0], np.sqrt(0.75) * np.array([1, 2.5, -2.75]))


def test_scan_closed_form_and_split():
    r = rng()
    x, A, I = r.standard_normal((3, 2, 40, 5))
    h0 = r.standard_normal((2, 5))
    y = K.scan(x, A, I, h0, K.UNIT)
    a, rest, beta, _, g = K.gates(A, I, K.UNIT)
    np.testing.assert_allclose(a + rest, 1)
    np.testing.assert_allclose(beta ** 2 + a ** 2, 1)
    for t in (0, 7, 39):
        want = np.prod(a[:, :t + 1], 1) * h0
        for j in range(t + 1):
            want += np.prod(a[:, j + 1:t + 1], 1) * (beta * g * x)[:, j]
        np.testing.assert_allclose(y[:, t], want)
    first = K.scan(x[:, :13], A[:, :13], I[:, :13], h0, K.UNIT)
    np.testing.assert_allclose(K.scan(x[:, 13:], A[:, 13:], I[:, 13:], first[:, -1], K.UNIT), y[:, 13:])


def test_scan_limits():
    x, h0 = np.ones((2, 1)), np.array([3.0])
    start, keep = np.full((2, 1), np.inf), np.full((2, 1), -np.inf)
    for scale in (K.PLAIN, K.CONVEX, K.UNIT):
        assert (K.scan(x, start, None, h0, scale) == 1).all()  # nothing kept, the whole input taken
    assert (K.scan(x, keep, None, h0, K.CONVEX) == 3).all()
    assert (K.scan(x, keep, None, h0, K.UNIT) == 3).all()
    for scale in (K.PLAIN, K.CONVEX, K.UNIT):
        for A in (start, keep):
            for g in K.scan_backward(x, A, None, h0, K.scan(x, A, None, h0, scale), x, None, scale):
                assert g is None or np.isfinite(g).all()


def difference(f, v, h=1e-6):
    out = np.empty(v.shape)
    for i in np.ndindex(v.shape):
        old = v[i]
        v[i] = old + h
        up = f()
        v[i] = old - h
        out[i] = (up - f()) / (2 * h)
        v[i] = old
    return out


@pytest.mark.parametrize("scale", [K.PLAIN, K.CONVEX, K.UNIT])
@pytest.mark.parametrize("gate", [True, False])
def test_scan_gradients_by_differences(scale, gate):
    r = rng()
    x, A, I = r.standard_normal((3, 9, 2))
    I = I if gate else None
    h0, dl = r.standard_normal((2, 2))
    dy = r.standard_normal((9, 2))

    def loss():
        y = K.scan(x, A, I, h0, scale)
        return np.sum(y * dy) + np.sum(y[-1] * dl)

    got = K.scan_backward(x, A, I, h0, K.scan(x, A, I, h0, scale), dy, dl, scale)
    for g, v in zip(got, (x, A, I, h0)):
        if v is not None:
            np.testing.assert_allclose(g, difference(loss, v), rtol=2e-7, atol=2e-8)


def test_norm_in_worked():
    r, p = np.array([[3.0, 0.0]]), np.array([[0.0, 8.0]])
    r2, u = K.norm_in(r, p, np.array([1.0, 0.5]), np.array([1.0, 10.0]), 0.0)
    np.testing.assert_allclose(r2, [[3, 4]])
    np.testing.assert_allclose(u, np.array([[3, 40]]) / np.sqrt(12.5))


@pytest.mark.parametrize("scaled", [True, False])
def test_norm_in_gradients_by_differences(scaled):
    g = rng()
    r, p, du, dr_out = g.standard_normal((4, 3, 5))
    w, s = 1 + 0.3 * g.standard_normal((2, 5))
    s = s if scaled else None

    def loss():
        r2, u = K.norm_in(r, p, s, w, 1e-3)
        return np.sum(r2 * dr_out) + np.sum(u * du)

    r2, _ = K.norm_in(r, p, s, w, 1e-3)
    dr, dp, dw, ds = K.norm_in_backward(du, dr_out, r2, p, s, w, 1e-3)
    for got, v in ((dr, r), (dp, p), (dw, w), (ds, s)):
        if v is not None:
            np.testing.assert_allclose(got, difference(loss, v), rtol=1e-6, atol=1e-8)


def test_norm_out_order():
    # two heads of two channels, three tokens: channel h d + c of token n is y[h, n, c]
    y = np.arange(1.0, 13.0).reshape(1, 2, 3, 2)
    z = np.full((1, 3, 4), 50.0)  # silu(50) = 50
    one = np.ones(4)
    o = K.norm_out(y, z, one, 1, True, 0.0)
    v = np.array([3.0, 4.0, 9.0, 10.0])  # token 1
    np.testing.assert_allclose(o[0, 1], v / np.sqrt(np.mean(v * v)))
    o = K.norm_out(y, z, one, 2, False, 0.0)
    np.testing.assert_allclose(o[0, 1, 2:], 50 * v[2:] / np.sqrt(np.mean(v[2:] ** 2)))


@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("groups", [1, 2])
def test_norm_out_gradients_by_differences(gate_first, groups):
    g = rng()
    y = g.standard_normal((2, 2, 3, 3))
    z, do = g.standard_normal((2, 2, 3, 6))
    w = 1 + 0.3 * g.standard_normal(6)

    def loss():
        return np.sum(K.norm_out(y, z, w, groups, gate_first, 1e-3) * do)

    got = K.norm_out_backward(do, y, z, w, groups, gate_first, 1e-3)
    for d, v in zip(got, (y, z, w)):
        np.testing.assert_allclose(d, difference(loss, v), rtol=1e-6, atol=1e-8)


def test_bounds_hold_for_fp32():
    """The bounds cover an evaluation in numpy's fp32 of the same definitions, and are not slack by orders."""
    g = rng()
    x, A, I = (g.standard_normal((3, 4, 300, 8)) - np.array([0, 3, 0]).reshape(3, 1, 1, 1)).astype(np.float32)
    y32 = np.empty(x.shape, np.float32)
    a, rest = 1 / (1 + np.exp(A)), 1 / (1 + np.exp(-A))
    u = np.sqrt(rest * (1 + a)) / (1 + np.exp(-I)) * x
    h = np.zeros((4, 8), np.float32)
    for t in range(300):
        h = a[:, t] * h + u[:, t]
        y32[:, t] = h
    A64 = A.astype(np.float64)
    err = np.abs(y32 - K.scan(x.astype(np.float64), A64, I.astype(np.float64), None, K.UNIT))
    bound = K.scan_bound(x.astype(np.float64), A64, I.astype(np.float64), None, K.UNIT)
    assert (err <= bound).all() and (err / bound).max() > 1e-2
    r, p = g.standard_normal((2, 5, 1000)).astype(np.float32)
    w = (1 + 0.1 * g.standard_normal(1000)).astype(np.float32)
    r2 = r + p
    u = r2 * (1 / np.sqrt(np.mean(r2 * r2, -1, keepdims=True) + np.float32(1e-5))) * w
    d = lambda v: v.astype(np.float64)  # noqa: E731
    _, want = K.norm_in(d(r), d(p), None, d(w), 1e-5)
    _, bound = K.norm_in_bound(d(r), d(p), None, d(w), 1e-5, "f32")
    assert (np.abs(u - want) <= bound).all()
