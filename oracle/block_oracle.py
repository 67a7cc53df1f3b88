"""Slow fp64 definitions (numpy) of the gated linear recurrence and of the norms
around a mixer block, with their gradients and first-order error bounds.

Recurrence, per channel (x, A_P, I_P [..,N,C]):
    a = 1 / (1 + e^{A_P}),  g = 1 / (1 + e^{-I_P}) or 1,
    beta = 1 | 1 - a | sqrt(1 - a^2),  h_t = a_t h_{t-1} + beta_t g_t x_t.
Norms:
    r' = r + s p,  u = w r' / sqrt(mean r'^2 + eps)
    t = y silu(z), o = w t / sqrt(mean t^2 + eps)   or   o = w silu(z) y / sqrt(mean y^2 + eps)

The bounds count roundings of U = 2^-24 of the fp32 evaluation: `*_bound`
return the largest error such an evaluation may have, element by element.
"""
from __future__ import annotations

import numpy as np

PLAIN, CONVEX, UNIT = 0, 1, 2
U = 2.0 ** -24
TINY = 1e-35  # what flushes to zero on the way


def sigmoid(x):
    with np.errstate(over="ignore"):
        e = np.exp(-np.abs(x))
        return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def gates(A, I, scale):
    """a, 1 - a, beta, d beta / d A_P, g"""
    a, rest = sigmoid(-A), sigmoid(A)
    if scale == PLAIN:
        beta, dbeta = np.ones_like(a), np.zeros_like(a)
    elif scale == CONVEX:
        beta, dbeta = rest, a * rest
    else:
        beta, dbeta = np.sqrt(rest * (1 + a)), a * a * np.sqrt(rest / (1 + a))
    return a, rest, beta, dbeta, (np.ones_like(a) if I is None else sigmoid(I))


def scan(x, A, I, h0, scale):
    """h [..,N,C], a token after the other"""
    a, _, beta, _, g = gates(A, I, scale)
    h = np.zeros(x.shape[:-2] + x.shape[-1:]) if h0 is None else h0.astype(np.float64)
    u = beta * g * x
    y = np.empty(x.shape)
    for t in range(x.shape[-2]):
        h = a[..., t, :] * h + u[..., t, :]
        y[..., t, :] = h
    return y


def _path(a, step, v, term, m):
    """For h_t = a_t h_{t-1} + v_t started from m: the sums of |terms|, and the
    roundings they carry: `step` for each step of a term, `term` at its start."""
    q = np.zeros_like(m)
    ms, qs = np.empty(a.shape), np.empty(a.shape)
    for t in range(a.shape[-2]):
        now = np.abs(v[..., t, :])
        q = a[..., t, :] * (q + step[..., t, :] * m) + term[..., t, :] * now
        m = a[..., t, :] * m + now
        ms[..., t, :], qs[..., t, :] = m, q
    return ms, qs


def size(x):
    """|x| as it counts in the exponential's error: beyond 104 the value is 0 or 1."""
    return 0.0 if x is None else np.minimum(np.abs(x), 104.0)


# The relative error of e^{-|A|} is |A| + 3 roundings: the product with log2 e is
# off by one (and log2 e by less), which the exponent turns into |A|, and the
# exponential itself by one ulp.  1 + e and its reciprocal: 3, the product: 1, so
# the smaller of a and 1 - a has |A| + 7; the larger has its own rounding and at
# most (|A| + 7) e^{-|A|} <= 7: 8.  Each carried step multiplies by a and rounds
# once: 9, and for A > 0, where a is the smaller, A more.  A term's own start:
# beta |A| + 7 or less (the root halves it, and adds 3), g |I| + 7, two products
# 2: under 30 + |A| + |I|.  Joining the shares of threads, waves, workgroups and
# spans: under 50 more.
STEP, TERM, JOIN = 9.0, 30.0, 50.0


def _step(A):
    return STEP + np.maximum(size(A) * np.sign(A), 0)


def scan_bound(x, A, I, h0, scale):
    a, _, beta, _, g = gates(A, I, scale)
    m = np.zeros(x.shape[:-2] + x.shape[-1:]) if h0 is None else np.abs(h0).astype(np.float64)
    ms, qs = _path(a, _step(A), beta * g * x, TERM + size(A) + size(I), m)
    return U * (qs + JOIN * ms) + TINY


def _reverse(a, dy, dlast):
    """The reverse recurrence's decays a_{t+1} and inputs, time reversed."""
    after = np.concatenate([a[..., 1:, :], np.zeros_like(a[..., :1, :])], -2)
    v = dy.astype(np.float64).copy()
    if dlast is not None:
        v[..., -1, :] += dlast
    return after[..., ::-1, :], v[..., ::-1, :]


def scan_backward(x, A, I, h0, y, dy, dlast, scale):
    """dx, dA, dI (None without I), dh0"""
    a, rest, beta, dbeta, g = gates(A, I, scale)
    after, v = _reverse(a, dy, dlast)
    lam = np.zeros(x.shape[:-2] + x.shape[-1:])
    out = np.empty(x.shape)
    for t in range(x.shape[-2]):
        lam = after[..., t, :] * lam + v[..., t, :]
        out[..., t, :] = lam
    lam = out[..., ::-1, :]
    prev = _before(y, h0)
    dx = lam * beta * g
    dA = lam * (dbeta * g * x - a * rest * prev)
    # 1 - g as sigmoid(-I): the difference has lost its digits from I = 36 on (e^-36 = 2^-52)
    dI = None if I is None else lam * beta * x * g * sigmoid(-I)
    return dx, dA, dI, a[..., 0, :] * lam[..., 0, :]


def _before(y, h0):
    first = np.zeros_like(y[..., :1, :]) if h0 is None else h0[..., None, :].astype(np.float64)
    return np.concatenate([first, y[..., :-1, :]], -2)


def scan_backward_bound(x, A, I, h0, y, dy, dlast, scale):
    a, rest, beta, dbeta, g = gates(A, I, scale)
    after, v = _reverse(a, dy, dlast)
    step = _step(A)
    step = np.concatenate([step[..., 1:, :], step[..., :1, :]], -2)[..., ::-1, :]
    ms, qs = _path(after, step, v, np.ones(x.shape), np.zeros(x.shape[:-2] + x.shape[-1:]))
    ms, qs = ms[..., ::-1, :], qs[..., ::-1, :]
    # lam's own bound, and under 60 + 3 |A| + |I| of the factors (a |A| + 8, 1 - a
    # as much, a^2 twice, the root, g and 1 - g |I| + 8 together, products, the sum)
    lam = U * (qs + (JOIN + 60 + 3 * size(A) + size(I)) * ms)
    prev = np.abs(_before(y, h0))
    dA = lam * (dbeta * g * np.abs(x) + a * rest * prev) + TINY
    dI = None if I is None else lam * beta * np.abs(x) * g * sigmoid(-I) + TINY
    return lam * beta * g + TINY, dA, dI, (lam * a)[..., 0, :] + TINY


# ---- norms ----


def norm_in(r, p, s, w, eps):
    r2 = r if p is None else r + (p if s is None else s * p)
    return r2, w * r2 / np.sqrt(np.mean(r2 * r2, -1, keepdims=True) + eps)


def _inv(t, eps):
    return 1 / np.sqrt(np.mean(t * t, -1, keepdims=True) + eps)


def norm_in_backward(du, dr_out, r, p, s, w, eps):
    """dr, dp, dw, ds over rows [R,E] (ds None without s)"""
    k = _inv(r, eps)
    c = du * w
    dr = (0 if dr_out is None else dr_out) + k * c - k ** 3 * np.mean(c * r, -1, keepdims=True) * r
    dw = np.sum(du * r * k, 0)
    return dr, (dr if s is None else s * dr), dw, (None if s is None else np.sum(dr * p, 0))


def rounding(dtype):
    """Half a step of the type, relative to the value."""
    return 2.0 ** -8 if dtype == "bf16" else U


def sum_roundings(n):
    """Roundings on a path of a sum of n values that no lane adds more than n / 64 + 64 of by itself."""
    return n / 64 + 64


def norm_in_bound(r, p, s, w, eps, dtype):
    r2, u = norm_in(r, p, s, w, eps)
    # k: half of the sum's relative error (its terms are squares), and root,
    # quotient and reciprocal; u: two products, r' itself, the final rounding
    rel = U * (0.5 * sum_roundings(r.shape[-1]) + 8)
    br = U * np.abs(r2) * 2 + TINY
    return br, np.abs(u) * (rel + rounding(dtype)) + np.abs(w) * _inv(r2, eps) * br + TINY


def norm_in_backward_bound(du, dr_out, r, p, s, w, eps):
    R, E = r.shape
    k, c = _inv(r, eps), np.abs(du * w)
    n = sum_roundings(E)
    dr = np.abs(norm_in_backward(du, dr_out, r, p, s, w, eps)[0])
    # k^3 carries three times k's error, the mean n of its own
    e = U * (2 * dr + (0.5 * n + 10) * k * c
             + (2.5 * n + 30) * k ** 3 * np.mean(c * np.abs(r), -1, keepdims=True) * np.abs(r)) + TINY
    dw = U * np.sum(np.abs(du * r) * k * (0.5 * n + 10 + R), 0) + TINY
    if s is None:
        return e, e, dw, None
    return e, np.abs(s) * (e + U * dr) + TINY, dw, np.sum(np.abs(p) * (e + U * (R + 2) * dr), 0) + TINY


def silu(z):
    return z * sigmoid(z)


def silu_slope(z):
    s = sigmoid(z)
    return s * (1 + z * (1 - s))


def _rows(y, groups):
    """[B,H,N,d] in head order -> [B,N,groups,E/groups]"""
    B, H, N, d = y.shape
    return y.transpose(0, 2, 1, 3).reshape(B, N, groups, H * d // groups)


def _heads(t, shape):
    B, H, N, d = shape
    return t.reshape(B, N, H, d).transpose(0, 2, 1, 3)


def norm_out(y, z, w, groups, gate_first, eps):
    t = _rows(y, groups)
    gate, w = silu(z).reshape(t.shape), w.reshape(groups, -1)
    if gate_first:
        t = t * gate
        o = w * t * _inv(t, eps)
    else:
        o = w * gate * t * _inv(t, eps)
    return o.reshape(z.shape)


def norm_out_bound(y, z, w, groups, gate_first, eps, dtype):
    o = np.abs(norm_out(y, z, w, groups, gate_first, eps))
    # silu: 12 + |z| roundings (exponential, sum, reciprocal, products); with the
    # gate first they enter the mean as well, twice
    near = 45 + 3 * np.max(size(z), initial=0)
    return o * (U * (0.5 * sum_roundings(y.shape[1] * y.shape[3] // groups) + near) + rounding(dtype)) + TINY


def norm_out_backward(do, y, z, w, groups, gate_first, eps):
    """dy [B,H,N,d], dz [B,N,Hd], dw [Hd]"""
    yr = _rows(y, groups)
    z4, do4, w4 = z.reshape(yr.shape), do.reshape(yr.shape), w.reshape(groups, -1)
    gate, slope = silu(z4), silu_slope(z4)
    t = yr * gate if gate_first else yr
    k = _inv(t, eps)
    c = do4 * w4 * (1 if gate_first else gate)
    dt = k * c - k ** 3 * np.mean(c * t, -1, keepdims=True) * t
    dy = dt * gate if gate_first else dt
    dz = dt * yr * slope if gate_first else do4 * w4 * yr * k * slope
    dw = np.sum(do4 * t * k * (1 if gate_first else gate), (0, 1))
    return _heads(dy, y.shape), dz.reshape(z.shape), dw.reshape(w.shape)


def norm_out_backward_bound(do, y, z, w, groups, gate_first, eps):
    yr = _rows(y, groups)
    z4, do4, w4 = z.reshape(yr.shape), np.abs(do.reshape(yr.shape)), np.abs(w.reshape(groups, -1))
    gate = np.abs(silu(z4))
    # the slope's own sum s (1 + z (1 - s)) cancels near its zero: bounded by its terms
    slope = sigmoid(z4) * (1 + np.abs(z4) * sigmoid(-z4))
    t = np.abs(yr) * gate if gate_first else np.abs(yr)
    k, n = _inv(t, eps), sum_roundings(yr.shape[-1])
    c = do4 * w4 * (1 if gate_first else gate)
    far = 4 * np.max(size(z), initial=0)  # of the logistic: |z| in silu and in its slope
    e = U * ((0.5 * n + 60 + far) * k * c + (2.5 * n + 150 + 3 * far) * k ** 3 * np.mean(c * t, -1, keepdims=True) * t)
    R = y.shape[0] * y.shape[2]
    if gate_first:
        dy, dz = e * gate, e * np.abs(yr) * slope
    else:
        dy, dz = e, U * (0.5 * n + 60 + far) * do4 * w4 * np.abs(yr) * k * slope
    dw = U * (0.5 * n + 60 + far + R) * np.sum(do4 * t * k * (1 if gate_first else gate), (0, 1))
    return _heads(dy, y.shape) + TINY, dz.reshape(z.shape) + TINY, dw.reshape(w.shape) + TINY
