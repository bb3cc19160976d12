"""Plain 64-bit reference of the gated recurrence (numpy, token by token), each
value with its magnitude: the same sum over the terms' absolute values, which
is what rounding errors scale with.

bar(L): each step of a run of L tokens rounds its decay, its input and its
state to 2^-24 of their values; the sixteen or so roundings of one token's own
factors (sigmoids with v_exp_f32 and v_rcp_f32 to a unit each, the root of 1 -
a^2 to 4e-7) count in full, those of a run as a random walk at four of its
standard deviations: 2^-23 (16 + 4 sqrt(L)).  A decay e^v has the relative
error of v times |v|, about 4.5 * 2^-24 |v|: magnitudes that carry a decay as a
factor count 1 + |v| / 8 of it (a^2: 1 + |v| / 4).  A gate r, or 1 - a^2, below
2^-126 (the smallest normal number) is 0 or not in fp32: then b and a^2 / b
(which enters as r a^2 / b, about b / 2 |A|) are off by all of their value, at
most 2^-63 sqrt(1 + 2 |A|), which bar(1) = 20 * 2^-23 > 2^-19 allows for once their
magnitude is counted 2^19 times.
"""
import math

import numpy as np

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # of a rounding, relative to the value


def bar(L):
    return 2.0 ** -23 * (16 + 4 * math.sqrt(L))


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def factors(ga, gx, A, ba, bx, unit, starts):
    """r, i, a, b, a^2 / b (0 where b is, and at a start), |v|, and
    how often the magnitudes of b and a^2 / b count."""
    r = sigmoid(ga + (0.0 if ba is None else ba))
    i = np.ones_like(r) if gx is None else sigmoid(gx + (0.0 if bx is None else bx))
    v = A * r
    a = np.exp(v)
    b = np.ones_like(a) if unit else np.sqrt(-np.expm1(2 * v))
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.zeros_like(a) if unit else np.where(b > 0, a * a / b, 0.0)
    if starts is not None:
        s = starts[..., None] != 0
        a, b, q = np.where(s, 0.0, a), np.where(s, 1.0, b), np.where(s, 0.0, q)
    return r, i, a, b, q, np.abs(v), np.where(np.minimum(r, 2 * np.abs(v)) < 2.0 ** -126, 2.0 ** 19, 1.0)


def scan(x, ga, gx, A, ba=None, bx=None, h0=None, starts=None, unit=False):
    """(h, |h|) of every token."""
    _, i, a, b, _, _, many = factors(ga, gx, A, ba, bx, unit, starts)
    u = b * i * x
    h = np.zeros_like(x[:, 0]) if h0 is None else h0.astype(np.float64)
    m = np.abs(h)
    y, my = np.empty_like(x), np.empty_like(x)
    for t in range(x.shape[1]):
        s = np.zeros(x.shape[0], bool) if starts is None else starts[:, t] != 0
        # nothing passes a start, not a NaN either
        h = np.where(s[:, None], 0.0, a[:, t] * h) + u[:, t]
        m = np.where(s[:, None], 0.0, a[:, t] * m) + (many * np.abs(u))[:, t]
        y[:, t], my[:, t] = h, m
    return y, my


def scan_bwd(x, ga, gx, A, dy, ba=None, bx=None, h0=None, starts=None, unit=False, dh_last=None):
    """{name: (gradient, magnitude)}."""
    r, i, a, b, q, v, many = factors(ga, gx, A, ba, bx, unit, starts)
    y, my = scan(x, ga, gx, A, ba, bx, h0, starts, unit)
    first = np.zeros_like(x[:, :1]) if h0 is None else h0[:, None].astype(np.float64)
    hp, mp = np.concatenate([first, y[:, :-1]], 1), np.concatenate([np.abs(first), my[:, :-1]], 1)
    lam, ml = np.empty_like(x), np.empty_like(x)
    c = np.zeros_like(x[:, 0]) if dh_last is None else dh_last.astype(np.float64)
    mc = np.abs(c)
    for t in range(x.shape[1] - 1, -1, -1):
        lam[:, t], ml[:, t] = dy[:, t] + c, np.abs(dy[:, t]) + mc
        c, mc = a[:, t] * lam[:, t], a[:, t] * ml[:, t]
    dv, mv = lam * (a * hp - q * i * x), ml * (a * (1 + v / 8) * mp + many * q * (1 + v / 4) * np.abs(i * x))
    dga, ma = dv * A * r * (1 - r), mv * np.abs(A) * r
    dx, mx = lam * b * i, many * ml * b * i
    dgx, mg = dx * x * (1 - i), mx * np.abs(x)
    both = (0, 1)
    out = dict(dx=(dx, mx), dgate_a=(dga, ma), dA=((dv * r).sum(both), (mv * r).sum(both)),
               dbias_a=(dga.sum(both), ma.sum(both)))
    if gx is not None:
        out.update(dgate_x=(dgx, mg), dbias_x=(dgx.sum(both), mg.sum(both)))
    out["dh0"] = (c, mc)
    return out
