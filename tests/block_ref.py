"""Plain 64-bit references of the block operators (numpy, token by token),
each value with its magnitude: the same sum over the terms' absolute values,
which is what rounding errors scale with."""
import numpy as np

EPS32, EPS16 = 2.0 ** -24, 2.0 ** -9  # unit roundoffs of fp32 and bf16


def steps(delta, bias, softplus, shape):
    """(step, d step / d delta)."""
    if delta is None:
        return np.ones(shape), np.zeros(shape)
    v = delta + (0.0 if bias is None else bias)
    if not softplus:
        return v, np.ones(shape)
    return np.logaddexp(v, 0.0), 1.0 / (1.0 + np.exp(-v))


def _heads(t, per):
    return np.repeat(t, per, axis=-2)


def scan(x, delta, A, Bm, Cm, D=None, h0=None, bias=None, softplus=False, unit=False):
    """y, |y|, h_last, |h_last|."""
    b, L, H, P = x.shape
    N, per = Bm.shape[-1], H // Bm.shape[2]
    s, _ = steps(delta, bias, softplus, (b, L, H))
    w = np.ones_like(s) if unit else s
    S = np.zeros((b, H, P, N)) if h0 is None else h0.astype(np.float64)
    M = np.abs(S)
    y, m = np.zeros(x.shape), np.zeros(x.shape)
    d = np.zeros(H) if D is None else D
    for t in range(L):
        with np.errstate(over="ignore", under="ignore"):
            e = np.exp(s[:, t] * A)[..., None, None]
        u = (w[:, t, :, None] * x[:, t])[..., None] * _heads(Bm[:, t], per)[:, :, None]
        S, M = e * S + u, e * M + np.abs(u)
        c = _heads(Cm[:, t], per)[:, :, None]
        y[:, t] = (S * c).sum(-1) + d[:, None] * x[:, t]
        m[:, t] = (M * np.abs(c)).sum(-1) + np.abs(d[:, None] * x[:, t])
    return y, m, S, M


def scan_bwd(x, delta, A, Bm, Cm, dy, D=None, h0=None, dh_last=None, bias=None, softplus=False, unit=False):
    """{name: (gradient, magnitude)}."""
    b, L, H, P = x.shape
    G, N = Bm.shape[2:]
    per = H // G
    s, ds_dv = steps(delta, bias, softplus, (b, L, H))
    w = np.ones_like(s) if unit else s
    e = np.exp(s * A)
    S = [np.zeros((b, H, P, N)) if h0 is None else h0.astype(np.float64)]
    M = [np.abs(S[0])]
    for t in range(L):
        u = (w[:, t, :, None] * x[:, t])[..., None] * _heads(Bm[:, t], per)[:, :, None]
        S.append(e[:, t, :, None, None] * S[-1] + u)
        M.append(e[:, t, :, None, None] * M[-1] + np.abs(u))
    d = np.zeros(H) if D is None else D
    lam = np.zeros((b, H, P, N)) if dh_last is None else dh_last.astype(np.float64)
    mam = np.abs(lam)
    z = lambda *sh: (np.zeros(sh), np.zeros(sh))  # noqa: E731
    dx, mdx = z(*x.shape)
    dB, mdB = z(*Bm.shape)
    dC, mdC = z(*Cm.shape)
    ds, mds = z(b, L, H)
    dA, mdA = z(H)
    grp = lambda v: v.reshape(b, G, per, N).sum(2)  # noqa: E731
    for t in range(L - 1, -1, -1):
        c, k = _heads(Cm[:, t], per)[:, :, None], _heads(Bm[:, t], per)[:, :, None]
        u = dy[:, t][..., None] * c
        lam, mam = lam + u, mam + np.abs(u)
        lb, mlb = (lam * k).sum(-1), (mam * np.abs(k)).sum(-1)
        wt = w[:, t, :, None]
        dx[:, t], mdx[:, t] = wt * lb + d[:, None] * dy[:, t], np.abs(wt) * mlb + np.abs(d[:, None] * dy[:, t])
        dB[:, t] = grp((lam * (wt * x[:, t])[..., None]).sum(2))
        mdB[:, t] = grp((mam * np.abs(wt * x[:, t])[..., None]).sum(2))
        dC[:, t] = grp((S[t + 1] * dy[:, t][..., None]).sum(2))
        mdC[:, t] = grp((M[t + 1] * np.abs(dy[:, t])[..., None]).sum(2))
        et = e[:, t, :, None, None]
        ga, mga = (lam * et * S[t]).sum((-1, -2)), (mam * et * M[t]).sum((-1, -2))
        dw, mdw = (lb * x[:, t]).sum(-1), (mlb * np.abs(x[:, t])).sum(-1)
        ds[:, t] = A * ga + (0.0 if unit else dw)
        mds[:, t] = np.abs(A) * mga + (0.0 if unit else mdw)
        dA += (s[:, t] * ga).sum(0)
        mdA += (np.abs(s[:, t]) * mga).sum(0)
        lam, mam = et * lam, et * mam
    out = dict(dx=(dx, mdx), dBm=(dB, mdB), dCm=(dC, mdC), dA=(dA, mdA), dh0=(lam, mam),
               dD=((x * dy).sum((0, 1, 3)), np.abs(x * dy).sum((0, 1, 3))), ddelta=(ds * ds_dv, mds * ds_dv))
    out["ddelta_bias"] = tuple(v.sum((0, 1)) for v in out["ddelta"])
    return out


def rms(u, groups, eps):
    v = u.reshape(u.shape[0], groups, -1)
    return (v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)).reshape(u.shape)


def add_norm(x, r, weight, gamma, scale, eps):
    """out, r'."""
    k = scale * (1.0 if gamma is None else gamma)
    v = k * x + (0.0 if r is None else r)
    return rms(v, 1, eps) * weight, v


def silu(z):
    return z / (1.0 + np.exp(-z))


def gated_norm(y, z, weight, groups, after, eps):
    f = 1.0 if z is None else silu(z)
    return rms(y, groups, eps) * weight * f if after else rms(y * f, groups, eps) * weight


def rms_bwd(u, d, weight, groups, eps):
    """(du, |du|, dweight, |dweight|) for rms(u) * weight."""
    n = u.shape[0]
    v, dh = u.reshape(n, groups, -1), (d * weight).reshape(n, groups, -1)
    inv = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    hat = v * inv
    m, am = (dh * hat).mean(-1, keepdims=True), (np.abs(dh * hat)).mean(-1, keepdims=True)
    du, mdu = inv * (dh - hat * m), inv * (np.abs(dh) + np.abs(hat) * am)
    h = hat.reshape(u.shape)
    return du.reshape(u.shape), mdu.reshape(u.shape), (d * h).sum(0), np.abs(d * h).sum(0)
