"""Performance cases of the gated recurrence, the norm with an 8-bit output and
the products with 4-bit weights.

Each operator in its plain form (elementary torch operations in 32 bits,
rounded once at the end) and, with `own` set, through the framework's kernels:

  step   one token per sequence, the state advanced in place (gated_state_update)
  scan   y and the final state of a prompt (gated_scan_fwd)
  train  a training pass: y and every gradient (gated_scan_fwd, gated_scan_bwd)
  norm8  residual add, residual scale and RMS norm, the result in 8 bits with
         one scale per row (add_norm_q8_fwd)
  q4     products of few rows with 4-bit weights and group scales (q4_linear),
         the rows in 16 or 32 bits or as norm8 leaves them

The recurrence, per sequence and channel, with r = sigmoid(gate_a + bias_a) and
i = sigmoid(gate_x + bias_x):
  a_t = exp(A r_t),   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t
(with unit: the input term is i_t x_t).  A token that starts a sequence has
a_t = 0.  The 4-bit values are 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives
(codes 0 to 7, and 8 to 15), two in a byte, the lower one first.
"""
import math
import random  # noqa: F401  (the type of draw's argument)

import torch

own = False

EPS = 1e-5
TOP = 448.0  # largest 8-bit value (e4m3)
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one sequence's next token on a small layer: latency
        dict(name="gated_step_one", kind="step", batch=1, dim=1536, dtype="bf16", unit=False),
        # a full serving batch on a large layer: the state's bytes
        dict(name="gated_step_batch256", kind="step", batch=256, dim=5120, dtype="bf16", unit=False),
        # a prompt on a small layer, from the projection's packed row
        dict(name="gated_scan_small", kind="scan", batch=2, seqlen=2048, dim=1536, dtype="bf16", packed=True, unit=False,
             h0=False, starts=False),
        # prompts on a large layer
        dict(name="gated_scan_large", kind="scan", batch=8, seqlen=2048, dim=5120, dtype="bf16", packed=True, unit=False,
             h0=False, starts=False),
        # one long document: few rows, a long axis; continues from a state
        dict(name="gated_scan_long", kind="scan", batch=1, seqlen=65536, dim=1536, dtype="bf16", packed=False, unit=False,
             h0=True, starts=False),
        # training of the large layer on sequences packed one after another
        dict(name="gated_train_large", kind="train", batch=8, seqlen=2048, dim=5120, dtype="bf16", packed=True,
             unit=False, h0=False, starts=True),
        # training in fp32, odd sizes, from a state
        dict(name="gated_train_f32", kind="train", batch=3, seqlen=777, dim=1001, dtype="f32", packed=False, unit=True,
             h0=True, starts=False),
        # the norm before a layer: a serving batch (latency), and a prompt's tokens
        dict(name="norm8_serve", kind="norm8", rows=256, dim=2560, dtype="bf16", residual="f32", gamma=False),
        dict(name="norm8_prompt", kind="norm8", rows=16384, dim=2560, dtype="bf16", residual="f32", gamma=True),
        # the input projection of a large layer for one sequence's token
        dict(name="q4_one", kind="q4", rows=1, inner=2560, outer=10576, group=128, dtype="bf16"),
        # the projection back for a small batch, finer groups
        dict(name="q4_few", kind="q4", rows=16, inner=5120, outer=2560, group=32, dtype="bf16"),
        # the input projection for a full serving batch, from 8-bit rows
        dict(name="q4_batch256", kind="q4", rows=256, inner=2560, outer=10576, group=128, dtype="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "scan", "scan", "train", "train", "norm8", "q4", "q4"])
    if kind == "norm8":
        dim = _log(rng, 64, 8192)
        return dict(kind=kind, rows=_log(rng, 1, min(16384, 16384 * 2560 // dim)), dim=dim,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.choice(["f32", "same"]),
                    gamma=rng.random() < 0.5)
    if kind == "q4":
        group = rng.choice([32, 64, 128])
        inner = group * _log(rng, 2, 8192 // group)
        return dict(kind=kind, rows=_log(rng, 1, 256), inner=inner, outer=_log(rng, 16, 10576 * 2560 // max(inner, 2560)),
                    group=group, dtype=rng.choice(["bf16", "bf16", "e4m3", "e4m3", "f32"]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([_log(rng, 16, 5120), 8 * _log(rng, 8, 640)])
    if kind == "step":
        return dict(kind=kind, batch=_log(rng, 1, 512), dim=dim, dtype=dtype, unit=rng.random() < 0.3)
    most = 8 * 2048 * 5120 // dim // (2 if dtype == "f32" else 1)
    tokens = _log(rng, 16, min(65536 if kind == "scan" else 16384, most))
    batch = max(1, min(_log(rng, 1, 16), tokens // 16))
    return dict(kind=kind, batch=batch, seqlen=max(1, tokens // batch), dim=dim, dtype=dtype, packed=rng.random() < 0.5,
                unit=rng.random() < 0.3, h0=rng.random() < 0.5, starts=rng.random() < 0.4)


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _type(case)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    s = dict(case=case)
    if case["kind"] == "norm8":
        rows, dim = case["rows"], case["dim"]
        rt = torch.float32 if case["residual"] == "f32" else dt
        s.update(x=randn(rows, dim).to(dt), residual=(4 * randn(rows, dim)).to(rt), weight=1 + 0.1 * randn(dim),
                 gamma=0.5 + 0.1 * randn(dim) if case["gamma"] else None, scale=0.7)
        return s
    if case["kind"] == "q4":
        rows, k, n, group = case["rows"], case["inner"], case["outer"], case["group"]
        # codes as rounding normal weights leaves them, with the scale of each group's largest
        w = (torch.randn(n, k // group, group, device="cuda", generator=g) / math.sqrt(k))
        scales = (w.abs().amax(-1) / VALUES[-1]).to(torch.bfloat16)
        code = torch.bucketize(w.abs() / scales.float()[..., None],
                               torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda"))
        code = torch.where(w < 0, code + 8, code).reshape(n, k // 2, 2).to(torch.uint8)
        s.update(weight=code[..., 0] | (code[..., 1] << 4), scales=scales)
        x = 2 * randn(rows, k)
        if case["dtype"] == "e4m3":
            xs = x.abs().amax(-1) / TOP
            s.update(x=(x / xs[:, None]).to(torch.float8_e4m3fn), x_scale=xs)
        else:
            s.update(x=x.to(dt), x_scale=None)
        return s
    b, d = case["batch"], case["dim"]
    # decays of 0.9 to 0.999 per token where the gate is half open
    u = torch.rand(d, device="cuda", generator=g)
    s.update(A=4 * torch.log(0.9 + 0.099 * u), bias_a=0.5 * randn(d), bias_x=0.5 * randn(d))
    if case["kind"] == "step":
        s.update(h=randn(b, d), x=randn(b, d).to(dt), gate_a=randn(b, d).to(dt), gate_x=randn(b, d).to(dt))
        return s
    L = case["seqlen"]
    if case["packed"]:  # x and the gates as one row, the way a layer's projection writes them
        row = randn(b, L, 3 * d).to(dt)
        x, ga, gx = (row[..., k * d:(k + 1) * d] for k in range(3))
    else:
        x, ga, gx = (randn(b, L, d).to(dt) for _ in range(3))
    s.update(x=x, gate_a=ga, gate_x=gx, h0=randn(b, d) if case["h0"] else None, starts=None)
    if case["starts"]:  # documents of about 300 tokens
        s.update(starts=torch.rand(b, L, device="cuda", generator=g) < 1 / 300)
    if case["kind"] == "train":
        s.update(dy=randn(b, L, d).to(dt), dh_last=randn(b, d) if case["h0"] else None)
    return s


# ------------------------------------------------------------ plain forms --
def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dimension 1 from 0, by doubling."""
    L, n = a.shape[1], 1
    while n < L:
        u = torch.cat([u[:, :n], u[:, n:] + a[:, n:] * u[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return u


def _plain_gates(s, starts=None):
    """The gates r and i, the decay a and the factor b of the input term."""
    r, i = _sigmoid(s["gate_a"].float() + s["bias_a"]), _sigmoid(s["gate_x"].float() + s["bias_x"])
    v = s["A"] * r
    a = torch.exp(v)
    b = torch.ones_like(a) if s["case"]["unit"] else torch.sqrt(-torch.expm1(2 * v))
    if starts is not None:
        a, b = a.masked_fill(starts[..., None], 0.0), b.masked_fill(starts[..., None], 1.0)
    return r, i, a, b


def _plain_recurrence(s):
    case, dt = s["case"], s["x"].dtype
    x, starts = s["x"].float(), s["starts"]
    r, i, a, b = _plain_gates(s, starts)
    h0 = torch.zeros_like(x[:, 0]) if s["h0"] is None else s["h0"]
    u = b * i * x
    u[:, 0] += a[:, 0] * h0
    h = _scan(a, u)
    out = dict(y=h.to(dt), h_last=h[:, -1].clone())
    if case["kind"] == "scan":
        return out
    # the adjoint of h: lam_t = dy_t + a_{t+1} lam_{t+1}
    lam = s["dy"].float().clone()
    if s["dh_last"] is not None:
        lam[:, -1] += s["dh_last"]
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    lam = _scan(later.flip(1), lam.flip(1)).flip(1)
    dv = a * torch.cat([h0[:, None], h[:, :-1]], 1)
    if not case["unit"]:
        dv = dv - a * a / b * i * x
    dv = lam * dv
    dga = dv * s["A"] * r * (1 - r)
    db = lam * b * i
    dgx = db * x * (1 - i)
    out.update(dx=db.to(dt), dgate_a=dga.to(dt), dgate_x=dgx.to(dt), dA=(dv * r).sum((0, 1)), dbias_a=dga.sum((0, 1)),
               dbias_x=dgx.sum((0, 1)))
    if s["h0"] is not None:
        out["dh0"] = a[:, 0] * lam[:, 0]
    return out


def _plain_step(s):
    h = s["h"]
    _, i, a, b = _plain_gates(s)
    h.copy_(a * h + b * i * s["x"].float())
    return dict(y=h.to(s["x"].dtype), h=h)


def _plain_norm8(s):
    x, w, gamma = s["x"].float(), s["weight"], s["gamma"]
    r = s["residual"].float() + (s["scale"] * x if gamma is None else s["scale"] * gamma * x)
    out = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * w
    scale = out.abs().amax(-1) / TOP
    return dict(out=(out / scale[:, None]).to(torch.float8_e4m3fn), scale=scale, residual=r.to(s["residual"].dtype))


def _values(weight, dtype):
    """The 4-bit values of packed codes."""
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=weight.device, dtype=dtype)
    return table[torch.stack([weight & 15, weight >> 4], -1).flatten(-2).long()]


def _plain_q4(s):
    case = s["case"]
    w = _values(s["weight"], torch.float32).unflatten(-1, (-1, case["group"])) * s["scales"].float()[..., None]
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = x * s["x_scale"][:, None]
    return torch.matmul(x, w.flatten(-2).t()).to(_type(case))


def _run_plain(s):
    return dict(step=_plain_step, scan=_plain_recurrence, train=_plain_recurrence, norm8=_plain_norm8,
                q4=_plain_q4)[s["case"]["kind"]](s)


# ------------------------------------------------------ the own kernels --
def _run_own(s):
    from selective_state_space_63_amd import gated, q4

    case = s["case"]
    kind = case["kind"]
    if kind == "step":
        y = gated.gated_state_update(s["h"], s["x"], s["gate_a"], s["gate_x"], s["A"], bias_a=s["bias_a"],
                                     bias_x=s["bias_x"], unit_input=case["unit"])
        return dict(y=y, h=s["h"])
    if kind == "norm8":
        out, scale, residual = q4.add_norm_q8_fwd(s["x"], s["weight"], residual=s["residual"], gamma=s["gamma"],
                                                  scale=s["scale"], eps=EPS)
        return dict(out=out, scale=scale, residual=residual)
    if kind == "q4":
        return q4.q4_linear(s["x"], s["weight"], s["scales"], x_scale=s["x_scale"])
    opts = dict(bias_a=s["bias_a"], bias_x=s["bias_x"], h0=s["h0"], starts=s["starts"], unit_input=case["unit"])
    if kind == "scan":
        y, h_last = gated.gated_scan_fwd(s["x"], s["gate_a"], s["gate_x"], s["A"], return_last_state=True, **opts)
        return dict(y=y, h_last=h_last)
    y, h_last, states = gated.gated_scan_fwd(s["x"], s["gate_a"], s["gate_x"], s["A"], return_last_state=True,
                                             return_states=True, **opts)
    g = gated.gated_scan_bwd(s["x"], s["gate_a"], s["gate_x"], s["A"], s["dy"], dh_last=s["dh_last"], states=states,
                             **opts)
    return dict(g, y=y, h_last=h_last)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ work --
def work(case):
    e = dict(bf16=2, f32=4, e4m3=1)[case["dtype"]]
    kind = case["kind"]
    if kind == "norm8":
        n, r = case["rows"] * case["dim"], 4 if case["residual"] == "f32" else e
        return dict(bytes=n * (e + 2 * r + 1) + 4 * case["rows"] + 8 * case["dim"], flops=10 * n)
    if kind == "q4":
        m, k, n = case["rows"], case["inner"], case["outer"]
        return dict(bytes=n * k // 2 + 2 * n * (k // case["group"]) + m * k * e + m * n * max(e, 2), flops=2 * m * k * n)
    b, d = case["batch"], case["dim"]
    if kind == "step":
        return dict(bytes=b * d * (8 + 4 * e) + 12 * d, flops=25 * b * d)
    n = b * case["seqlen"] * d
    mask = b * case["seqlen"] if case["starts"] else 0
    state = 4 * b * d * (2 if case["h0"] else 1)
    # x, both gates -> y; then dy, and x and the gates again -> dx and the gates' gradients
    if kind == "scan":
        return dict(bytes=4 * e * n + mask + state, flops=25 * n)
    return dict(bytes=11 * e * n + 2 * mask + 2 * state, flops=80 * n)


# ---------------------------------------------------- the definitions, 64 bits --
def _d(t):
    return None if t is None else t.double()


def _exact_recurrence(s):
    """Token by token, forwards and, for a training pass, backwards."""
    case = s["case"]
    step = case["kind"] == "step"
    x, ga, gx, A = (_d(s[k]) for k in ("x", "gate_a", "gate_x", "A"))
    r, i = torch.sigmoid(ga + _d(s["bias_a"])), torch.sigmoid(gx + _d(s["bias_x"]))
    v = r * A
    a = torch.exp(v)
    # 1 - a^2 as -2 sinh(v) e^v
    b = torch.ones_like(a) if case["unit"] else torch.sqrt(-2 * torch.sinh(v) * a)
    if step:
        h = a * _d(s["h"]) + b * i * x
        return dict(y=h, h=h)
    first = torch.zeros_like(a[..., :1], dtype=torch.bool) if s["starts"] is None else s["starts"][..., None]
    a, b = torch.where(first, 0.0, a), torch.where(first, 1.0, b)
    u = b * i * x
    h0 = torch.zeros_like(x[:, 0]) if s["h0"] is None else _d(s["h0"])
    y, h = torch.empty_like(x), h0
    for t in range(x.shape[1]):
        h = torch.addcmul(u[:, t], a[:, t], h, out=y[:, t])
    out = dict(y=y, h_last=y[:, -1])
    if case["kind"] == "scan":
        return out
    lam = _d(s["dy"]).clone()
    if s["dh_last"] is not None:
        lam[:, -1] += _d(s["dh_last"])
    for t in range(x.shape[1] - 2, -1, -1):
        lam[:, t].addcmul_(a[:, t + 1], lam[:, t + 1])
    before = torch.cat([h0[:, None], y[:, :-1]], 1)
    dv = lam * before * a
    if not case["unit"]:
        dv = dv + torch.where(first, 0.0, lam * i * x * (b - 1 / b))  # db/dv = -a^2 / b = (b^2 - 1) / b
    dr, di = dv * A, lam * b * x
    dga, dgx = dr * r * (1 - r), di * i * (1 - i)
    out.update(dx=lam * b * i, dgate_a=dga, dgate_x=dgx, dA=(dv * r).sum((0, 1)), dbias_a=dga.sum((0, 1)),
               dbias_x=dgx.sum((0, 1)))
    if s["h0"] is not None:
        out["dh0"] = a[:, 0] * lam[:, 0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm8":
        x, w = _d(s["x"]), _d(s["weight"])
        r = _d(s["residual"]) + s["scale"] * (1.0 if s["gamma"] is None else _d(s["gamma"])) * x
        out = w * r / torch.sqrt((r * r).sum(-1, keepdim=True) / case["dim"] + EPS)
        scale = out.abs().max(-1).values / TOP
        return dict(out=out / scale[:, None], scale=scale, residual=r)
    if kind == "q4":
        # the sums over each group on their own, then the scales
        k, group = case["inner"], case["group"]
        y = torch.zeros(case["rows"], case["outer"], dtype=torch.float64, device="cuda")
        for at in range(0, k, group):
            w = _values(s["weight"][:, at // 2:(at + group) // 2], torch.float64)
            y += torch.matmul(_d(s["x"][:, at:at + group]), w.t().contiguous()) * _d(s["scales"][:, at // group])
        return y if s["x_scale"] is None else y * _d(s["x_scale"])[:, None]
    return _exact_recurrence(s)
