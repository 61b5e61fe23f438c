"""The selective state-space mixer's operators and the norm in front of it, as
measurable cases: inputs, one pass of each operator (the library's entry points
where `own` is set, elementary torch operations otherwise), its definition in
64 bits, and the bytes and operations it cannot do without.

Kinds of case:
  fwd       the selective scan over equal-length sequences (training, prefill)
  varlen    packed prompts of any length with the causal convolution fused in,
            states and windows in pools
  step      one token per sequence on the same pools
  bwd       the gradients of the scan
  conv_bwd  the gradients of the causal convolution with SiLU
  norm      residual addition and RMSNorm with an 8-bit output and scales
  norm_bwd  the gradients of residual addition and RMSNorm
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one interactive session: a handful of sequences, where latency counts
        dict(name="step_few", kind="step", N=4, D=2048, n=16, dtype="bf16"),
        # the serving loop's full batch (1,280 sequences), pages in any order
        dict(name="step_full", kind="step", N=1280, D=4096, n=16, dtype="bf16"),
        # prompts of a busy server: lengths from one token to thousands, packed
        dict(name="varlen_ragged", kind="varlen", lens="4096,1,777,2048,0,63,3000,129,1500,17,2500,1200,640,33",
             D=4096, n=16, dtype="bf16"),
        # the training shape: eight sequences of 2,048 tokens
        dict(name="fwd_train", kind="fwd", B=8, T=2048, D=2048, n=16, z=True, h0=False, dtype="bf16"),
        # a short odd call in the validation type, without the output gate
        dict(name="fwd_small_fp32", kind="fwd", B=2, T=333, D=516, n=8, z=False, h0=True, dtype="fp32"),
        # a training step's gradients
        dict(name="bwd_train", kind="bwd", B=4, T=2048, D=2048, n=16, z=True, h0=False, dtype="bf16"),
        # gradients with a state carried in and out (truncated sequences), odd sizes
        dict(name="bwd_small_fp32", kind="bwd", B=2, T=301, D=516, n=16, z=True, h0=True, dtype="fp32"),
        # the convolution's gradients at the training shape
        dict(name="conv_bwd_train", kind="conv_bwd", B=8, T=2048, D=4096, dtype="bf16"),
        dict(name="conv_bwd_small", kind="conv_bwd", B=3, T=53, D=1032, dtype="bf16"),
        # a decode batch's norm in front of an 8-bit projection, blocks of 128
        dict(name="norm_few", kind="norm", rows=8, D=4096, group=128, dtype="bf16"),
        # a prefill batch's, one scale a row
        dict(name="norm_prefill", kind="norm", rows=16384, D=4096, group=0, dtype="bf16"),
        # training
        dict(name="norm_bwd_train", kind="norm_bwd", rows=16384, D=2048, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _channels(rng, lo, hi):
    return max(8, _log_int(rng, lo, hi) // 8 * 8)


def draw(rng):
    """A case of the listed ones' ranges: any kind, sizes over their logarithm,
    the product of the sizes capped at that of the largest listed case."""
    kind = rng.choice(["fwd", "varlen", "step", "bwd", "conv_bwd", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind in ("fwd", "bwd"):
        B, D, n = _log_int(rng, 1, 8), _channels(rng, 64, 4096), rng.choice([8, 16, 16, 32])
        cap = (1 << 27) if kind == "bwd" else (1 << 28)
        T = _log_int(rng, 1, max(2, min(8192, cap // (B * D * n))))
        return dict(kind=kind, B=B, T=T, D=D, n=n, z=rng.random() < 0.7, h0=rng.random() < 0.5, dtype=dtype)
    if kind == "varlen":
        D, n = _channels(rng, 64, 4096), rng.choice([8, 16, 16, 32])
        room = min(8192, (1 << 28) // (D * n))
        lens = [min(_log_int(rng, 1, 4096), room) for _ in range(rng.randint(1, 16))]
        while len(lens) > 1 and sum(lens) > room:
            lens.pop()
        return dict(kind=kind, lens=",".join(str(v) for v in lens), D=D, n=n, dtype=dtype)
    if kind == "step":
        return dict(kind=kind, N=_log_int(rng, 1, 1280), D=_channels(rng, 64, 4096), n=rng.choice([8, 16, 16]),
                    dtype=dtype)
    if kind == "conv_bwd":
        B, T, D = _log_int(rng, 1, 8), _log_int(rng, 1, 2048), _channels(rng, 64, 4096)
        return dict(kind=kind, B=B, T=T, D=D, dtype="bf16" if B * T * D > 1 << 25 else dtype)
    rows, D = _log_int(rng, 1, 16384), _channels(rng, 64, 8192)
    rows = max(1, min(rows, (1 << 25) // D))
    if kind == "norm":
        return dict(kind=kind, rows=rows, D=D, group=rng.choice([0, 128]), dtype=dtype)
    return dict(kind=kind, rows=rows, D=D, dtype=dtype)


# ------------------------------------------------------------------ inputs
class _Gen:
    """Seeded normal and uniform tensors on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device="cuda") * std).to(dtype)

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=self.g, device="cuda") * (hi - lo) + lo


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _scan_inputs(g, lead, D, n, dt, gate):
    """What a layer's projections and parameters give the scan: steps whose
    softplus spreads over 1e-3 .. 1e-1, rates -1 .. -n, unit B and C."""
    step = torch.exp(g.uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
    s = dict(x=g.normal(*lead, D, dtype=dt), dt=g.normal(*lead, D, std=0.7, dtype=dt),
             A=-torch.arange(1, n + 1, device="cuda").float() * torch.exp(g.normal(D, n, std=0.1)),
             Bm=g.normal(*lead, n, dtype=dt), Cm=g.normal(*lead, n, dtype=dt), skip=1.0 + g.normal(D, std=0.1),
             dt_bias=step + torch.log(-torch.expm1(-step)), z=None)
    if gate:
        s["z"] = g.normal(*lead, D, dtype=dt)
    return s


def _conv_inputs(g, D):
    return dict(conv_w=g.normal(D, 4, std=0.5), conv_b=g.normal(D, std=0.1))


def prepare(case, seed):
    g, dt, kind = _Gen(seed), _dtype(case), case["kind"]
    if kind in ("fwd", "bwd"):
        B, T, D, n = case["B"], case["T"], case["D"], case["n"]
        s = _scan_inputs(g, (B, T), D, n, dt, case["z"])
        s["h0"] = g.normal(B, D, n, std=0.1) if case["h0"] else None
        if kind == "bwd":
            s["dy"] = g.normal(B, T, D, dtype=dt)
            s["dhT"] = g.normal(B, D, n, std=0.1) if case["h0"] else None
    elif kind == "varlen":
        D, n = case["D"], case["n"]
        lens = [int(v) for v in case["lens"].split(",")]
        cu = [0]
        for v in lens:
            cu.append(cu[-1] + v)
        s = _scan_inputs(g, (cu[-1],), D, n, dt, True)
        s.update(_conv_inputs(g, D))
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["slots"] = torch.randperm(len(lens) + 3, generator=g.g, device="cuda")[: len(lens)].to(torch.int32)
        s["pool"] = g.normal(len(lens) + 3, D, n, std=0.1)
        s["win"] = g.normal(len(lens) + 3, 4, D)
    elif kind == "step":
        N, D, n = case["N"], case["D"], case["n"]
        s = _scan_inputs(g, (N,), D, n, dt, True)
        s.update(_conv_inputs(g, D))
        s["slots"] = torch.randperm(N, generator=g.g, device="cuda").to(torch.int32)
        s["pool"] = g.normal(N, D, n, std=0.1)
        s["win"] = g.normal(N, 4, D)
    elif kind == "conv_bwd":
        B, T, D = case["B"], case["T"], case["D"]
        s = _conv_inputs(g, D)
        s.update(x=g.normal(B, T, D, dtype=dt), dy=g.normal(B, T, D, dtype=dt), win=g.normal(B, 4, D))
    else:
        rows, D = case["rows"], case["D"]
        s = dict(x=g.normal(rows, D, dtype=dt), w=1.0 + g.normal(D, std=0.1))
        if kind == "norm":
            s["res"] = g.normal(rows, D, std=3.0, dtype=dt)
            s["group"] = case["group"]
        else:
            s["dy"] = g.normal(rows, D, dtype=dt)
            s["ds"] = g.normal(rows, D, dtype=dt)
    s["kind"] = kind
    return s


# ------------------------------------------------------------- plain forms
def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))


def _silu(v):
    return v / (1 + torch.exp(-v))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 (h_{-1} = 0), by doubling: after
    the step of stride k every (a, b) spans its last 2k tokens."""
    k, T = 1, a.shape[1]
    while k < T:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        if 2 * k < T:
            a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _discretise(s, u):
    """The steps and the per-token decay and input of every (channel, state)."""
    v = s["dt"].float() + s["dt_bias"]
    delta = _softplus(v)
    a = torch.exp(delta[..., None] * s["A"])
    b = (delta * u)[..., None] * s["Bm"].float()[..., None, :]
    return v, delta, a, b


def _readout(s, u, h):
    y = (h * s["Cm"].float()[..., None, :]).sum(-1) + s["skip"] * u
    return y if s["z"] is None else y * _silu(s["z"].float())


def _plain_fwd(s):
    x = s["x"].float()
    _, _, a, b = _discretise(s, x)
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    h = _scan(a, b)
    return {"y": _readout(s, x, h).to(s["x"].dtype), "hT": h[:, -1].clone()}


def _plain_varlen(s):
    x, cu, slots = s["x"].float(), s["cu"].long(), s["slots"].long()
    lens = cu[1:] - cu[:-1]
    live = torch.nonzero(lens > 0)[:, 0]
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device=x.device), lens)
    first, slot = cu[:-1][seq], slots[seq]
    t = torch.arange(x.shape[0], device=x.device)

    def at(pos, first, slot):   # the input at a position, from the window before the sequence's first token
        inside = pos >= first
        row = (4 + pos - first).clamp(0, 3)
        return torch.where(inside[:, None], x[pos.clamp(min=0)], s["win"][slot, row])

    acc = s["conv_b"] + sum(s["conv_w"][:, j] * at(t - 3 + j, first, slot) for j in range(4))
    u = _silu(acc)
    _, _, a, b = _discretise(s, u)
    start = cu[:-1][live]
    b[start] += a[start] * s["pool"][slots[live]]
    a[start] = 0
    h = _scan(a[None], b[None])[0]
    y = _readout(s, u, h).to(s["x"].dtype)
    end, sl = cu[1:][live], slots[live]
    win = torch.stack([at(end - 4 + k, start, sl) for k in range(4)], 1)
    s["pool"][sl] = h[end - 1]
    s["win"][sl] = win
    return {"y": y, "pool": s["pool"], "win": s["win"]}


def _plain_step(s):
    x, slots = s["x"].float(), s["slots"].long()
    win = torch.cat([s["win"][slots][:, 1:], x[:, None]], 1)
    u = _silu((win * s["conv_w"].t()).sum(1) + s["conv_b"])
    _, _, a, b = _discretise(s, u)
    h = a * s["pool"][slots] + b
    s["pool"][slots] = h
    s["win"][slots] = win
    return {"y": _readout(s, u, h).to(s["x"].dtype), "pool": s["pool"], "win": s["win"]}


def _plain_bwd(s):
    x, dy, dt = s["x"].float(), s["dy"].float(), s["x"].dtype
    v, delta, a, b = _discretise(s, x)
    Bm, Cm = s["Bm"].float()[..., None, :], s["Cm"].float()[..., None, :]
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    h = _scan(a, b)
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sig = 1 / (1 + torch.exp(-z))
        y = (h * Cm).sum(-1) + s["skip"] * x
        out["dz"] = (dy * y * sig * (1 + z * (1 - sig))).to(dt)
        dy = dy * z * sig
    # G_t = C_t dy_t + a_{t+1} G_{t+1}, from the last token back
    c = dy[..., None] * Cm
    if s["dhT"] is not None:
        c[:, -1] += s["dhT"]
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    G = _scan(later.flip(1), c.flip(1)).flip(1)
    prev = torch.cat([(torch.zeros_like(h[:, 0]) if s["h0"] is None else s["h0"])[:, None], h[:, :-1]], 1)
    da = G * prev * a
    gb = (G * Bm).sum(-1)
    ddelta = (da * s["A"]).sum(-1) + gb * x
    dv = ddelta * torch.where(v > 20, torch.ones_like(v), 1 / (1 + torch.exp(-v)))
    out["dx"] = (gb * delta + s["skip"] * dy).to(dt)
    out["ddt"] = dv.to(dt)
    out["dA"] = (da * delta[..., None]).sum((0, 1))
    out["dB"] = (G * (delta * x)[..., None]).sum(2).to(dt)
    out["dC"] = (dy[..., None] * h).sum(2).to(dt)
    out["dskip"] = (dy * x).sum((0, 1))
    out["ddt_bias"] = dv.sum((0, 1))
    if s["h0"] is not None:
        out["dh0"] = a[:, 0] * G[:, 0]
    return out


def _plain_conv_bwd(s):
    x, dy, w = s["x"].float(), s["dy"].float(), s["conv_w"]
    T = x.shape[1]
    past = torch.cat([s["win"][:, 1:], x], 1)
    acc = s["conv_b"] + sum(w[:, j] * past[:, j:j + T] for j in range(4))
    sig = 1 / (1 + torch.exp(-acc))
    dp = dy * sig * (1 + acc * (1 - sig))
    ahead = torch.cat([dp, torch.zeros_like(dp[:, :1]).expand(-1, 3, -1)], 1)
    dx = sum(w[:, j] * ahead[:, 3 - j:3 - j + T] for j in range(4))
    dw = torch.stack([(dp * past[:, j:j + T]).sum((0, 1)) for j in range(4)], 1)
    return {"dx": dx.to(s["x"].dtype), "dw": dw, "db": dp.sum((0, 1))}


def _groups(y, group):
    """[rows, D] as [rows, groups, group], the last group filled with zeros."""
    D = y.shape[1]
    group = group or D
    pad = -D % group
    return torch.cat([y, y.new_zeros(y.shape[0], pad)], 1).view(y.shape[0], -1, group)


def _plain_norm(s):
    r = s["x"].float() + s["res"].float()
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["w"]
    blocks = _groups(y, s["group"])
    top = blocks.abs().amax(2, keepdim=True)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    q = (blocks / scale).clamp(-E4M3_MAX, E4M3_MAX).reshape(y.shape[0], -1)[:, : y.shape[1]]
    return {"res": r.to(s["x"].dtype), "y8": q.to(torch.float8_e4m3fn), "scale": scale[:, :, 0]}


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    xn, g = x * r, dy * s["w"]
    dx = r * (g - xn * (g * xn).mean(1, keepdim=True)) + s["ds"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xn).sum(0)}


_PLAIN = dict(fwd=_plain_fwd, varlen=_plain_varlen, step=_plain_step, bwd=_plain_bwd, conv_bwd=_plain_conv_bwd,
              norm=_plain_norm, norm_bwd=_plain_norm_bwd)


# ------------------------------------------------- the library's operators
def _own(s):
    import linear_attention_chunk_gb300 as gla
    kind = s["kind"]
    if kind == "fwd":
        y, hT = gla.gla_ssm_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["skip"], s["z"], s["dt_bias"], s["h0"])
        return {"y": y, "hT": hT}
    if kind == "varlen":
        y = gla.gla_ssm_varlen(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["cu"], s["pool"], s["skip"], s["z"],
                               s["dt_bias"], s["slots"], conv_w=s["conv_w"], conv_b=s["conv_b"], win_pool=s["win"])
        return {"y": y, "pool": s["pool"], "win": s["win"]}
    if kind == "step":
        y = gla.gla_ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["pool"], s["skip"], s["z"], s["dt_bias"],
                             s["slots"], conv_w=s["conv_w"], conv_b=s["conv_b"], win_pool=s["win"])
        return {"y": y, "pool": s["pool"], "win": s["win"]}
    if kind == "bwd":
        names = ("dx", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias", "dh0")
        got = gla.gla_ssm_bwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], s["skip"], s["z"], s["dt_bias"],
                              s["h0"], s["dhT"], want_dh0=s["h0"] is not None)
        return {k: v for k, v in zip(names, got) if v is not None}
    if kind == "conv_bwd":
        dx, dw, db = gla.gla_conv1d_bwd(s["x"], s["conv_w"], s["conv_b"], s["dy"], s["win"])
        return {"dx": dx, "dw": dw, "db": db}
    if kind == "norm":
        y8, scale, r = gla.gla_rmsnorm_q8(s["x"], s["w"], s["res"], EPS, s["group"])
        return {"res": r, "y8": y8, "scale": scale}
    dx, dw = gla.gla_rmsnorm_bwd(s["x"], s["w"], s["dy"], s["ds"], EPS)
    return {"dx": dx, "dw": dw}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["kind"]](state)


# ------------------------------------------------------ floors of the work
def work(case):
    """Every input read once and every output written once. Operations per
    (token, channel, state): the decay's product and exponential, the input's
    product, two multiply-adds forward; the adjoint's, the three sums' and the
    parameters' multiply-adds on top of those backward."""
    e, kind, D = (2 if case["dtype"] == "bf16" else 4), case["kind"], case["D"]
    if kind in ("fwd", "bwd"):
        rows, n, gate = case["B"] * case["T"], case["n"], 1 if case["z"] else 0
        states = case["B"] * D * n * 4
        if kind == "fwd":
            return {"bytes": rows * D * e * (3 + gate) + rows * 2 * n * e + D * n * 4 + states * (2 if case["h0"] else 1),
                    "flops": rows * D * (7 * n + 10)}
        return {"bytes": rows * D * e * (5 + 2 * gate) + rows * 4 * n * e + 2 * D * n * 4 + states * (3 if case["h0"] else 0),
                "flops": rows * D * (24 * n + 20)}
    if kind == "varlen":
        lens = [int(v) for v in case["lens"].split(",")]
        rows, n, live = sum(lens), case["n"], sum(v > 0 for v in lens)
        return {"bytes": rows * D * e * 4 + rows * 2 * n * e + D * n * 4 + live * D * (2 * n + 7) * 4,
                "flops": rows * D * (7 * n + 22)}
    if kind == "step":
        N, n = case["N"], case["n"]
        return {"bytes": N * D * e * 4 + N * 2 * n * e + D * n * 4 + N * D * (2 * n + 7) * 4, "flops": N * D * (7 * n + 22)}
    if kind == "conv_bwd":
        rows = case["B"] * case["T"]
        return {"bytes": rows * D * e * 3 + case["B"] * 3 * D * 4 + 2 * D * 5 * 4, "flops": rows * D * 34}
    rows = case["rows"]
    if kind == "norm":
        groups = 1 if not case["group"] else -(-D // case["group"])
        return {"bytes": rows * D * (3 * e + 1) + rows * groups * 4 + D * 4, "flops": rows * D * 8}
    return {"bytes": rows * D * e * 4 + 2 * D * 4, "flops": rows * D * 11}


# ------------------------------------------------- the definition, 64 bits
def _d(t):
    return None if t is None else t.double()


def _march(u, delta, A, Bm, h):
    """The recurrence token by token: yields the state after each token."""
    for t in range(u.shape[1]):
        h = torch.exp(delta[:, t, :, None] * A) * h + (delta[:, t] * u[:, t])[..., None] * Bm[:, t, None, :]
        yield t, h


def _exact_delta(dt, bias):
    v = _d(dt) + _d(bias)
    return v, torch.logaddexp(v, torch.zeros_like(v))


def _exact_scan(u, s, h, take=slice(None)):
    """y and the last state of sequences [B, T, D] from the state h."""
    _, delta = _exact_delta(s["dt"][take], s["dt_bias"])
    Bm, Cm, A = _d(s["Bm"][take]), _d(s["Cm"][take]), _d(s["A"])
    if u.dim() == 2:
        u, delta, Bm, Cm = u[None], delta[None], Bm[None], Cm[None]
    y = torch.empty_like(u)
    for t, h in _march(u, delta, A, Bm, h):
        y[:, t] = (h * Cm[:, t, None, :]).sum(-1)
    y += _d(s["skip"]) * u
    if s["z"] is not None:
        z = _d(s["z"][take])
        y = y * (z * torch.sigmoid(z))
    return y, h


def _exact_conv(rows, s):
    """SiLU of the width-4 filter over [..., 3 + T, D] rows, oldest first."""
    T, w = rows.shape[-2] - 3, _d(s["conv_w"])
    acc = _d(s["conv_b"]) + sum(rows[..., j:j + T, :] * w[:, j] for j in range(4))
    return acc * torch.sigmoid(acc), acc


def _exact_bwd(s):
    x, dy = _d(s["x"]), _d(s["dy"])
    Bm, Cm, A = _d(s["Bm"]), _d(s["Cm"]), _d(s["A"])
    v, delta = _exact_delta(s["dt"], s["dt_bias"])
    B, T, D = x.shape
    n = A.shape[1]
    h0 = torch.zeros(B, D, n, dtype=torch.float64, device=x.device) if s["h0"] is None else _d(s["h0"])
    hs = torch.empty(T + 1, B, D, n, dtype=torch.float64, device=x.device)
    hs[0] = h0
    for t, h in _march(x, delta, A, Bm, h0):
        hs[t + 1] = h
    out = {}
    if s["z"] is not None:
        z = _d(s["z"])
        gate = torch.sigmoid(z)
        y = torch.einsum("tbdn,btn->btd", hs[1:], Cm) + _d(s["skip"]) * x
        out["dz"] = dy * y * (gate + z * gate * (1 - gate))
        dy = dy * z * gate
    G = torch.zeros_like(h0) if s["dhT"] is None else _d(s["dhT"])
    gb, ga = torch.empty_like(x), torch.empty_like(x)
    dB, dC, dA = torch.empty_like(Bm), torch.empty_like(Cm), torch.zeros_like(A)
    for t in reversed(range(T)):
        G = G + dy[:, t, :, None] * Cm[:, t, None, :]
        dC[:, t] = (dy[:, t, :, None] * hs[t + 1]).sum(1)
        dB[:, t] = (G * (delta[:, t] * x[:, t])[..., None]).sum(1)
        gb[:, t] = (G * Bm[:, t, None, :]).sum(-1)
        G = G * torch.exp(delta[:, t, :, None] * A)
        da = G * hs[t]
        ga[:, t] = (da * A).sum(-1)
        dA += (da * delta[:, t, :, None]).sum(0)
    dv = (ga + gb * x) * torch.sigmoid(v)
    out.update(dx=gb * delta + _d(s["skip"]) * dy, ddt=dv, dA=dA, dB=dB, dC=dC, dskip=(dy * x).sum((0, 1)),
               ddt_bias=dv.sum((0, 1)))
    if s["h0"] is not None:
        out["dh0"] = G
    return out


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    if kind == "fwd":
        h0 = _d(s["h0"]) if s["h0"] is not None else torch.zeros(case["B"], case["D"], case["n"], dtype=torch.float64,
                                                                 device="cuda")
        y, h = _exact_scan(_d(s["x"]), s, h0)
        return {"y": y, "hT": h}
    if kind == "varlen":
        cu, slots = s["cu"].tolist(), s["slots"].tolist()
        y, pool, win = torch.empty_like(s["x"], dtype=torch.float64), _d(s["pool"]), _d(s["win"])
        for i, slot in enumerate(slots):
            lo, hi = cu[i], cu[i + 1]
            if hi > lo:
                rows = torch.cat([win[slot, 1:], _d(s["x"][lo:hi])])
                got, h = _exact_scan(_exact_conv(rows, s)[0], s, pool[slot][None], slice(lo, hi))
                y[lo:hi], pool[slot] = got[0], h[0]
                win[slot] = torch.cat([win[slot, :1], rows])[-4:]
        return {"y": y, "pool": pool, "win": win}
    if kind == "step":
        slots = s["slots"].long()
        pool, win = _d(s["pool"]), _d(s["win"])
        rows = torch.cat([win[slots, 1:], _d(s["x"])[:, None]], 1)
        one = {k: (v[:, None] if k in ("dt", "Bm", "Cm", "z") else v) for k, v in s.items() if k != "slots"}
        y, h = _exact_scan(_exact_conv(rows, s)[0], one, pool[slots])
        pool[slots], win[slots] = h, rows
        return {"y": y[:, 0], "pool": pool, "win": win}
    if kind == "bwd":
        return _exact_bwd(s)
    if kind == "conv_bwd":
        x, dy, w = _d(s["x"]), _d(s["dy"]), _d(s["conv_w"])
        B, T, D = x.shape
        rows = torch.cat([_d(s["win"])[:, 1:], x], 1)
        _, acc = _exact_conv(rows, s)
        gate = torch.sigmoid(acc)
        dacc = dy * (gate + acc * gate * (1 - gate))
        drows = torch.zeros_like(rows)
        for j in range(4):
            drows[:, j:j + T] += dacc * w[:, j]
        dw = torch.stack([torch.einsum("btd,btd->d", dacc, rows[:, j:j + T]) for j in range(4)], 1)
        return {"dx": drows[:, 3:], "dw": dw, "db": dacc.sum((0, 1))}
    x = _d(s["x"]) + (_d(s["res"]) if kind == "norm" else 0)
    ms = x.square().mean(1, keepdim=True) + EPS
    if kind == "norm":
        y = x / ms.sqrt() * _d(s["w"])
        group = s["group"] or y.shape[1]
        parts = y.split(group, 1)
        scales = [p.abs().amax(1, keepdim=True) / E4M3_MAX for p in parts]
        return {"res": x, "y8": torch.cat([p / q for p, q in zip(parts, scales)], 1), "scale": torch.cat(scales, 1)}
    g = _d(s["dy"]) * _d(s["w"])
    dx = g / ms.sqrt() - x * (g * x).mean(1, keepdim=True) / ms ** 1.5
    return {"dx": dx + _d(s["ds"]), "dw": (_d(s["dy"]) * x / ms.sqrt()).sum(0)}
