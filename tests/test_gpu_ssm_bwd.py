"""The gradients of the selective state-space scan (gla_ssm_bwd) on the GPU:
against autograd through the definition in float64, against differences of the
library's own forward, on the edges of its tiles and segments, and a training
pass and a serving pass that use the operators together.

Tolerances follow ssm_plain: every output is a sum of products of decays
(off by STEP relative a token), and is held to STEP * tokens * (the same sum
of absolute values) plus half a step of its type. The sums of absolute values
are the same gradients of a scan whose inputs are all positive and whose
gates' slopes are bounded by 1.1 (SiLU', and SiLU(z) <= |z|)."""
import pytest
import torch

import ssm_plain as plain
from ssm_plain import F64, STEP, d, half_step
from test_gpu_ssm import BF, FP, call_fwd, inputs

pytestmark = pytest.mark.gpu
NAMES = ("dx", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias", "dh0")


@pytest.fixture(scope="module")
def gla():
    import linear_attention_chunk_gb300 as m
    from linear_attention_chunk_gb300.build import build
    build()
    return m


def extras(s, state, seed):
    B, T, D = s["x"].shape
    N = s["A"].shape[1]
    g = torch.Generator().manual_seed(seed)
    dy = torch.randn(B, T, D, generator=g).to(s["x"].dtype).cuda()
    if not state:
        return dy, None, None
    return dy, torch.randn(B, D, N, generator=g).cuda(), torch.randn(B, D, N, generator=g).cuda()


def call(gla, s, dy, h0, dhT, **kw):
    return dict(zip(NAMES, gla.gla_ssm_bwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], dy, s["skip"], s["z"],
                                           s["dt_bias"], h0, dhT, **kw)))


def reference(s, dy, h0, dhT, soft=True):
    """The gradients in float64 and the sums of absolute values behind them."""
    x, dt, A, Bm, Cm, g = (d(v) for v in (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], dy))
    B, T, D = x.shape
    N = A.shape[1]
    skip = torch.zeros(D, dtype=F64) if s["skip"] is None else d(s["skip"])
    v = dt + (0 if s["dt_bias"] is None else d(s["dt_bias"]))
    delta = plain.softplus(v) if soft else v
    slope = torch.sigmoid(v) if soft else torch.ones_like(v)
    h0 = torch.zeros(B, D, N, dtype=F64) if h0 is None else d(h0)
    dhT = torch.zeros(B, D, N, dtype=F64) if dhT is None else d(dhT)
    a = torch.exp(delta[..., None] * A)

    def run(x, delta_u, Bm, Cm, g, skip, h, c, A, z, dy, y_slope):
        hs = [h]
        for t in range(T):
            hs.append(a[:, t] * hs[-1] + (delta_u[:, t] * x[:, t])[..., None] * Bm[:, t, None])
        o = {k: torch.zeros(B, T, D, dtype=F64) for k in ("dx", "ddt", "dz")}
        o.update(dB=torch.zeros(B, T, N, dtype=F64), dC=torch.zeros(B, T, N, dtype=F64), dA=torch.zeros(D, N, dtype=F64))
        for t in reversed(range(T)):
            G = g[:, t, :, None] * Cm[:, t, None] + c
            o["dC"][:, t] = (g[:, t, :, None] * hs[t + 1]).sum(1)
            o["dB"][:, t] = ((delta_u[:, t] * x[:, t])[..., None] * G).sum(1)
            gb = (G * Bm[:, t, None]).sum(-1)
            c = a[:, t] * G
            P = c * hs[t]
            o["dA"] += (P * delta_u[:, t][..., None]).sum(0)
            o["ddt"][:, t] = ((P * A).sum(-1) + gb * x[:, t]) * slope[:, t]
            o["dx"][:, t] = gb * delta_u[:, t] + skip * g[:, t]
            if z is not None:
                y = (hs[t + 1] * Cm[:, t, None]).sum(-1) + skip * x[:, t]
                o["dz"][:, t] = dy[:, t] * y * y_slope[:, t]
        o.update(dskip=(g * x).sum((0, 1)), ddt_bias=o["ddt"].sum((0, 1)), dh0=c)
        return o
    z = None if s["z"] is None else d(s["z"])
    if z is not None:
        sg = torch.sigmoid(z)
        gate, ys = z * sg, sg * (1 + z * (1 - sg))
    else:
        gate, ys = torch.ones_like(x), None
    ref = run(x, delta, Bm, Cm, g * gate, skip, h0, dhT, A, z, g, ys)
    mag = run(x.abs(), delta.abs(), Bm.abs(), Cm.abs(), (g * gate).abs(), skip.abs(), h0.abs(), dhT.abs(), A.abs(), z,
              g.abs(), None if z is None else torch.full_like(x, 1.1))
    mag["ddt_bias"] = mag["ddt"].sum((0, 1))
    return ref, mag


def check(got, ref, mag, tokens):
    for k, v in got.items():
        if v is None:
            continue
        tol = half_step(v.dtype) * ref[k].abs() + STEP * (tokens + 32) * mag[k] + 1e-30
        assert d(v).shape == ref[k].shape, k
        over = (d(v) - ref[k]).abs() / tol
        assert (over <= 1).all(), (k, float(over.max()))


def autograd(s, dy, h0, dhT):
    """The gradients by autograd through the definition, all in float64."""
    leaf = {k: (None if v is None else d(v).requires_grad_()) for k, v in s.items()}
    h = d(h0).requires_grad_()
    total = 0
    for b in range(s["x"].shape[0]):
        delta = plain.softplus(leaf["dt"][b] + leaf["dt_bias"])
        hb = h[b]
        for t in range(s["x"].shape[1]):
            u = leaf["x"][b, t]
            hb = torch.exp(delta[t][:, None] * leaf["A"]) * hb + (delta[t] * u)[:, None] * leaf["Bm"][b, t]
            y = ((hb * leaf["Cm"][b, t]).sum(-1) + leaf["skip"] * u) * plain.silu(leaf["z"][b, t])
            total = total + (y * d(dy)[b, t]).sum()
        total = total + (hb * d(dhT)[b]).sum()
    total.backward()
    return dict(dx=leaf["x"].grad, ddt=leaf["dt"].grad, dA=leaf["A"].grad, dB=leaf["Bm"].grad, dC=leaf["Cm"].grad,
                dskip=leaf["skip"].grad, dz=leaf["z"].grad, ddt_bias=leaf["dt_bias"].grad, dh0=h.grad)


def test_the_written_gradients_are_autograd_s():
    """On the CPU values of a small case: the formulas the kernels are held to."""
    s = inputs((2, 9), 8, 8, FP, 3)
    dy, h0, dhT = extras(s, True, 4)
    ref, _ = reference(s, dy, h0, dhT)
    for k, v in autograd(s, dy, h0, dhT).items():
        assert torch.allclose(ref[k], v, rtol=1e-10, atol=1e-12), k


@pytest.mark.parametrize("dtype,B,T,D,N,gate,bias,skip,state", [
    (BF, 1, 1, 8, 16, True, True, True, True), (FP, 2, 17, 72, 16, True, True, True, True),
    (FP, 1, 16, 4, 8, False, False, False, False), (BF, 2, 70, 136, 16, True, True, True, False),
    (FP, 3, 33, 260, 8, True, True, False, True), (FP, 1, 40, 68, 32, True, True, True, True),
    (BF, 1, 130, 64, 32, False, True, True, True), (FP, 1, 1000, 16, 16, True, True, True, True),
    (FP, 2, 203, 132, 16, True, True, True, False), (BF, 1, 5, 1032, 16, True, True, True, True),
    (FP, 1, 64, 128, 16, True, False, True, True), (BF, 3, 257, 40, 8, True, True, True, True)])
def test_gradients_match_the_formulas(gla, dtype, B, T, D, N, gate, bias, skip, state):
    s = inputs((B, T), D, N, dtype, 300 + T, gate, bias, skip)
    dy, h0, dhT = extras(s, state, T)
    got = call(gla, s, dy, h0, dhT)
    gla.gla_check()
    for k, v in (("dz", gate), ("ddt_bias", bias), ("dskip", skip)):
        assert (got[k] is not None) == v
    check(got, *reference(s, dy, h0, dhT), T)
    again = call(gla, s, dy, h0, dhT)
    assert all(v is None or torch.equal(v, again[k]) for k, v in got.items())


def test_raw_steps_strided_rows_and_unwanted_outputs(gla):
    B, T, D, N = 2, 50, 72, 16
    s = inputs((B, T), D, N, FP, 21)
    s["dt"] = torch.rand(B, T, D, device="cuda") * 0.1
    s["dt_bias"] = None
    dy, h0, dhT = extras(s, True, 5)
    got = call(gla, s, dy, h0, dhT, softplus=False)
    gla.gla_check()
    check(got, *reference(s, dy, h0, dhT, soft=False), T)
    xz, dbc = torch.zeros(B, T, 3 * D, device="cuda"), torch.zeros(B, T, 3 + 2 * N, device="cuda")
    xz[..., :D], xz[..., D:2 * D], xz[..., 2 * D:] = s["x"], s["z"], dy
    dbc[..., 3:3 + N], dbc[..., 3 + N:] = s["Bm"], s["Cm"]
    t = dict(s, x=xz[..., :D], z=xz[..., D:2 * D], Bm=dbc[..., 3:3 + N], Cm=dbc[..., 3 + N:])
    other = call(gla, t, xz[..., 2 * D:], h0, dhT, softplus=False, want_dh0=False)
    gla.gla_check()
    assert other["dh0"] is None
    assert all(v is None or torch.equal(v, got[k]) for k, v in other.items())


def test_against_differences_of_the_forward(gla):
    """fp32, (L(p + e v) - L(p - e v)) / 2e per input: off by the forward's
    rounding (STEP * T of the sum of |y dy|) / e and the third derivative's e^2."""
    B, T, D, N = 1, 24, 16, 16
    s = inputs((B, T), D, N, FP, 31)
    dy, h0, dhT = extras(s, True, 6)
    got = call(gla, s, dy, h0, dhT)

    def loss(s, h0):
        y, hT = call_fwd(gla, s, h0)
        return (y.double() * dy.double()).sum().item() + (hT.double() * dhT.double()).sum().item()
    y, hT = call_fwd(gla, s, h0)
    size = (y * dy).abs().sum().item() + (hT * dhT).abs().sum().item()
    e = 3e-3
    for name, out in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("skip", "dskip"),
                      ("z", "dz"), ("dt_bias", "ddt_bias"), ("h0", "dh0")):
        base = h0 if name == "h0" else s[name]
        v = torch.randn(base.shape, generator=torch.Generator().manual_seed(8)).cuda()
        if name in ("dt_bias", "A"):
            v = v * 0.3
        vals = [loss(s, (h0 + k * v).contiguous()) if name == "h0" else loss(dict(s, **{name: (base + k * v).contiguous()}), h0)
                for k in (e, -e)]
        want = (vals[0] - vals[1]) / (2 * e)
        have = (got[out].double() * v.double()).sum().item()
        assert abs(want - have) <= STEP * T * size / e + 10 * e * e * (size + abs(have)), name


def test_steps_that_clear_or_keep_the_state(gla):
    s = inputs((1, 60), 16, 16, FP, 41)
    s["dt"][0, 20:24] = 60.0
    s["dt"][0, 30:40] = -200.0
    dy, h0, dhT = extras(s, True, 7)
    got = call(gla, s, dy, h0, dhT)
    gla.gla_check()
    assert all(torch.isfinite(v).all() for v in got.values())
    check(got, *reference(s, dy, h0, dhT), 60)


def test_no_tokens(gla):
    s = inputs((2, 4), 16, 16, BF, 2)
    e = {k: (v[:, :0].contiguous() if k in ("x", "dt", "z", "Bm", "Cm") else v) for k, v in s.items()}
    dhT = torch.randn(2, 16, 16, device="cuda")
    got = call(gla, e, e["x"], None, dhT)
    gla.gla_check()
    assert torch.equal(got["dh0"], dhT) and not got["dA"].any() and not got["dskip"].any() and got["dB"].shape == (2, 0, 16)


def test_nan_in_one_sequence_stays_there(gla):
    s = inputs((3, 40), 24, 16, FP, 51)
    dy, h0, dhT = extras(s, True, 9)
    clean = call(gla, s, dy, h0, dhT)
    s["x"][1, 7, 3] = float("nan")
    got = call(gla, s, dy, h0, dhT)
    gla.gla_check()
    for k in ("dx", "ddt", "dB", "dC", "dz", "dh0"):
        assert torch.equal(got[k][[0, 2]], clean[k][[0, 2]]), k
    assert torch.isnan(got["dA"][3]).all() and not torch.isnan(got["dA"][4]).any()


@pytest.mark.parametrize("T", [16, 21])
def test_an_infinite_last_input_leaves_finite_what_does_not_depend_on_it(gla, T):
    s = inputs((1, T), 16, 16, FP, 52)
    dy, h0, dhT = extras(s, True, 9)
    s["x"][0, T - 1, 3] = float("inf")
    got = call(gla, s, dy, h0, dhT)
    ref, _ = reference(s, dy, h0, dhT)
    gla.gla_check()
    for k in ("dA", "dx", "dh0"):                             # none reads the last state
        assert torch.isfinite(ref[k]).all() and torch.isfinite(got[k]).all(), k
    assert torch.isinf(got["dskip"][3]) and torch.isfinite(got["dskip"][:3]).all()


def test_capture_beside_an_eager_call_and_another_stream(gla):
    s = inputs((1, 300), 64, 16, BF, 61)
    dy, h0, dhT = extras(s, True, 10)
    want = call(gla, s, dy, h0, dhT)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(gla, s, dy, h0, dhT, stream=side)
    g = torch.cuda.CUDAGraph()
    side.synchronize()
    with torch.cuda.graph(g):
        rep = call(gla, s, dy, h0, dhT)
    g.replay()
    torch.cuda.synchronize()
    for k in NAMES:
        assert torch.equal(got[k], want[k]) and torch.equal(rep[k], want[k]), k


def test_a_training_pass_of_the_block(gla):
    """norm -> convolution -> scan, forward and back, as a layer trains: every
    gradient against autograd through the same graph in float64. Between the
    operators the activations stay fp32, so the tolerance is the
    operators' own: rounding of sums of O(100) terms, 1e-4 of each gradient's largest value."""
    B, T, D, N = 2, 37, 64, 16
    s = inputs((B, T), D, N, FP, 71)
    g = torch.Generator().manual_seed(3)
    rn = lambda *sh, std=1.0: (torch.randn(*sh, generator=g) * std).cuda()  # noqa: E731
    x, res, w, cw, cb, dy = rn(B, T, D), rn(B, T, D), 1 + rn(D, std=0.1), rn(D, 4, std=0.5), rn(D, std=0.1), rn(B, T, D)
    n, st = gla.gla_rmsnorm(x, w, res, 1e-6)
    u, _ = gla.gla_conv1d_fwd(n, cw, cb, want_window=False)
    t = dict(s, x=u)
    y, _ = call_fwd(gla, t)
    got = call(gla, t, dy, None, None)
    dn, dcw, dcb = gla.gla_conv1d_bwd(n, cw, cb, got["dx"])
    dx, dw = gla.gla_rmsnorm_bwd(st, w, dn, dy)             # dy also reaches the residual stream
    gla.gla_check()
    leaves = {k: d(v).requires_grad_() for k, v in (("x", x), ("w", w), ("cw", cw), ("cb", cb), ("A", s["A"]))}
    r = leaves["x"] + d(res)
    nn = r / (r.square().mean(-1, keepdim=True) + 1e-6).sqrt() * leaves["w"]
    rows = torch.cat([torch.zeros(B, 3, D, dtype=F64), nn], 1)
    uu = plain.silu(leaves["cb"] + sum(rows[:, j:j + T] * leaves["cw"][:, j] for j in range(4)))
    delta = plain.softplus(d(s["dt"]) + d(s["dt_bias"]))
    h, ys = torch.zeros(B, D, N, dtype=F64), []
    for k in range(T):
        h = torch.exp(delta[:, k, :, None] * leaves["A"]) * h + (delta[:, k] * uu[:, k])[..., None] * d(s["Bm"])[:, k, None]
        ys.append((h * d(s["Cm"])[:, k, None]).sum(-1) + d(s["skip"]) * uu[:, k])
    yy = torch.stack(ys, 1) * plain.silu(d(s["z"]))
    assert ((d(y) - yy).abs().max() / yy.abs().max()) <= 1e-4
    ((yy * d(dy)).sum() + (r * d(dy)).sum()).backward()
    for name, have in (("x", dx), ("w", dw), ("cw", dcw), ("cb", dcb), ("A", got["dA"])):
        want = leaves[name].grad
        assert (d(have) - want).abs().max() <= 1e-4 * want.abs().max(), name


@pytest.mark.parametrize("dtype,B,T,D,N,gate,state", [
    (BF, 620, 37, 8, 16, True, True), (FP, 620, 17, 12, 8, True, False), (FP, 613, 32, 4, 32, False, True),
    (BF, 86, 33, 968, 16, True, True), (FP, 620, 48, 4, 16, True, True)])
def test_more_chains_than_the_gpu_holds_are_not_cut(gla, dtype, B, T, D, N, gate, state):
    test_gradients_match_the_formulas(gla, dtype, B, T, D, N, gate, True, True, state)
    assert gla.gla_last_launch_count() == 3                 # states entering the tiles, gradients, sums


def test_many_short_segments(gla):
    test_gradients_match_the_formulas(gla, FP, 1, 2100, 12, 16, True, True, True, True)
    assert gla.gla_last_launch_count() == 4                 # and the states carried between segments
