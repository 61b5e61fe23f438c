"""Trees of drafted tokens over the state pool on the GPU (gla_tree_fwd,
gla_tree_commit, gla_conv1d_tree) against the definition in float64
(tree_plain.py, which derives the tolerances)."""
import pytest
import torch

import tree_plain as plain
from tree_plain import forest, half_step

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def gla():
    import linear_attention_chunk_gb300 as m
    from linear_attention_chunk_gb300.build import build
    build()
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Case:
    """Inputs of the calls on the GPU, and on the host in float64."""

    def __init__(self, dtype, sizes, H, dk, dv, shape="mixed", gated=False, seed=0, spare=2, behind=3, gates=0.2, D=0):
        g = torch.Generator().manual_seed(seed)

        def rn(*s, std=1.0):
            return torch.randn(*s, generator=g) * std

        self.cu, self.parents = forest(sizes, shape, seed)
        T, N = self.cu[-1], len(sizes)
        self.N, self.T, self.H, self.dk, self.dv, self.dtype, self.scale = N, T, H, dk, dv, dtype, dk ** -0.5
        self.slots = torch.randperm(N + spare, generator=g)[:N].tolist()
        rows = T + behind                    # rows of no tree: left as they were
        self.parents += [-1] * behind
        self.q, self.v = rn(rows, H, dk).to(dtype).cuda(), rn(rows, H, dv).to(dtype).cuda()
        self.k = torch.nn.functional.normalize(rn(rows, H, dk), dim=-1).to(dtype).cuda()
        self.pool = rn(N + spare, H, dk, dv, std=0.3).cuda()
        self.gated = gated
        if gated:
            self.log = (-torch.rand(rows, H, generator=g) * gates).cuda()
        else:
            self.log = torch.log1p(-torch.exp2(-5 - 7 * torch.arange(H) / max(1, H - 1))).cuda()
        self.last = [int(torch.randint(-1, n, (1,), generator=g)) if n else -1 for n in sizes]
        self.D = D
        if D:
            self.x, self.win = rn(rows, D).to(dtype).cuda(), rn(N + spare, 4, D).cuda()
            self.w, self.b = rn(D, 4, std=0.5).cuda(), rn(D, std=0.2).cuda()

    def tree_args(self):
        return ints(self.cu), ints(self.parents)

    def logs(self):
        log = self.log.double().cpu()
        return log if self.gated else log.expand(self.q.shape[0], -1)

    def host(self):
        return [t.double().cpu() for t in (self.q, self.k, self.v)]

    def fwd(self, gla, **kw):
        f = gla.gla_tree_fwd_gated if self.gated else gla.gla_tree_fwd
        return f(self.q, self.k, self.v, self.log, *self.tree_args(), self.pool, ints(self.slots), self.scale, **kw)

    def fwd_ref(self):
        q, k, v = self.host()
        return plain.tree_fwd(q, k, v, self.logs(), self.scale, self.cu, self.parents, self.slots, self.pool.double().cpu())

    def commit(self, gla, windows=True, **kw):
        f = gla.gla_tree_commit_gated if self.gated else gla.gla_tree_commit
        if self.D and windows:
            kw.update(x=self.x, win_pool=self.win)
        return f(self.k, self.v, self.log, *self.tree_args(), ints(self.last), self.pool, ints(self.slots), **kw)

    def commit_ref(self):
        _, k, v = self.host()
        return plain.commit(k, v, self.logs(), self.cu, self.parents, self.last, self.slots, self.pool.double().cpu())


def near(got, ref, tol, name="o"):
    g = got.double().cpu()
    assert g.shape == ref.shape
    tol = half_step(got.dtype) * ref.abs() + tol + 1e-30
    off = (g - ref).abs()
    assert (off <= tol).all(), (name, float((off / tol).max()), off.argmax())


SIZES = [[1], [2], [7, 12], [64], [0, 5, 0, 17, 64, 1], [31, 32, 33, 15, 16, 17], [0, 0], [9, 63, 48, 8]]
HEADS = [(BF, 2, 96, 192), (BF, 5, 96, 192), (FP, 1, 96, 192), (FP, 3, 5, 7), (FP, 2, 128, 256), (FP, 1, 1, 1),
         (FP, 2, 33, 130), (FP, 4, 64, 64)]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("dtype,H,dk,dv", HEADS, ids=str)
@pytest.mark.parametrize("gated", [False, True])
def test_forward(gla, sizes, dtype, H, dk, dv, gated):
    c = Case(dtype, sizes, H, dk, dv, gated=gated, seed=len(sizes))
    before = c.pool.clone()
    o = torch.full((c.q.shape[0], H, dv), 7.0, dtype=dtype, device="cuda")
    assert c.fwd(gla, o=o) is o
    gla.gla_check()
    ref, tol = c.fwd_ref()
    near(o[: c.T], ref[: c.T], tol[: c.T])
    assert (o[c.T:] == 7).all() and torch.equal(c.pool, before)


@pytest.mark.parametrize("shape", ["chain", "star", "binary", "mixed"])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("gated", [False, True])
def test_shapes_of_trees(gla, shape, dtype, gated):
    c = Case(dtype, [64, 40, 3], 3, 96, 192, shape=shape, gated=gated, seed=5, gates=1.0)
    o = c.fwd(gla)
    gla.gla_check()
    ref, tol = c.fwd_ref()
    near(o[: c.T], ref[: c.T], tol[: c.T])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_decays_of_zero_and_strong_ones(gla, dtype):
    """log decays of -inf, -80, -200 and -3 a node; a page that holds NaN and inf is cleared with the rest."""
    c = Case(dtype, [64, 33], 2, 96, 192, gated=True, seed=6, gates=3.0)
    pick = torch.rand(c.log.shape, generator=torch.Generator().manual_seed(1))
    c.log[pick.cuda() < 0.1] = -INF
    c.log[(pick.cuda() > 0.95)] = -80.0
    c.log[(pick.cuda() > 0.98)] = -200.0
    ref, tol = c.fwd_ref()
    near(c.fwd(gla)[: c.T], ref[: c.T], tol[: c.T])
    c.log[c.cu[0]:c.cu[1]][[i for i in range(64) if c.parents[i] < 0]] = -INF      # every path of tree 0 clears its page
    ref, tol = c.fwd_ref()
    c.pool[c.slots[0]] = NAN
    c.pool[c.slots[0], :, ::3] = INF
    near(c.fwd(gla)[: c.T], ref[: c.T], tol[: c.T])
    c.last = [63, 32]
    ref, tol = plain.commit(*c.host()[1:], c.logs(), c.cu, c.parents, c.last, c.slots, torch.nan_to_num(c.pool.double().cpu()))
    c.commit(gla)
    used = [c.slots[0], c.slots[1]]
    near(c.pool[used], ref[used], tol[used], "pool")
    gla.gla_check()


def test_lambda_zero_and_one(gla):
    c = Case(BF, [20, 64], 2, 96, 192, shape="chain", seed=7)
    c.log = torch.tensor([-INF, 0.0]).cuda()
    near(c.fwd(gla)[: c.T], *[t[: c.T] for t in c.fwd_ref()])
    gla.gla_check()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("where", ["k", "v", "q"])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_a_node_that_is_not_finite_stays_on_its_paths(gla, dtype, where, value):
    c = Case(dtype, [40, 16], 2, 96, 192, shape="binary", seed=8)
    clean = c.fwd(gla).clone()
    getattr(c, where)[5, 1, ::7] = value
    o = c.fwd(gla)
    gla.gla_check()
    below = [i for i in range(40) if 5 in plain.way(c.parents[:40], i)]
    hit = below if where != "q" else [5]
    other = [i for i in range(c.T) if i not in hit]
    assert torch.equal(o[other], clean[other]) and torch.equal(o[hit, 0], clean[hit, 0])
    bad = ~torch.isfinite(o[hit, 1].float())
    # of v, its channels; of k and q, all of them (node 5 alone may have an exact 0 x inf either way: never finite)
    assert bad[:, ::7].all() and (where != "v" or not bad[:, 1].any())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_a_page_that_is_not_finite_stays_in_its_channel(gla, dtype):
    c = Case(dtype, [40, 16], 2, 96, 192, seed=9)
    clean = c.fwd(gla)[: c.T].clone()       # (rows behind the last tree are not written)
    c.pool[c.slots[0], 1, 3, 50] = NAN
    c.pool[c.slots[0], 1, 9, 70] = INF
    o = c.fwd(gla)[: c.T]
    gla.gla_check()
    same = torch.ones(192, dtype=torch.bool)
    same[[50, 70]] = False
    assert torch.equal(o[:, 0], clean[:, 0]) and torch.equal(o[40:], clean[40:])
    assert torch.equal(o[:40, 1][:, same], clean[:40, 1][:, same])
    assert not torch.isfinite(o[:40, 1][:, [50, 70]].float()).any()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_infinities_of_a_page_keep_their_sign(gla, dtype):
    """One infinity a channel: it reaches every node with the sign that q gives it. Numbers next to fp32's largest stay numbers."""
    c = Case(dtype, [40, 16], 2, 96, 192, seed=9)
    c.q = torch.where(c.q == 0, torch.ones_like(c.q), c.q)
    c.pool[c.slots[0], 1, 3, 50] = INF
    c.pool[c.slots[0], 1, 9, 70] = -INF
    o = c.fwd(gla)
    gla.gla_check()
    up = c.q[:40, 1] > 0
    assert torch.equal(o[:40, 1, 50] == INF, up[:, 3]) and torch.equal(o[:40, 1, 50] == -INF, ~up[:, 3])
    assert torch.equal(o[:40, 1, 70] == -INF, up[:, 9]) and torch.equal(o[:40, 1, 70] == INF, ~up[:, 9])
    c.q *= 2.0 ** -20
    c.pool[c.slots[0], :, 5, ::3] = 3.4e38      # (bf16's largest is 3.3895e38)
    c.pool[c.slots[0], 1, 3, 50] = c.pool[c.slots[0], 1, 9, 70] = 3.402823e38
    ref, tol = c.fwd_ref()
    near(c.fwd(gla)[: c.T], ref[: c.T], tol[: c.T])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_zero_times_infinity_is_not_hidden(gla, dtype):
    """A node's score of 0 with an infinite v on its path gives NaN; cut off by a decay of 0, nothing."""
    c = Case(dtype, [40, 16], 2, 96, 192, shape="chain", gated=True, seed=10)
    c.v[5, 1, 20] = INF
    c.q[8, 1] = 0
    c.log[20, 1] = -INF
    o = c.fwd(gla)[: c.T].float()
    gla.gla_check()
    assert o[8, 1, 20].isnan() and not o[8, 1, :20].any() and not o[8, 1, 21:].any()
    assert not o[5:20, 1, 20].isfinite().any()
    o[5:20, 1, 20] = 0
    assert o.isfinite().all()


def test_column_ranges_of_a_projection(gla):
    c = Case(BF, [17, 64, 3], 3, 96, 192, seed=10)
    want = c.fwd(gla)
    wide = torch.full((c.q.shape[0] + 2, 3 * (96 * 2 + 192) + 40), NAN, dtype=BF, device="cuda")
    parts = [wide[1:-1, a:b].unflatten(1, (3, -1)) for a, b in ((8, 296), (296, 584), (592, 1168))]
    for part, t in zip(parts, (c.q, c.k, c.v)):
        part.copy_(t)
    c.q, c.k, c.v = parts
    assert torch.equal(c.fwd(gla)[: c.T], want[: c.T])
    pool = c.pool.clone()
    c.commit(gla)
    got, c.pool = c.pool, pool
    c.k, c.v = (t.contiguous() for t in (c.k, c.v))
    c.commit(gla)
    assert torch.equal(got, c.pool)
    gla.gla_check()


def test_sequences_may_read_one_slot(gla):
    """A prompt continued by several sequences before its page is forked."""
    c = Case(BF, [9, 30, 64], 2, 96, 192, seed=11)
    c.slots = [1, 1, 1]
    near(c.fwd(gla)[: c.T], *[t[: c.T] for t in c.fwd_ref()])
    gla.gla_check()


def test_without_slots(gla):
    c = Case(BF, [9, 30], 2, 96, 192, seed=12)
    c.slots = [0, 1]
    o = gla.gla_tree_fwd(c.q, c.k, c.v, c.log, *c.tree_args(), c.pool)
    near(o[: c.T], *[t[: c.T] for t in c.fwd_ref()])
    gla.gla_check()


BAD = dict(slot=lambda c: c.slots.__setitem__(1, 99), low_slot=lambda c: c.slots.__setitem__(1, -1),
           parent=lambda c: c.parents.__setitem__(c.cu[1] + 3, 3), low_parent=lambda c: c.parents.__setitem__(c.cu[1], -2),
           offset=lambda c: c.cu.__setitem__(2, 10 ** 6), many=lambda c: None)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("what", list(BAD) + ["last", "low_last"])
def test_a_bad_entry_skips_its_sequence(gla, dtype, what):
    sizes = [12, 65 if what == "many" else 20, 7]
    c = Case(dtype, sizes, 2, 96, 192, seed=13, D=16)
    good, win = c.pool.clone(), c.win.clone()
    c.last = [11, 4, 6]
    if what in BAD:
        ref, tol = c.fwd_ref()
        BAD[what](c)
        o = torch.full((c.q.shape[0], 2, 192), 7.0, dtype=dtype, device="cuda")
        y = torch.full((c.q.shape[0], 16), 7.0, dtype=dtype, device="cuda")
        c.fwd(gla, o=o)
        with pytest.raises(gla.GlaError) as e:
            gla.gla_check()
        assert e.value.status == gla.GLA_ERR_INVALID_ARG
        a, b = 12, 12 + sizes[1]
        near(o[:a], ref[:a], tol[:a])
        assert (o[a:b] == 7).all()
        if what != "offset":                  # (that moves the next tree's start as well)
            near(o[b:c.T], ref[b:c.T], tol[b:c.T])
        gla.gla_conv1d_tree(c.x, c.w, c.b, *c.tree_args(), c.win, ints(c.slots), y=y)
        with pytest.raises(gla.GlaError):
            gla.gla_check()
        assert (y[a:b] == 7).all() and not (y[:a] == 7).all()
    else:
        c.last[1] = 20 if what == "last" else -2
    c.commit(gla)
    with pytest.raises(gla.GlaError) as e:
        gla.gla_check()
    assert e.value.status == gla.GLA_ERR_INVALID_ARG
    same = [s for s in range(5) if s not in (c.slots[0], c.slots[2])]
    assert torch.equal(c.pool[same], good[same]) and torch.equal(c.win[same], win[same])
    assert not torch.equal(c.pool[c.slots[0]], good[c.slots[0]])
    gla.gla_check()


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("dtype,H,dk,dv", HEADS, ids=str)
@pytest.mark.parametrize("gated", [False, True])
def test_commit(gla, sizes, dtype, H, dk, dv, gated):
    c = Case(dtype, sizes, H, dk, dv, gated=gated, seed=20 + len(sizes), D=24 if dtype == BF else 12)
    ref, tol = c.commit_ref()
    before, win = c.pool.clone(), plain.windows(c.x.double().cpu(), c.cu, c.parents, c.last, c.slots, c.win.double().cpu())
    assert c.commit(gla) is c.pool
    gla.gla_check()
    near(c.pool, ref, tol, "pool")
    assert torch.equal(c.win.double().cpu(), win)
    still = [s for s in range(len(sizes) + 2) if s not in [c.slots[n] for n in range(c.N) if c.last[n] >= 0]]
    assert torch.equal(c.pool[still], before[still])


@pytest.mark.parametrize("shape", ["chain", "star"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_commit_of_long_and_short_paths(gla, shape, dtype):
    c = Case(dtype, [64, 64, 3, 1, 2], 2, 96, 192, shape=shape, gated=True, seed=31, D=1032)
    c.last = [63, 30, 2, 0, -1]
    ref, tol = c.commit_ref()
    win = plain.windows(c.x.double().cpu(), c.cu, c.parents, c.last, c.slots, c.win.double().cpu())
    c.commit(gla)
    gla.gla_check()
    near(c.pool, ref, tol, "pool")
    assert torch.equal(c.win.double().cpu(), win)


@pytest.mark.parametrize("dtype,D", [(BF, 8), (BF, 24), (BF, 1032), (BF, 4096), (FP, 4), (FP, 516), (FP, 2052), (BF, 2048)])
@pytest.mark.parametrize("shape", ["chain", "star", "mixed"])
def test_convolution(gla, dtype, D, shape):
    c = Case(dtype, [5, 0, 64, 1, 33], 1, 96 if dtype == BF else 4, 192 if dtype == BF else 4, shape=shape, seed=40, D=D)
    y = torch.full((c.x.shape[0], D), 7.0, dtype=dtype, device="cuda")
    win = c.win.clone()
    wide = torch.full((c.x.shape[0], D + 16), NAN, dtype=dtype, device="cuda")
    wide[:, 8: 8 + D] = c.x
    for x, b in ((c.x, c.b), (wide[:, 8: 8 + D], c.b), (c.x, None)):
        y.fill_(7.0)
        assert gla.gla_conv1d_tree(x, c.w, b, *c.tree_args(), c.win, ints(c.slots), y=y) is y
        gla.gla_check()
        ref, tol = plain.conv_tree(c.x.double().cpu(), c.w.double().cpu(), torch.zeros(D).double() if b is None else b.double().cpu(),
                                   c.cu, c.parents, c.slots, c.win.double().cpu())
        near(y[: c.T], ref[: c.T], tol[: c.T], "y")
        assert (y[c.T:] == 7).all() and torch.equal(c.win, win)


@pytest.mark.parametrize("dtype,D,N", [(BF, 2056, 300), (FP, 1028, 700), (BF, 20008, 90), (FP, 20004, 50)])
def test_convolution_of_many(gla, dtype, D, N):
    """More trees than CTAs a block of channels, and more blocks than SMs; a bad tree among them is skipped alone."""
    c = Case(dtype, [(11 * n) % 23 for n in range(N)], 1, 96 if dtype == BF else 4, 192 if dtype == BF else 4, seed=41, D=D)
    ref, tol = plain.conv_tree(c.x.double().cpu(), c.w.double().cpu(), c.b.double().cpu(), c.cu, c.parents, c.slots, c.win.double().cpu())
    near(gla.gla_conv1d_tree(c.x, c.w, c.b, *c.tree_args(), c.win, ints(c.slots))[: c.T], ref[: c.T], tol[: c.T], "y")
    gla.gla_check()
    a, b = c.cu[7], c.cu[8]                  # 8 nodes
    c.parents[a + 3] = 3
    y = torch.full((c.x.shape[0], D), 7.0, dtype=dtype, device="cuda")
    gla.gla_conv1d_tree(c.x, c.w, c.b, *c.tree_args(), c.win, ints(c.slots), y=y)
    with pytest.raises(gla.GlaError):
        gla.gla_check()
    assert (y[a:b] == 7).all() and b - a == 8
    near(y[:a], ref[:a], tol[:a], "y")
    near(y[b: c.T], ref[b: c.T], tol[b: c.T], "y")


@pytest.mark.parametrize("sizes", [[12, 5], [64, 64]], ids=str)
def test_same_as_steps_along_every_path(gla, sizes):
    """A tree's outputs are those of the serving step run along each path from a copy of the page, up to both kernels' errors."""
    c = Case(BF, sizes, 2, 96, 192, seed=50, D=32)
    o = c.fwd(gla)
    y = gla.gla_conv1d_tree(c.x, c.w, c.b, *c.tree_args(), c.win, ints(c.slots))
    for n, first, par in plain.each(c.cu, c.parents):
        for i in (0, len(par) // 2, len(par) - 1):
            S, win = c.pool[c.slots[n]][None].clone(), c.win[c.slots[n]][None].clone()
            for j in plain.way(par, i):
                t = first + j
                step = gla.gla_decode_step(c.q[t][None], c.k[t][None], c.v[t][None], c.log, S, c.scale)
                conv = gla.gla_conv1d_step(c.x[t][None], c.w, c.b, win)
            ref, tol = c.fwd_ref()
            near(o[t], step[0].double().cpu(), 2 * tol[t] + half_step(BF) * ref[t].abs())
            # the step's SiLU is a (1 + tanh(a/2)) / 2 with the approximate tanh, 2^-11 relative: |a| 2^-12, |a| < 8
            both = 2 * half_step(BF) * conv[0].double().cpu().abs() + 2e-3
            assert ((y[t].double().cpu() - conv[0].double().cpu()).abs() <= both).all()
    gla.gla_check()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_slots_past_32_bits(gla, dtype):
    """A pool of more than 2^31 floats and packed rows past 2^31 elements: the last slot, the last rows."""
    H, dk, dv = 16, 96, 192
    c = Case(dtype, [33], H, dk, dv, seed=60, behind=0)
    n_slots = (1 << 31) // (H * dk * dv) + 2
    pool = torch.empty(n_slots, H, dk, dv, device="cuda")
    pool[-1] = c.pool[c.slots[0]]
    rows = (1 << 31) // (H * dv) + 40
    v = torch.empty(rows, H, dv, dtype=dtype, device="cuda")
    q, k = (torch.empty(rows, H, dk, dtype=dtype, device="cuda") for _ in range(2))
    for t, s in ((q, c.q), (k, c.k), (v, c.v)):
        t[-33:] = s
    parents = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    parents[-33:] = ints(c.parents)
    o = gla.gla_tree_fwd(q, k, v, c.log, ints([rows - 33, rows]), parents, pool, ints([n_slots - 1]), c.scale)
    gla.gla_check()
    ref, tol = c.fwd_ref()
    near(o[-33:], ref, tol)
    c.last = [32]
    ref, tol = c.commit_ref()
    gla.gla_tree_commit(k, v, c.log, ints([rows - 33, rows]), parents, ints(c.last), pool, ints([n_slots - 1]))
    gla.gla_check()
    near(pool[-1], ref[c.slots[0]], tol[c.slots[0]], "pool")


def test_captured_and_replayed_with_other_trees(gla):
    """The trees are device data: a captured step follows what is written into them before each replay."""
    a, b = (Case(BF, [24, 40], 2, 96, 192, shape=s, seed=70 + i, D=64) for i, s in enumerate(("mixed", "chain")))
    cu, par = a.tree_args()
    slots, last = ints(a.slots), ints(a.last)
    o, y = torch.empty_like(a.v), torch.empty_like(a.x)
    q, k, v, x, pool, win = (t.clone() for t in (a.q, a.k, a.v, a.x, a.pool, a.win))

    def step():
        gla.gla_conv1d_tree(x, a.w, a.b, cu, par, win, slots, y=y)
        gla.gla_tree_fwd(q, k, v, a.log, cu, par, pool, slots, a.scale, o=o)
        gla.gla_tree_commit(k, v, a.log, cu, par, last, pool, slots, x=x, win_pool=win)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for c in (a, b):
        c.w, c.b, c.log = a.w, a.b, a.log
        for t, s in ((q, c.q), (k, c.k), (v, c.v), (x, c.x), (pool, c.pool), (win, c.win), (par, ints(c.parents)),
                     (cu, ints(c.cu)), (slots, ints(c.slots)), (last, ints(c.last))):
            t.copy_(s)
        g.replay()
        torch.cuda.synchronize()
        near(o[: c.T], *[t[: c.T] for t in c.fwd_ref()])
        ref, tol = c.commit_ref()
        near(pool, ref, tol, "pool")
        assert torch.equal(win.double().cpu(), plain.windows(c.x.double().cpu(), c.cu, c.parents, c.last, c.slots, c.win.double().cpu()))
    gla.gla_check()


def test_two_calls_at_once_and_on_a_stream(gla):
    cases = [Case(BF, [64] * 40, 16, 96, 192, seed=80 + i, gated=bool(i)) for i in range(2)]
    alone = [c.fwd(gla) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [c.fwd(gla, stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a[: c.T], b[: c.T]) for a, b, c in zip(alone, got, cases))
    gla.gla_check()


@pytest.mark.parametrize("N", [1, 3, 11, 60])
def test_every_unit_of_many(gla, N):
    """More (sequence, head) pairs than CTAs run at a time, of uneven trees: each is its own result."""
    H = 16
    c = Case(BF, [(7 * n) % 65 for n in range(N)], H, 96, 192, seed=90 + N, gated=True)
    whole = c.fwd(gla)
    for n in range(0, N, max(1, N // 6)):
        a, b = c.cu[n], c.cu[n + 1]
        if a == b:
            continue
        one = gla.gla_tree_fwd_gated(c.q[a:b], c.k[a:b], c.v[a:b], c.log[a:b].contiguous(), ints([0, b - a]),
                                     ints(c.parents[a:b]), c.pool, ints([c.slots[n]]), c.scale)
        assert torch.equal(one, whole[a:b])
    ref, tol = c.fwd_ref()
    near(whole[: c.T], ref[: c.T], tol[: c.T])
    gla.gla_check()


def test_refusals(gla):
    c = Case(BF, [9, 3], 2, 96, 192, seed=99, D=16)
    cu, par = c.tree_args()
    sl, last = ints(c.slots), ints(c.last)

    def refused(f, *a, **kw):
        with pytest.raises(gla.GlaError):
            f(*a, **kw)

    f = gla.gla_tree_fwd
    refused(f, c.q, c.k, c.v, c.log.double(), cu, par, c.pool, sl)
    refused(f, c.q, c.k, c.v.float(), c.log, cu, par, c.pool, sl)
    refused(f, c.q[:-1], c.k, c.v, c.log, cu, par, c.pool, sl)
    refused(f, c.q, c.k, c.v, c.log, cu.long(), par, c.pool, sl)
    refused(f, c.q, c.k, c.v, c.log, cu, par[:-1], c.pool, sl)
    refused(f, c.q, c.k, c.v, c.log, cu, par, c.pool[:1], None)
    refused(f, c.q, c.k, c.v, c.log, cu, par, c.pool.bfloat16(), sl)
    refused(f, c.q, c.k, c.v, c.log, cu, par, c.pool, sl[:1])
    refused(f, c.q.cpu(), c.k, c.v, c.log, cu, par, c.pool, sl)
    refused(f, c.q, c.k.cpu(), c.v, c.log, cu, par, c.pool, sl)
    refused(f, c.q, c.k, c.v, c.log, cu[:0], par, c.pool, sl)
    refused(f, c.q, c.k, c.v, c.log, cu, par, c.pool, sl, o=c.v)
    refused(f, c.q.transpose(1, 2).contiguous().transpose(1, 2), c.k, c.v, c.log, cu, par, c.pool, sl)
    refused(f, *(torch.zeros(12, 2, d, dtype=BF, device="cuda") for d in (64, 64, 64)), c.log, cu, par[:12],
            torch.zeros(4, 2, 64, 64, device="cuda"), sl)
    refused(gla.gla_tree_fwd_gated, c.q, c.k, c.v, c.log, cu, par, c.pool, sl)
    g = gla.gla_tree_commit
    refused(g, c.k, c.v, c.log, cu, par, last[:1], c.pool, sl)
    refused(g, c.k, c.v, c.log, cu, par, last, c.pool, sl, x=c.x)
    refused(g, c.k, c.v, c.log, cu, par, last, c.pool, sl, win_pool=c.win)
    refused(g, c.k, c.v, c.log, cu, par, last, c.pool, sl, x=c.x[:, :12], win_pool=c.win[:, :, :12].contiguous())
    refused(gla.gla_conv1d_tree, c.x, c.w, c.b, cu, par, c.win[:, :3], sl)
    refused(gla.gla_conv1d_tree, c.x, c.w[:, :3], c.b, cu, par, c.win, sl)
    refused(gla.gla_conv1d_tree, c.x, c.w, c.b, cu, par, c.win, sl, y=c.x)
    gla.gla_check()
    empty = torch.zeros(0, 2, 96, dtype=BF, device="cuda")
    assert f(empty, empty, torch.zeros(0, 2, 192, dtype=BF, device="cuda"), c.log, ints([0, 0, 0]), ints([]), c.pool, sl).shape == (0, 2, 192)
    assert f(empty, empty, torch.zeros(0, 2, 192, dtype=BF, device="cuda"), c.log, ints([0]), ints([]), c.pool).shape == (0, 2, 192)
    gla.gla_check()
