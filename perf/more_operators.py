"""Drafted tokens over the state pool, the pool's pages and the layer norm, as
measurable cases: inputs, one pass of each operator (the library's entry points
where `own` is set, elementary torch operations otherwise), its definition in
64 bits, and the bytes and operations it cannot do without.

Kinds of case:
  tree      outputs of every drafted token of a tree, from the sequence's state
            page, which stays as it is
  commit    the accepted path of each tree taken into the state and window pages
  conv      the causal convolution with SiLU along each path of the trees
  fork      pages copied (one prompt continued several times) and pages cleared,
            in the pools of several layers
  compact   pages in use moved to the front of the pools
  norm      residual addition and layer norm
  norm_bwd  the gradients of residual addition and layer norm
"""
import functools
import math
import random

import torch

own = False

EPS = 1e-6
MOST_NODES = 64


# ------------------------------------------------------------------- cases
def listed():
    return [
        # an interactive session: two sequences with a small tree each, where latency counts
        dict(name="tree_few", kind="tree", N=2, lo=7, hi=12, depth=4, H=16, dk=96, dv=192, gated=False, fused=False,
             dtype="bf16"),
        # a serving batch whose draft model proposes up to 32 tokens a sequence, ragged
        dict(name="tree_serve", kind="tree", N=256, lo=1, hi=32, depth=8, H=16, dk=96, dv=192, gated=False, fused=True,
             dtype="bf16"),
        # wide trees with the per-token decay
        dict(name="tree_wide_gated", kind="tree", N=128, lo=48, hi=64, depth=16, H=16, dk=96, dv=192, gated=True,
             fused=False, dtype="bf16"),
        # the serving loop's full batch (1,280 sequences) keeps what was accepted, windows included
        dict(name="commit_full", kind="commit", N=1280, lo=4, hi=24, depth=6, H=16, dk=96, dv=192, gated=False, D=2048,
             dtype="bf16"),
        # a few sequences in the validation type, odd head sizes
        dict(name="commit_small_fp32", kind="commit", N=3, lo=1, hi=17, depth=9, H=5, dk=40, dv=76, gated=True, D=516,
             dtype="fp32"),
        # the convolution in front of the mixer for the serving batch's trees
        dict(name="conv_serve", kind="conv", N=256, lo=16, hi=64, depth=8, D=4096, dtype="bf16"),
        dict(name="conv_small_fp32", kind="conv", N=3, lo=1, hi=9, depth=5, D=516, dtype="fp32"),
        # four prompts, each continued eight times, and the pages of ended sequences cleared, in eight layers
        dict(name="fork_layers", kind="fork", slots=64, sources=4, copies=8, clears=12, layers=8, H=16, D=2048),
        # a pool with holes closed up, in six layers
        dict(name="compact_layers", kind="compact", slots=256, live=160, moves=60, layers=6, H=16, D=2048),
        # the layer norm in front of a layer at the training shape
        dict(name="norm_train", kind="norm", rows=16384, D=2048, res=True, dtype="bf16"),
        dict(name="norm_bwd_train", kind="norm_bwd", rows=16384, D=2048, dtype="bf16"),
        # a short odd call in the validation type
        dict(name="norm_bwd_small_fp32", kind="norm_bwd", rows=333, D=516, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges: any kind, sizes over their logarithm,
    their products capped at those of the largest listed cases."""
    kind = rng.choice(["tree", "tree", "commit", "commit", "conv", "fork", "compact", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind in ("tree", "commit", "conv"):
        hi = _log_int(rng, 1, MOST_NODES)
        lo, depth = rng.randint(1, hi), _log_int(rng, 1, max(2, hi))
    if kind in ("tree", "commit"):
        H = rng.choice([1, 3, 8, 16, 16])
        dk, dv = (96, 192) if dtype == "bf16" else (_log_int(rng, 8, 128), _log_int(rng, 8, 256))
    if kind == "tree":
        N = _log_int(rng, 1, min(256, (1 << 17) // (H * hi)))
        return dict(kind=kind, N=N, lo=lo, hi=hi, depth=depth, H=H, dk=dk, dv=dv, gated=rng.random() < 0.5,
                    fused=dtype == "bf16" and rng.random() < 0.5, dtype=dtype)
    if kind == "commit":
        return dict(kind=kind, N=_log_int(rng, 1, min(1280, 1280 * 24 // hi)), lo=lo, hi=hi, depth=min(depth, 16), H=H,
                    dk=dk, dv=dv, gated=rng.random() < 0.5,
                    D=_log_int(rng, 64, 2048) // 8 * 8 if rng.random() < 0.7 else 0, dtype=dtype)
    if kind == "conv":
        D = _log_int(rng, 64, 4096) // 8 * 8
        return dict(kind=kind, N=_log_int(rng, 1, min(1280, (1 << 26) // (D * hi))), lo=lo, hi=hi, depth=depth, D=D,
                    dtype=dtype)
    if kind == "fork":
        copies, sources = rng.randint(1, 8), rng.randint(1, 6)
        return dict(kind=kind, slots=sources * (copies + 1) + rng.randint(0, 8), sources=sources, copies=copies, clears=0,
                    layers=rng.randint(1, 8), H=rng.choice([1, 4, 16]), D=_log_int(rng, 64, 2048) // 8 * 8)
    if kind == "compact":
        slots = _log_int(rng, 2, 256)
        live = rng.randint(1, slots - 1)
        return dict(kind=kind, slots=slots, live=live, moves=rng.randint(1, min(live, slots - live, 60)),
                    layers=rng.randint(1, 6), H=rng.choice([1, 4, 16]), D=_log_int(rng, 64, 2048) // 8 * 8)
    rows, D = _log_int(rng, 1, 16384), _log_int(rng, 64, 8192) // 8 * 8
    rows = max(1, min(rows, (1 << 25) // D // (1 if dtype == "bf16" else 2)))
    if kind == "norm":
        return dict(kind=kind, rows=rows, D=D, res=rng.random() < 0.7, dtype=dtype)
    return dict(kind=kind, rows=rows, D=D, dtype=dtype)


# ------------------------------------------------------------------ inputs
class _Gen:
    """Seeded normal and uniform tensors on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device="cuda") * std).to(dtype)

    def perm(self, n):
        return torch.randperm(n, generator=self.g, device="cuda")


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case):
    """Nodes of each tree, by the case alone."""
    rng = random.Random(case["N"] * 4096 + case["lo"] * 64 + case["hi"])
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["N"])]


def _accepts(case):
    """Whether each sequence keeps some of its tree: of a serving batch, most do."""
    return [n % 16 != 15 for n in range(case["N"])]


def _trees(case, seed):
    """Offsets of the packed trees, each node's parent (-1: the sequence's
    state itself) and the last accepted node of each tree, on the GPU."""
    rng = random.Random(seed)
    cu, parents, last = [0], [], []
    for n, keep in zip(_lens(case), _accepts(case)):
        par, depth = [], []
        for i in range(n):
            p = i - 1 if rng.random() < 0.4 else rng.randint(-1, i - 1)
            while p >= 0 and depth[p] >= case["depth"]:
                p = par[p]
            par.append(p)
            depth.append(1 if p < 0 else depth[p] + 1)
        parents += par
        cu.append(cu[-1] + n)
        last.append(rng.randint(0, n - 1) if keep else -1)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    return ints(cu), ints(parents), ints(last)


def _pages(g, case):
    """The pools of several layers, states and windows."""
    H, D, n = case["H"], case["D"], case["slots"]
    return [g.normal(n, *shape, std=0.1) for _ in range(case["layers"]) for shape in ((H, 96, 192), (4, D))]


def prepare(case, seed):
    g, kind = _Gen(seed), case["kind"]
    if kind in ("tree", "commit", "conv"):
        cu, parents, last = _trees(case, seed)
        N, T, dt = case["N"], sum(_lens(case)), _dtype(case)
        spare = N + 3
        s = dict(cu=cu, parents=parents, most=case["hi"], slots=g.perm(spare)[:N].to(torch.int32))
    if kind in ("tree", "commit"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        if kind == "tree" and case["fused"]:    # column ranges of the layer's projection
            wide = g.normal(T, H * (2 * dk + dv), dtype=dt)
            q, k, v = (t.unflatten(1, (H, -1)) for t in wide.split([H * dk, H * dk, H * dv], 1))
        else:
            q, k, v = (g.normal(T, H, d, dtype=dt) for d in (dk, dk, dv))
        k.copy_(torch.nn.functional.normalize(k.float(), dim=-1))
        s.update(q=q, k=k, v=v, pool=g.normal(spare, H, dk, dv, std=0.1), g=None, lam=None, scale=dk ** -0.5)
        if case["gated"]:
            s["g"] = torch.nn.functional.logsigmoid(g.normal(T, H)) / 16
        else:
            s["lam"] = torch.log1p(-torch.exp2(-5 - 7 * torch.arange(H, device="cuda") / max(1, H - 1)))
        if kind == "commit":
            s.update(last=last, x=None, win=None)
            if case["D"]:
                s.update(x=g.normal(T, case["D"], dtype=dt), win=g.normal(spare, 4, case["D"]))
    elif kind == "conv":
        D = case["D"]
        s.update(x=g.normal(T, D, dtype=dt), w=g.normal(D, 4, std=0.5), b=g.normal(D, std=0.1), win=g.normal(spare, 4, D))
    elif kind == "fork":
        order = g.perm(case["slots"]).to(torch.int32)
        n = case["sources"] * case["copies"]
        src = order[: case["sources"]].repeat_interleave(case["copies"])
        dst = order[case["sources"]: case["sources"] + n]
        free = order[case["sources"] + n:][: case["clears"]]
        s = dict(pools=_pages(g, case), src=src.contiguous(), dst=dst.contiguous(), free=free.contiguous())
    elif kind == "compact":
        live = torch.zeros(case["slots"], dtype=torch.bool, device="cuda")
        front, back = g.perm(case["live"]), g.perm(case["slots"] - case["live"])
        live[front[case["moves"]:]] = True
        live[case["live"] + back[: case["moves"]]] = True
        s = dict(pools=_pages(g, case), live=live)
    else:
        rows, D, dt = case["rows"], case["D"], _dtype(case)
        s = dict(x=g.normal(rows, D, dtype=dt) + 0.5, w=1.0 + g.normal(D, std=0.1), b=g.normal(D, std=0.1))
        s["x"] = s["x"].to(dt)
        if kind == "norm":
            s["res"] = g.normal(rows, D, std=3.0, dtype=dt) if case["res"] else None
        else:
            s["dy"] = g.normal(rows, D, dtype=dt)
            s["ds"] = g.normal(rows, D, dtype=dt)
    s["kind"] = kind
    return s


# ------------------------------------------------------------- plain forms
def _padded(s):
    """Packed trees as rows of a batch: the packed index of node i of tree n
    [N, M], which of them there are, and whether node j lies on the path from
    the state to node i, itself included, [N, M, M]."""
    cu = s["cu"].long()
    i = torch.arange(s["most"], device=cu.device)
    at = cu[:-1, None] + i
    there = at < cu[1:, None]
    at = at.clamp(max=int(s["parents"].numel()) - 1)
    par = torch.where(there, s["parents"].long()[at], -1)
    up = torch.eye(len(i), device=cu.device) + (par[:, :, None] == i).float()
    path = functools.reduce(lambda r, _: (r @ r > 0).float(), range(6), up)   # up to 2^6 steps
    return at, there, path > 0.5


def _decays(s, at, path):
    """The decay of the state at node i [N, H, M], and that from node j to node
    i where j is on i's path, else 0, [N, H, M, M]."""
    if s["g"] is not None:
        step = s["g"][at].double().transpose(1, 2)
    else:
        step = s["lam"].double()[None, :, None].expand(at.shape[0], -1, at.shape[1])
    total = (path.double()[:, None] @ step[..., None])[..., 0]
    gap = torch.where(path[:, None], total[..., :, None] - total[..., None, :], -math.inf)
    return torch.exp(total).float(), torch.exp(gap).float()


def _plain_tree(s):
    at, there, path = _padded(s)
    far, w = _decays(s, at, path)
    q, k, v = (s[c][at].float().transpose(1, 2) for c in "qkv")
    pool = s["pool"][s["slots"].long()]
    o = far[..., None] * (q @ pool) + (q @ k.transpose(2, 3) * w) @ v
    out = torch.empty(s["v"].shape, dtype=s["v"].dtype, device=q.device)
    out[at[there]] = (s["scale"] * o).transpose(1, 2)[there].to(out.dtype)
    return {"o": out}


def _plain_commit(s):
    at, there, path = _padded(s)
    far, w = _decays(s, at, path)
    n = torch.arange(at.shape[0], device=at.device)
    last, slots = s["last"].long(), s["slots"].long()
    keep = last >= 0
    row = last.clamp(min=0)
    k, v = (s[c][at].float().transpose(1, 2) for c in "kv")
    new = far[n, :, row, None, None] * s["pool"][slots] + (k * w[n, :, row, :, None]).transpose(2, 3) @ v
    s["pool"][slots[keep]] = new[keep]
    out = {"pool": s["pool"]}
    if s["x"] is not None:
        old = s["win"][slots]
        on = path[n, row]                                  # the accepted path, oldest first: its last four inputs
        count = on.sum(1)
        place = on.long().cumsum(1) - count[:, None]       # 0: the last one, -1: the one before it
        from_end = torch.arange(-3, 1, device=at.device)
        pick = (on[:, None] & (place[:, None] == from_end[:, None])).float()        # [N, 4, M]
        taken = pick @ s["x"][at].float()
        have = pick.sum(2) > 0
        shift = (torch.arange(4, device=at.device) + count[:, None]).clamp(max=3)
        moved = torch.gather(old, 1, shift[..., None].expand(-1, -1, old.shape[2]))
        s["win"][slots[keep]] = torch.where(have[..., None], taken, moved)[keep]
        out["win"] = s["win"]
    return out


def _plain_conv(s):
    x, cu, par = s["x"].float(), s["cu"].long(), s["parents"].long()
    seq = torch.repeat_interleave(torch.arange(cu.numel() - 1, device=x.device), cu[1:] - cu[:-1])
    slot, first = s["slots"].long()[seq], cu[:-1][seq]

    def up(a):      # one step towards the root: nodes as packed indices, -1 - r r steps behind the root
        return torch.where(a >= 0, torch.where(par[a.clamp(min=0)] >= 0, first + par[a.clamp(min=0)], -1), a - 1)

    def value(a):
        return torch.where((a >= 0)[:, None], x[a.clamp(min=0)], s["win"][slot, (4 + a).clamp(0, 3)])

    a0 = torch.arange(x.shape[0], device=x.device)
    a1 = up(a0)
    a2 = up(a1)
    a3 = up(a2)
    acc = s["b"] + sum(s["w"][:, j] * value(a) for j, a in enumerate((a3, a2, a1, a0)))
    return {"y": (acc / (1 + torch.exp(-acc))).to(s["x"].dtype)}


def _moved(pool, dst, src):
    pool[dst] = pool[src]
    return pool


def _cleared(pool, at):
    pool[at] = 0
    return pool


def _plain_fork(s):
    src, dst, free = s["src"].long(), s["dst"].long(), s["free"].long()
    return {"pools": [_cleared(_moved(p, dst, src), free) for p in s["pools"]]}


def _plain_compact(s):
    live = s["live"]
    i = torch.arange(live.numel(), device=live.device)
    count = live.sum()
    dst, src = i[~live & (i < count)], i[live & (i >= count)]     # both in ascending order
    moved = torch.where(live, i, -1)
    moved[src] = dst
    return {"map": moved.to(torch.int32), "count": count.to(torch.int32).view(1),
            "pools": [_moved(p, dst, src) for p in s["pools"]]}


def _plain_norm(s):
    r = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
    c = r - r.mean(1, keepdim=True)
    y = c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS) * s["w"] + s["b"]
    out = {"y": y.to(s["x"].dtype)}
    if s["res"] is not None:
        out["s"] = r.to(s["x"].dtype)
    return out


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    c = x - x.mean(1, keepdim=True)
    r = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    xn, g = c * r, dy * s["w"]
    dx = r * (g - g.mean(1, keepdim=True) - xn * (g * xn).mean(1, keepdim=True)) + s["ds"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xn).sum(0), "db": dy.sum(0)}


_PLAIN = dict(tree=_plain_tree, commit=_plain_commit, conv=_plain_conv, fork=_plain_fork, compact=_plain_compact,
              norm=_plain_norm, norm_bwd=_plain_norm_bwd)


# ------------------------------------------------- the library's operators
def _own(s):
    import linear_attention_chunk_gb300 as gla
    kind = s["kind"]
    if kind == "tree":
        if s["g"] is not None:
            o = gla.gla_tree_fwd_gated(s["q"], s["k"], s["v"], s["g"], s["cu"], s["parents"], s["pool"], s["slots"],
                                       s["scale"])
        else:
            o = gla.gla_tree_fwd(s["q"], s["k"], s["v"], s["lam"], s["cu"], s["parents"], s["pool"], s["slots"], s["scale"])
        return {"o": o}
    if kind == "commit":
        if s["g"] is not None:
            gla.gla_tree_commit_gated(s["k"], s["v"], s["g"], s["cu"], s["parents"], s["last"], s["pool"], s["slots"],
                                      x=s["x"], win_pool=s["win"])
        else:
            gla.gla_tree_commit(s["k"], s["v"], s["lam"], s["cu"], s["parents"], s["last"], s["pool"], s["slots"],
                                x=s["x"], win_pool=s["win"])
        return {"pool": s["pool"]} if s["x"] is None else {"pool": s["pool"], "win": s["win"]}
    if kind == "conv":
        return {"y": gla.gla_conv1d_tree(s["x"], s["w"], s["b"], s["cu"], s["parents"], s["win"], s["slots"])}
    if kind == "fork":
        gla.gla_pages_copy(s["pools"], s["src"], s["dst"])
        gla.gla_pages_clear(s["pools"], s["free"])
        return {"pools": s["pools"]}
    if kind == "compact":
        moved, count = gla.gla_pages_compact(s["pools"], s["live"])
        return {"map": moved, "count": count, "pools": s["pools"]}
    if kind == "norm":
        y, r = gla.gla_layernorm(s["x"], s["w"], s["b"], s["res"], EPS)
        return {"y": y} if s["res"] is None else {"y": y, "s": r}
    dx, dw, db = gla.gla_layernorm_bwd(s["x"], s["w"], s["dy"], s["ds"], EPS)
    return {"dx": dx, "dw": dw, "db": db}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["kind"]](state)


# ------------------------------------------------------ floors of the work
def work(case):
    """Every input read once and every output written once. Operations: for a
    drafted token and head the state's readout and the token's own product with
    its key and value (its path's tokens come on top); for an accepted path one
    step of the state; four taps, SiLU; the norm's sums and its line."""
    kind = case["kind"]
    if kind in ("fork", "compact"):
        page = (case["H"] * 96 * 192 + 4 * case["D"]) * 4 * case["layers"]
        if kind == "fork":
            n = case["sources"] + case["sources"] * case["copies"] + case["clears"]
        else:
            n = 2 * case["moves"]
        return {"bytes": n * page + case["slots"] * 4, "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    if kind in ("norm", "norm_bwd"):
        rows, D = case["rows"], case["D"]
        if kind == "norm":
            return {"bytes": rows * D * e * (4 if case["res"] else 2) + 2 * D * 4, "flops": rows * D * 9}
        return {"bytes": rows * D * e * 4 + 3 * D * 4, "flops": rows * D * 15}
    N, T = case["N"], sum(_lens(case))
    if kind == "conv":
        D = case["D"]
        return {"bytes": T * D * e * 2 + N * D * 3 * 4 + D * 5 * 4, "flops": T * D * 12}
    H, dk, dv = case["H"], case["dk"], case["dv"]
    gates = T * H * 4 if case["gated"] else H * 4
    if kind == "tree":
        return {"bytes": N * H * dk * dv * 4 + T * H * 2 * (dk + dv) * e + gates,
                "flops": T * H * 2 * (dk * dv + dk + dv)}
    live = sum(_accepts(case))
    return {"bytes": live * (H * (2 * dk * dv * 4 + (dk + dv) * e) + case["D"] * (4 * 4 + 4 * e)),
            "flops": live * H * 3 * dk * dv}


# ------------------------------------------------- the definition, 64 bits
def _d(t):
    return None if t is None else t.double()


def _each_tree(s):
    """Slot, first packed token and parents of every sequence."""
    cu, par = s["cu"].tolist(), s["parents"].tolist()
    for n, slot in enumerate(s["slots"].tolist()):
        yield n, slot, cu[n], par[cu[n]:cu[n + 1]]


def _way(par, i):
    """The nodes from the root's child down to node i."""
    way = []
    while i >= 0:
        way.append(i)
        i = par[i]
    return way[::-1]


def _step(s, S, t):
    """The state after packed token t."""
    log = s["g"][t] if s["g"] is not None else s["lam"]
    return torch.exp(_d(log))[:, None, None] * S + _d(s["k"][t])[:, :, None] * _d(s["v"][t])[:, None, :]


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    if kind == "tree":
        o = torch.empty(s["v"].shape, dtype=torch.float64, device="cuda")
        for _, slot, first, par in _each_tree(s):
            root, states = _d(s["pool"][slot]), []
            for i, p in enumerate(par):
                states.append(_step(s, root if p < 0 else states[p], first + i))
                o[first + i] = s["scale"] * (_d(s["q"][first + i])[:, :, None] * states[i]).sum(1)
        return {"o": o}
    if kind == "commit":
        out = {"pool": _d(s["pool"])}
        if s["x"] is not None:
            out["win"] = _d(s["win"])
        last = s["last"].tolist()
        for n, slot, first, par in _each_tree(s):
            way = _way(par, last[n])
            for i in way:
                out["pool"][slot] = _step(s, out["pool"][slot], first + i)
            if way and s["x"] is not None:
                rows = [out["win"][slot]] + [_d(s["x"][first + i])[None] for i in way]
                out["win"][slot] = torch.cat(rows)[-4:]
        return out
    if kind == "conv":
        y, w, x = torch.empty_like(s["x"], dtype=torch.float64), _d(s["w"]), _d(s["x"])
        for _, slot, first, par in _each_tree(s):
            behind = _d(s["win"][slot, 1:])
            for i in range(len(par)):
                way = [first + j for j in _way(par, i)[-4:]]
                rows = torch.cat([behind, x[way]])[-4:]
                acc = _d(s["b"]) + (rows * w.t()).sum(0)
                y[first + i] = acc * torch.sigmoid(acc)
        return {"y": y}
    if kind == "fork":
        pools = [p.double() for p in s["pools"]]
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            for p in pools:
                p[b] = p[a]
        for a in s["free"].tolist():
            for p in pools:
                p[a] = 0
        return {"pools": pools}
    if kind == "compact":
        pools, live = [p.double() for p in s["pools"]], s["live"].tolist()
        count = sum(live)
        holes = [i for i in range(count) if not live[i]]
        for i in range(count, len(live)):
            if live[i]:
                to = holes.pop(0)
                for p in pools:
                    p[to] = p[i]
        return {"map": None, "count": None, "pools": pools}
    x = _d(s["x"])
    if kind == "norm" and s["res"] is not None:
        x = x + _d(s["res"])
    D = x.shape[1]
    mu = x.mean(1, keepdim=True)
    sd = ((x * x).mean(1, keepdim=True) - mu * mu + EPS).sqrt()
    n = (x - mu) / sd
    if kind == "norm":
        out = {"y": n * _d(s["w"]) + _d(s["b"])}
        if s["res"] is not None:
            out["s"] = x
        return out
    g = _d(s["dy"]) * _d(s["w"])
    dx = (D * g - g.sum(1, keepdim=True) - n * (g * n).sum(1, keepdim=True)) / (D * sd)
    return {"dx": dx + _d(s["ds"]), "dw": (_d(s["dy"]) * n).sum(0), "db": _d(s["dy"]).sum(0)}
