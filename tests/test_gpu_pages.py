"""Copying, clearing and compacting the pages of the pools on the GPU. Pages are
moved as they are, so every comparison is for equality."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gla():
    import linear_attention_chunk_gb300 as m
    from linear_attention_chunk_gb300.build import build
    build()
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def pools(n, seed=0):
    """Pools of several element types and page sizes: a state's, a window's, one
    of a few bytes, one that is no multiple of 16 bytes, one over several chunks."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def bits(*shape):
        return torch.randint(-2 ** 31, 2 ** 31 - 1, shape, generator=g, device="cuda", dtype=torch.int32)

    return [bits(n, 3, 96, 192).view(torch.float32), bits(n, 4, 1032).view(torch.bfloat16), bits(n, 4).view(torch.uint8),
            bits(n, 5, 7), bits(n, 100003), bits(n, 8192)]


def clones(ps):
    return [p.clone() for p in ps]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("n,src,dst", [(4, [0], [3]), (9, [2, 2, 2, 5], [0, 1, 8, 7]), (3, [1, 2], [1, 0]), (2, [], []),
                                       (40, [7] * 30, list(range(8, 38)))], ids=str)
def test_copy(gla, n, src, dst):
    ps = pools(n)
    want = clones(ps)
    for p in want:
        for a, b in zip(src, dst):
            p[b] = p[a]
    gla.gla_pages_copy(ps, ints(src), ints(dst))
    gla.gla_check()
    assert same(ps, want)
    one = pools(n)[1]
    gla.gla_pages_copy(one, ints(src), ints(dst))
    assert same([one], [want[1]])


def test_slices_of_the_lists(gla):
    """The lists need an int's alignment only."""
    order = ints([9, 3, 5, 1, 2])
    ps = pools(6)
    want = clones(ps)
    for p in want:
        p[2] = p[3]
        p[4 - 3] = 0
    gla.gla_pages_copy(ps, order[1:2], order[4:])
    gla.gla_pages_clear(ps, order[3:4])
    gla.gla_check()
    assert same(ps, want)


@pytest.mark.parametrize("at", [[], [0], [3, 1], list(range(9))], ids=str)
def test_clear(gla, at):
    ps = pools(9)
    want = clones(ps)
    for p in want:
        p[at] = 0
    gla.gla_pages_clear(ps, ints(at))
    gla.gla_check()
    assert same(ps, want)


def test_a_page_outside_the_pool_is_skipped(gla):
    ps = pools(6)
    want = clones(ps)
    for p in want:
        p[5] = p[0]
    for src, dst in (([0, 6, 1, -1], [5, 1, 6, 2]), ([0, 2 ** 31 - 1], [5, 1])):
        gla.gla_pages_copy(ps, ints(src), ints(dst))
        with pytest.raises(gla.GlaError) as e:
            gla.gla_check()
        assert e.value.status == gla.GLA_ERR_INVALID_ARG and same(ps, want)
    for p in want:
        p[2] = 0
    gla.gla_pages_clear(ps, ints([2, 6, -5]))
    with pytest.raises(gla.GlaError):
        gla.gla_check()
    assert same(ps, want)


def plan(live):
    count = sum(live)
    holes = [i for i in range(count) if not live[i]]
    to = [i if on else -1 for i, on in enumerate(live)]
    for i in range(count, len(live)):
        if live[i]:
            to[i] = holes.pop(0)
    return to, count


@pytest.mark.parametrize("n", [1, 2, 7, 64, 255, 256, 257, 1024, 1025, 4095, 4096, 4097, 5000])
@pytest.mark.parametrize("share", [0.0, 0.05, 0.5, 0.95, 1.0])
def test_compact(gla, n, share):
    rng = random.Random(n * 10 + int(share * 100))
    live = [rng.random() < share for _ in range(n)]
    wide = pools(n)[:4] if n < 100 else [torch.arange(n * 8, dtype=torch.int32, device="cuda").view(n, 8),
                                          torch.arange(n * 3, dtype=torch.int32, device="cuda").view(n, 3)]
    to, count = plan(live)
    want = clones(wide)
    for p, q in zip(wide, want):
        for i, j in enumerate(to):
            if j >= 0 and j != i:
                q[j] = p[i]
    mask = torch.tensor(live).cuda()
    got, k = gla.gla_pages_compact(wide, mask)
    gla.gla_check()
    assert got.tolist() == to and k.tolist() == [count] and same(wide, want)
    again, k = gla.gla_pages_compact(wide, (torch.arange(n) < count).cuda().to(torch.uint8) * 3)
    gla.gla_check()
    assert again.tolist() == [i if i < count else -1 for i in range(n)] and k.tolist() == [count] and same(wide, want)


@pytest.mark.parametrize("n", [50, 4100])
def test_captured_with_a_mask_that_changes(gla, n):
    ps = pools(n)[:2] if n < 100 else [torch.arange(n * 8, dtype=torch.int32, device="cuda").view(n, 8)]
    live = torch.zeros(n, dtype=torch.bool, device="cuda")
    ws = torch.empty(gla.gla_pages_compact_workspace_size(n), dtype=torch.uint8, device="cuda")
    gla.gla_pages_compact(ps, live, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        to, count = gla.gla_pages_compact(ps, live, workspace=ws)
    for seed in range(4):
        rng = random.Random(seed)
        on = [rng.random() < 0.6 for _ in range(n)]
        live.copy_(torch.tensor(on))
        want = clones(ps)
        ref, k = plan(on)
        for p, q in zip(ps, want):
            for i, j in enumerate(ref):
                if j >= 0:
                    q[j] = p[i]
        graph.replay()
        torch.cuda.synchronize()
        assert to.tolist() == ref and count.tolist() == [k] and same(ps, want)
    gla.gla_check()


def test_pages_past_32_bits(gla):
    """A pool of more than 2^32 bytes, and pages of more than 2^31."""
    p = torch.zeros(9, 1 << 27, dtype=torch.int32, device="cuda")           # 9 pages of 512 MB
    p[8] = torch.arange(1 << 27, dtype=torch.int32, device="cuda")
    gla.gla_pages_copy(p, ints([8]), ints([0]))
    gla.gla_check()
    assert torch.equal(p[0], p[8]) and not p[1:8].any()
    q = torch.zeros(2, (1 << 29) + 5, dtype=torch.int32, device="cuda")     # pages of 2 GB and 20 bytes: not 16-byte aligned
    q[1, -9:] = 3
    gla.gla_pages_copy(q, ints([1]), ints([0]))
    gla.gla_check()
    assert torch.equal(q[0], q[1])


def test_stream_and_many_pools(gla):
    ps = [torch.full((3, 64), float(i), device="cuda") for i in range(128)]
    for p in ps:
        p[1] += 1000
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gla.gla_pages_copy(ps, ints([1]), ints([2]), stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all((p[2] == i + 1000).all() and (p[0] == i).all() for i, p in enumerate(ps))
    with pytest.raises(gla.GlaError):
        gla.gla_pages_copy(ps + [ps[0]], ints([1]), ints([2]))
    gla.gla_check()


def test_refusals(gla):
    p = torch.zeros(4, 8, device="cuda")
    one = ints([1])
    live = torch.ones(4, dtype=torch.bool, device="cuda")
    for f in (lambda: gla.gla_pages_copy([], one, one), lambda: gla.gla_pages_copy([p, p[:3]], one, one),
              lambda: gla.gla_pages_copy(p.t(), one, one), lambda: gla.gla_pages_copy(p.cpu(), one, one),
              lambda: gla.gla_pages_copy(p, one, ints([1, 2])), lambda: gla.gla_pages_copy(p, one.long(), one.long()),
              lambda: gla.gla_pages_copy(p, one.cpu(), one), lambda: gla.gla_pages_clear(p, one.view(1, 1)),
              lambda: gla.gla_pages_copy(torch.zeros(4, 3, dtype=torch.bfloat16, device="cuda"), one, one),
              lambda: gla.gla_pages_compact(p, live[:3]), lambda: gla.gla_pages_compact(p, live.int()),
              lambda: gla.gla_pages_compact(torch.zeros(4097, 4, device="cuda"), torch.ones(4097, dtype=torch.bool, device="cuda"),
                                            workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(gla.GlaError):
            f()
    none = torch.zeros(0, 8, device="cuda")
    to, count = gla.gla_pages_compact(none, live[:0])
    assert to.numel() == 0 and count.tolist() == [0]
    gla.gla_pages_copy(none, ints([]), ints([]))
    gla.gla_check()
