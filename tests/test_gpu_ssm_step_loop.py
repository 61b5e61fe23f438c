"""The serving step (gla_ssm_step) with several times more groups of sequences
than the GPU holds CTAs: every CTA takes several turns, through all stages of
its ring, and the last group is ragged. Against the definition in float64, and
with bad slots in later turns."""
import pytest
import torch

import test_gpu_ssm as ssm
from ssm_plain import close, d
from test_gpu_ssm import BF, FP, gla  # noqa: F401

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


GROUP = 4          # sequences a warp takes at once


def rows_of(D):
    """Groups that one wave of CTAs takes (32 channels a CTA, at most six an SM)."""
    return max(1, 6 * sms() // -(-D // 32))


def step_case(dtype, n, D, N, filt, seed):
    s = ssm.inputs((n,), D, N, dtype, seed)
    pool, win, w, b = ssm.pools(n + 2, D, N, seed + 1)
    if not filt:
        w = b = win = None
    slots = torch.randperm(n + 2, generator=torch.Generator().manual_seed(seed))[:n].tolist()
    return s, pool, win, w, b, slots


def step_reference(s, slots, pool, win, w, b):
    return ssm.ref_packed(s, list(range(len(slots) + 1)), slots, pool, win, w, b)


@pytest.mark.parametrize("dtype,D,N,filt", [
    (BF, 1032, 16, True), (BF, 1032, 16, False), (FP, 1032, 16, True), (FP, 1036, 16, False), (BF, 1032, 8, True),
    (FP, 1036, 8, False), (BF, 2056, 32, True), (FP, 2052, 32, True), (BF, 2056, 32, False), (FP, 2052, 32, False)])
def test_step_of_many_groups(gla, dtype, D, N, filt):  # noqa: F811
    n = GROUP * (4 * rows_of(D) + 3) + 3                    # five turns of the first CTAs, a last group of three
    s, pool, win, w, b, slots = step_case(dtype, n, D, N, filt, 30 + N)
    p1, w1 = pool.clone(), None if win is None else win.clone()
    y = ssm.call_step(gla, s, p1, ssm.i32(slots), w, b, w1)
    gla.gla_check()
    for i, (ry, my, rh, mh, nw) in enumerate(step_reference(s, slots, pool, win, w, b)):
        close(y[i:i + 1], ry, my, 1, f"y of {i}")
        close(p1[slots[i]], rh, mh, 1, f"state of {i}")
        assert nw is None or torch.equal(d(w1[slots[i]]), nw)
    rest = [k for k in range(n + 2) if k not in set(slots)]
    assert torch.equal(p1[rest], pool[rest]) and (w1 is None or torch.equal(w1[rest], win[rest]))


@pytest.mark.parametrize("dtype,N,filt", [(BF, 16, True), (FP, 8, False), (BF, 32, True)])
def test_step_with_bad_slots_in_later_turns(gla, dtype, N, filt):  # noqa: F811
    D = 1032
    turn = GROUP * rows_of(D)
    n = 3 * turn + 2 * GROUP + 2
    s, pool, win, w, b, slots = step_case(dtype, n, D, N, filt, 50 + N)
    p0, w0 = pool.clone(), None if win is None else win.clone()
    y0 = ssm.call_step(gla, s, p0, ssm.i32(slots), w, b, w0)
    gla.gla_check()
    hurt = {5: n + 2, turn + 2: -1, 2 * turn: 1 << 30, 3 * turn + 7: -(1 << 31), n - 1: n + 9}
    bad = [hurt.get(i, v) for i, v in enumerate(slots)]
    p1, w1 = pool.clone(), None if win is None else win.clone()
    y = torch.full((n, D), 7.0, dtype=dtype, device="cuda")
    ssm.call_step(gla, s, p1, ssm.i32(bad), w, b, w1, y=y)
    with pytest.raises(gla.GlaError) as e:
        gla.gla_check()
    assert e.value.status == gla.GLA_ERR_INVALID_ARG
    gone = sorted(hurt)
    kept = [i for i in range(n) if i not in hurt]
    lost, live = [slots[i] for i in gone], [slots[i] for i in kept]
    assert (y[gone] == 7).all() and torch.equal(y[kept], y0[kept])
    assert torch.equal(p1[lost], pool[lost]) and torch.equal(p1[live], p0[live])
    if filt:
        assert torch.equal(w1[lost], win[lost]) and torch.equal(w1[live], w0[live])
