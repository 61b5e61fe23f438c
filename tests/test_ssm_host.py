"""Refusals of the selective state-space entry points, all on the host: bad
arguments get the documented status before anything is launched. The fake
addresses are never dereferenced."""
import pytest

from linear_attention_chunk_gb300 import binding
from linear_attention_chunk_gb300.build import build

FAKE = 0x10000   # 16-byte aligned
ODD = 0x10008    # 8-byte aligned only


@pytest.fixture(scope="module")
def L():
    build()
    return binding.lib()


def test_selective_scan_rejects_bad_arguments(L):
    base = dict(x=FAKE, ldx=64, dt=FAKE + 0x100, ldt=64, A=FAKE, Bm=FAKE, ldb=16, Cm=FAKE, ldc=16, skip=None, z=None,
                ldz=0, bias=None, sp=1, h0=None, B=2, T=50, D=64, N=16, dtype=0, y=FAKE + 0x200, hT=None, cw=None,
                cb=None, cu=FAKE, slots=None, pool=FAKE, win=None, n_slots=4, nseq=3)

    def head(a):
        return [a["x"], a["ldx"], a["dt"], a["ldt"], a["A"], a["Bm"], a["ldb"], a["Cm"], a["ldc"], a["skip"], a["z"],
                a["ldz"], a["bias"], a["sp"]]

    def fwd(**kw):
        a = dict(base, **kw)
        return L.gla_ssm_fwd(*head(a), a["h0"], a["B"], a["T"], a["D"], a["N"], a["dtype"], a["y"], a["hT"], None, 0,
                             None)

    def var(**kw):
        a = dict(base, **kw)
        return L.gla_ssm_varlen(*head(a), a["cw"], a["cb"], a["cu"], a["slots"], a["pool"], a["win"], a["n_slots"],
                                a["nseq"], a["T"], a["D"], a["N"], a["dtype"], a["y"], None, 0, None)

    def step(**kw):
        a = dict(base, **kw)
        return L.gla_ssm_step(*head(a), a["cw"], a["cb"], a["slots"], a["pool"], a["win"], a["n_slots"], a["nseq"],
                              a["D"], a["N"], a["dtype"], a["y"], None)
    for f in (fwd, var, step):
        for kw in (dict(x=None), dict(x=ODD), dict(ldx=56), dict(ldx=68), dict(dt=None), dict(A=ODD), dict(Bm=None),
                   dict(Bm=FAKE + 1), dict(ldb=15), dict(Cm=None), dict(z=ODD, ldz=64), dict(z=FAKE, ldz=60),
                   dict(y=None), dict(y=FAKE), dict(y=ODD), dict(dtype=2), dict(skip=ODD), dict(bias=ODD)):
            assert f(**kw) == binding.GLA_ERR_INVALID_ARG, (f.__name__, kw)
            assert L.gla_last_launch_count() == 0
        for kw in (dict(D=60), dict(D=0), dict(N=12), dict(N=64)):
            assert f(**kw) == binding.GLA_ERR_UNSUPPORTED, (f.__name__, kw)
    assert fwd(B=-1) == fwd(T=-1) == fwd(h0=ODD) == fwd(hT=ODD) == binding.GLA_ERR_INVALID_ARG
    assert fwd(B=1 << 20, T=1 << 20) == binding.GLA_ERR_INVALID_ARG       # too large
    assert fwd(B=0) == fwd(T=0) == binding.GLA_OK                         # nothing to do
    for f in (var, step):
        assert f(nseq=-1) == f(pool=None) == f(pool=ODD) == f(slots=ODD) == binding.GLA_ERR_INVALID_ARG
        assert f(n_slots=2) == f(n_slots=-1) == binding.GLA_ERR_INVALID_ARG
        assert f(cw=FAKE) == f(win=FAKE) == f(cb=FAKE) == binding.GLA_ERR_INVALID_ARG   # filter and windows together
        assert f(cw=ODD, win=FAKE) == binding.GLA_ERR_INVALID_ARG
        assert f(nseq=0) == binding.GLA_OK
    assert var(cu=None) == var(T=-1) == binding.GLA_ERR_INVALID_ARG
    assert var(T=0) == binding.GLA_OK                                     # every sequence empty
    assert binding.gla_ssm_fwd_workspace_size(1, 4096, 64, 16) > 0
    assert binding.gla_ssm_fwd_workspace_size(1, 16, 64, 16) == 0
    assert binding.gla_ssm_fwd_workspace_size(64, 2048, 4096, 16) == 0    # enough chains
    assert binding.gla_ssm_varlen_workspace_size(2, 5000, 64, 16) > 0
    assert binding.gla_ssm_varlen_workspace_size(2, 5000, 64, 12) == 0    # invalid
