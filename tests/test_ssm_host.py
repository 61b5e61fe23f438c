"""Refusals of the selective state-space, Conv1d-gradient and norm entry points, all on the host: bad
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
        for kw in (dict(x=None), dict(x=ODD), dict(ldx=56), dict(ldx=68), dict(ldx=1 << 31), dict(dt=None), dict(A=ODD), dict(Bm=None),
                   dict(Bm=FAKE + 1), dict(ldb=15), dict(Cm=None), dict(z=ODD, ldz=64), dict(z=FAKE, ldz=60),
                   dict(y=None), dict(y=FAKE), dict(y=ODD), dict(dtype=2), dict(skip=ODD), dict(bias=ODD)):
            assert f(**kw) == binding.GLA_ERR_INVALID_ARG, (f.__name__, kw)
            assert L.gla_last_launch_count() == 0
        for kw in (dict(D=60), dict(D=62, dtype=1), dict(D=0), dict(N=12), dict(N=64),
                   dict(D=1 << 26, ldx=1 << 26, ldt=1 << 26)):
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


def test_conv_backward_rejects_bad_arguments(L):
    def bwd(**kw):
        a = dict(x=FAKE, w=FAKE, b=None, dy=FAKE + 0x100, win=None, B=2, T=50, D=64, dt=0, dx=FAKE + 0x200, dw=FAKE,
                 db=None, ws=FAKE, n=1 << 30)
        a.update(kw)
        return L.gla_conv1d_bwd(a["x"], a["w"], a["b"], a["dy"], a["win"], a["B"], a["T"], a["D"], a["dt"], a["dx"],
                                a["dw"], a["db"], a["ws"], a["n"], None)
    for kw in (dict(x=None), dict(x=ODD), dict(w=None), dict(b=ODD), dict(dy=None), dict(win=ODD), dict(dx=None),
               dict(dx=FAKE), dict(dx=FAKE + 0x100), dict(dw=None), dict(dw=ODD), dict(db=ODD), dict(dt=4), dict(B=-1),
               dict(T=-1), dict(ws=None), dict(ws=ODD)):
        assert bwd(**kw) == binding.GLA_ERR_INVALID_ARG, kw
    assert bwd(D=12) == bwd(D=0) == binding.GLA_ERR_UNSUPPORTED
    assert bwd(B=1, T=(1 << 31) - 256, D=8) == binding.GLA_ERR_INVALID_ARG          # token numbers past an int
    assert binding.gla_conv1d_bwd_workspace_size(1, (1 << 31) - 256, 8) == 0
    assert binding.gla_conv1d_bwd_workspace_size(1, (1 << 31) - 257, 8) > 0
    need = binding.gla_conv1d_bwd_workspace_size(2, 50, 64)
    assert need >= 2 * 5 * 64 * 4 and bwd(n=need - 1) == binding.GLA_ERR_WORKSPACE
    assert binding.gla_conv1d_bwd_workspace_size(0, 50, 64) == 0


def test_norm_rejects_bad_arguments(L):
    def fwd(**kw):
        a = dict(x=FAKE, res=None, w=None, eps=1e-6, rows=4, D=256, group=0, dt=0, s=None, y=FAKE + 0x100, y8=None,
                 scale=None)
        a.update(kw)
        return L.gla_rmsnorm_fwd(a["x"], a["res"], a["w"], a["eps"], a["rows"], a["D"], a["group"], a["dt"], a["s"],
                                 a["y"], a["y8"], a["scale"], None)
    for kw in (dict(x=None), dict(x=ODD), dict(res=ODD), dict(w=ODD), dict(eps=-1.0), dict(eps=float("nan")),
               dict(rows=-1), dict(rows=1 << 31), dict(dt=3), dict(s=ODD), dict(y=ODD), dict(y=FAKE),
               dict(y8=FAKE + 0x200), dict(scale=FAKE), dict(y8=FAKE + 0x100, scale=FAKE),
               dict(y8=FAKE, scale=FAKE), dict(s=FAKE + 0x100)):
        assert fwd(**kw) == binding.GLA_ERR_INVALID_ARG, kw
    for kw in (dict(D=12), dict(D=0), dict(D=8200), dict(D=6, dt=1), dict(group=16), dict(group=-1), dict(group=256)):
        assert fwd(**kw) == binding.GLA_ERR_UNSUPPORTED, kw
    assert fwd(rows=0) == fwd(y=None) == binding.GLA_OK

    def bwd(**kw):
        a = dict(s=FAKE, w=None, dy=FAKE + 0x100, ds=None, eps=1e-6, rows=4, D=256, dt=0, dx=FAKE + 0x200, dw=FAKE,
                 ws=FAKE, n=1 << 30)
        a.update(kw)
        return L.gla_rmsnorm_bwd(a["s"], a["w"], a["dy"], a["ds"], a["eps"], a["rows"], a["D"], a["dt"], a["dx"],
                                 a["dw"], a["ws"], a["n"], None)
    for kw in (dict(s=None), dict(dy=None), dict(dy=ODD), dict(ds=ODD), dict(dx=None), dict(dx=FAKE), dict(dw=ODD),
               dict(w=ODD), dict(eps=-1.0), dict(rows=-2), dict(ws=None)):
        assert bwd(**kw) == binding.GLA_ERR_INVALID_ARG, kw
    assert bwd(D=8200) == bwd(D=4) == binding.GLA_ERR_UNSUPPORTED
    need = binding.gla_rmsnorm_bwd_workspace_size(4, 256)
    assert need == 4 * 256 * 4 and bwd(n=need - 1) == binding.GLA_ERR_WORKSPACE
    assert bwd(rows=0, dw=None) == binding.GLA_OK


def test_selective_scan_backward_rejects_bad_arguments(L):
    def bwd(**kw):
        a = dict(x=FAKE, ldx=64, dt=FAKE, ldt=64, A=FAKE, Bm=FAKE, ldb=16, Cm=FAKE, ldc=16, skip=None, z=None, ldz=0,
                 bias=None, h0=None, dy=FAKE, ldg=64, dhT=None, B=2, T=50, D=64, N=16, dtype=0, dx=FAKE + 0x100,
                 ddt=FAKE + 0x200, dA=FAKE, dB=FAKE + 0x300, dC=FAKE + 0x400, dskip=None, dz=None, db=None, dh0=None,
                 ws=FAKE, n=1 << 40)
        a.update(kw)
        return L.gla_ssm_bwd(a["x"], a["ldx"], a["dt"], a["ldt"], a["A"], a["Bm"], a["ldb"], a["Cm"], a["ldc"],
                             a["skip"], a["z"], a["ldz"], a["bias"], 1, a["h0"], a["dy"], a["ldg"], a["dhT"], a["B"],
                             a["T"], a["D"], a["N"], a["dtype"], a["dx"], a["ddt"], a["dA"], a["dB"], a["dC"],
                             a["dskip"], a["dz"], a["db"], a["dh0"], a["ws"], a["n"], None)
    for kw in (dict(x=None), dict(ldx=60), dict(dt=ODD), dict(A=None), dict(Bm=None), dict(Cm=FAKE + 1), dict(dy=None),
               dict(dy=ODD), dict(ldg=63), dict(dx=None), dict(ddt=None), dict(dA=None), dict(dB=None), dict(dC=ODD),
               dict(dskip=ODD), dict(db=ODD), dict(dh0=ODD), dict(dhT=ODD), dict(h0=ODD), dict(dx=FAKE),
               dict(z=FAKE, ldz=64), dict(dz=FAKE + 0x500), dict(ws=None), dict(dtype=9), dict(B=-1), dict(T=-1),
               dict(dh0=FAKE, h0=FAKE), dict(dh0=FAKE, dhT=FAKE)):
        assert bwd(**kw) == binding.GLA_ERR_INVALID_ARG, kw
    assert bwd(D=4) == bwd(N=24) == binding.GLA_ERR_UNSUPPORTED
    need = binding.gla_ssm_bwd_workspace_size(2, 50, 64, 16)
    assert need > 0 and bwd(n=need - 1) == binding.GLA_ERR_WORKSPACE
    assert binding.gla_ssm_bwd_workspace_size(2, 0, 64, 16) == 0
