"""Buffers that the norms' entry points must not be given: an output or a workspace over something that other
workgroups of the same launch still read (no GPU, nothing is launched)."""
import pytest

M = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from linear_recurrent_sequence_amd import retention
    return retention.load()


def _lnb(lib, **kw):
    a = dict(dy=1 * M, x=2 * M, w=3 * M, mean=4 * M, rstd=5 * M, ds=6 * M, dx=7 * M, dw=8 * M, db=9 * M, rows=4, D=64,
             xt=1, dyt=1, dxt=1, ws=10 * M, wsb=M)
    a.update(kw)
    return lib.ret_layer_norm_bwd(*list(a.values()), None, None)


@pytest.mark.parametrize("kw", [
    dict(ws=3 * M), dict(ws=4 * M), dict(ws=5 * M),          # the workspace over weight, mean, rstd
    dict(w=10 * M + 512), dict(mean=11 * M - 16), dict(rstd=10 * M),
    dict(dw=3 * M), dict(db=3 * M + 16), dict(dw=4 * M), dict(db=5 * M), dict(dw=M), dict(db=2 * M), dict(dw=6 * M),
    dict(dx=3 * M), dict(dx=4 * M), dict(dx=6 * M + 16),
], ids=str)
def test_layer_norm_gradients(lib, kw):
    assert _lnb(lib, **kw) == -1
    assert b"overlaps" in lib.ret_last_error()


def _epb(lib, **kw):
    a = dict(dy=1 * M, o=2 * M, gate=3 * M, w=4 * M, b=5 * M, do=6 * M, dg=7 * M, dw=8 * M, db=9 * M, rows=4, H=2, dv=64,
             t1=1, t2=1, t3=1, t4=1, t5=1, eps=1e-5, ws=10 * M, wsb=M)
    a.update(kw)
    return lib.ret_msr_epilogue_bwd(*list(a.values()), None, None)


@pytest.mark.parametrize("kw", [
    dict(ws=4 * M), dict(ws=5 * M), dict(w=10 * M + 512), dict(b=11 * M - 16),  # the workspace over weight, bias
    dict(dw=4 * M), dict(db=5 * M), dict(dw=5 * M + 16), dict(dw=M), dict(db=3 * M), dict(do=4 * M), dict(dg=5 * M),
    dict(do=M + 16), dict(dg=2 * M, t5=0), dict(do=7 * M),
], ids=str)
def test_epilogue_gradients(lib, kw):
    assert _epb(lib, **kw) == -1
    assert b"overlaps" in lib.ret_last_error()


def _ln(lib, **kw):
    a = dict(x=1 * M, res=2 * M, w=3 * M, b=4 * M, y=5 * M, sum=6 * M, mean=7 * M, rstd=8 * M, rows=4, D=64, xt=1, yt=1,
             eps=1e-5)
    a.update(kw)
    return lib.ret_layer_norm_fwd(*list(a.values()), None, None)


@pytest.mark.parametrize("kw", [
    dict(y=3 * M), dict(y=4 * M + 16), dict(sum=3 * M), dict(sum=4 * M), dict(mean=3 * M), dict(rstd=4 * M),
    dict(mean=M), dict(rstd=2 * M), dict(y=6 * M), dict(y=M + 16), dict(sum=2 * M, y=2 * M), dict(y=2 * M, yt=0),
    dict(mean=8 * M),
], ids=str)
def test_layer_norm(lib, kw):
    assert _ln(lib, **kw) == -1
    assert b"overlaps" in lib.ret_last_error()
