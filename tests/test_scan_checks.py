"""Refusals and workspace queries of the selective scan, the short convolution and RMS norm (no GPU, nothing is launched), by
the C entry points and by the binding."""
import pytest

M = 1 << 24


@pytest.fixture(scope="module")
def lib():
    from linear_recurrent_sequence_amd import retention
    return retention.load()


def _scan(lib, **kw):
    a = dict(u=1 * M, dt=2 * M, A=3 * M, b=4 * M, bl=0, c=5 * M, cl=0, skip=6 * M, z=7 * M, zl=0, bias=8 * M, y=9 * M, B=1,
             N=300, D=64, S=16, G=1, ind=1, outd=1, sp=1, lengths=None, sin=None, sout=None, ws=12 * M, wsb=M)
    a.update(kw)
    return lib.ret_selective_scan_fwd(*list(a.values()), None, None)


def _step(lib, **kw):
    a = dict(u=1 * M, dt=2 * M, A=3 * M, b=4 * M, bl=0, c=5 * M, cl=0, skip=6 * M, z=7 * M, zl=0, bias=8 * M, y=9 * M,
             state=10 * M, B=1, D=64, S=16, G=1, ind=1, outd=1, sp=1)
    a.update(kw)
    return lib.ret_selective_scan_step(*list(a.values()), None, None)


def _bwd(lib, **kw):
    a = dict(u=1 * M, dt=2 * M, A=3 * M, b=4 * M, bl=0, c=5 * M, cl=0, skip=6 * M, z=7 * M, zl=0, bias=8 * M, dy=9 * M,
             du=20 * M, ddt=21 * M, dA=22 * M, db=23 * M, dc=24 * M, dskip=25 * M, dz=26 * M, dbias=27 * M, B=1, N=300, D=64,
             S=16, G=1, ind=1, outd=1, sp=1, lengths=None, sin=None, dsout=None, dsin=None, ws=30 * M, wsb=M)
    a.update(kw)
    return lib.ret_selective_scan_bwd(*list(a.values()), None, None)


@pytest.mark.parametrize("fn", [_scan, _step, _bwd])
@pytest.mark.parametrize("kw,status", [
    (dict(u=None), -1), (dict(dt=None), -1), (dict(A=None), -1), (dict(b=None), -1), (dict(c=None), -1),
    (dict(B=0), -1), (dict(D=0), -1), (dict(D=-64), -1), (dict(S=0), -1), (dict(G=0), -1),
    (dict(S=4), -2), (dict(S=12), -2), (dict(S=128), -2), (dict(G=3), -1), (dict(G=8), -2), (dict(D=96, G=4), -2),
    (dict(ind=2), -1), (dict(outd=-1), -1), (dict(ind=0, outd=1), -1),
    (dict(zl=63), -1), (dict(bl=15), -1), (dict(cl=-16), -1), (dict(zl=1 << 33), -2), (dict(bl=1 << 40), -2),
    (dict(u=M + 1), -1), (dict(b=4 * M + 1), -1), (dict(A=3 * M + 4), -1), (dict(skip=6 * M + 2), -1),
    (dict(D=1 << 27), -2),
], ids=str)
def test_refusals(lib, fn, kw, status):
    assert fn(lib, **kw) == status
    assert lib.ret_last_error() != b""


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), -1), (dict(N=0), -1), (dict(N=-5), -1), (dict(y=M), -1), (dict(y=7 * M), -1), (dict(sout=9 * M), -1),
    (dict(sin=11 * M, sout=11 * M + 64), -1), (dict(sout=3 * M), -1), (dict(lengths=11 * M + 2), -1),
    (dict(sin=11 * M + 8), -1), (dict(y=9 * M + 1), -1), (dict(D=48, N=5000, ws=None), -3), (dict(D=48, N=5000, wsb=64), -3),
    (dict(D=48, N=5000, ws=M), -1), (dict(B=1 << 20, N=1 << 20), -2),
    (dict(zl=200, y=7 * M + 200), -1),    # y between rows of z
], ids=str)
def test_sequence_refusals(lib, kw, status):
    assert _scan(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(state=None), -1), (dict(y=None), -1), (dict(state=9 * M), -1), (dict(state=3 * M), -1), (dict(state=10 * M + 4), -1),
    (dict(B=1 << 30), -2),
], ids=str)
def test_step_refusals(lib, kw, status):
    assert _step(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), -1), (dict(du=None), -1), (dict(ddt=None), -1), (dict(db=None), -1), (dict(dc=None), -1),
    (dict(z=None), -1), (dict(skip=None), -1), (dict(du=M), -1), (dict(dz=9 * M), -1), (dict(db=23 * M, dc=23 * M), -1),
    (dict(dA=3 * M), -1), (dict(dsout=31 * M, dsin=31 * M), -1), (dict(ws=None), -3), (dict(wsb=1 << 16), -3),
    (dict(ws=9 * M), -1), (dict(dsin=31 * M + 8), -1), (dict(dskip=25 * M + 2), -1), (dict(B=70000), -2),
], ids=str)
def test_gradient_refusals(lib, kw, status):
    assert _bwd(lib, **kw) == status


def test_scan_workspaces(lib):
    q = lambda *a: lib.ret_selective_scan_workspace_bytes(*a, None)  # noqa: E731
    g = lib.ret_selective_scan_bwd_workspace_bytes
    for bad in [(0, 64, 64, 16, 1, 1), (1, 0, 64, 16, 1, 1), (1, 64, 64, 24, 1, 1), (1, 64, 64, 16, 8, 1), (1, 64, 64, 16, 1, 7)]:
        assert q(*bad) == 0 and g(*bad) == 0
    assert q(64, 4096, 4096, 16, 1, 1) == 256             # no segments
    assert q(1, 65536, 1024, 16, 1, 1) > 1024 * 16 * 4     # some
    assert 0 < g(1, 64, 64, 16, 1, 1) < g(1, 640, 64, 16, 1, 1)


def _conv(lib, **kw):
    a = dict(x=1 * M, ld=0, w=2 * M, b=3 * M, y=4 * M, B=2, N=40, D=64, W=4, ind=1, outd=1, act=1, lengths=None, sin=None,
             sout=None)
    a.update(kw)
    return lib.ret_short_conv_fwd(*list(a.values()), None, None)


def _conv_bwd(lib, **kw):
    a = dict(dy=5 * M, x=1 * M, ld=0, w=2 * M, b=3 * M, y=4 * M, dw=6 * M, db=7 * M, B=2, N=40, D=64, W=4, ind=1, outd=1,
             act=1, lengths=None, sin=None, dsout=None, dsin=None, ws=8 * M, wsb=M)
    a.update(kw)
    return lib.ret_short_conv_bwd(*list(a.values()), None, None)


def _conv_step(lib, **kw):
    a = dict(x=1 * M, ld=0, w=2 * M, b=3 * M, y=4 * M, state=5 * M, B=2, D=64, W=4, ind=1, outd=1, act=1)
    a.update(kw)
    return lib.ret_short_conv_step(*list(a.values()), None, None)


@pytest.mark.parametrize("fn", [_conv, _conv_bwd, _conv_step])
@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(B=0), -1), (dict(D=0), -1), (dict(W=1), -2),
    (dict(W=5), -2), (dict(W=-1), -2), (dict(ind=3), -1), (dict(ind=0), -1), (dict(act=2), -1), (dict(ld=63), -1),
    (dict(ld=-64), -1), (dict(ld=1 << 33), -2), (dict(y=M), -1), (dict(y=2 * M), -1), (dict(x=M + 1), -1),
    (dict(y=4 * M + 8), -1), (dict(w=2 * M + 4), -1), (dict(D=(1 << 28) + 8), -2),
], ids=str)
def test_conv_refusals(lib, fn, kw, status):
    assert fn(lib, **kw) == status
    assert lib.ret_last_error() != b""


def test_conv_state_and_gradient_refusals(lib):
    assert _conv(lib, N=0) == -1 and _conv_bwd(lib, N=-1) == -1
    assert _conv(lib, sin=5 * M, sout=5 * M + 32) == -1 and _conv(lib, sout=M) == -1 and _conv(lib, lengths=5 * M + 1) == -1
    assert _conv(lib, B=1 << 30, N=1 << 20) == -2 and _conv(lib, B=1 << 20, N=1 << 15, D=8) == -2
    assert _conv_step(lib, state=None) == -1 and _conv_step(lib, state=M) == -1 and _conv_step(lib, state=4 * M) == -1
    assert _conv_bwd(lib, dy=None) == -1 and _conv_bwd(lib, dw=7 * M) == -1 and _conv_bwd(lib, dsin=4 * M) == -1
    assert _conv_bwd(lib, ws=None) == -3 and _conv_bwd(lib, wsb=100) == -3 and _conv_bwd(lib, ws=5 * M) == -1
    assert _conv_bwd(lib, dsout=9 * M, dsin=9 * M) == -1
    q = lib.ret_short_conv_bwd_workspace_bytes
    assert q(2, 40, 64, 5) == 0 and q(0, 40, 64, 4) == 0 and q(2, 40, 64, 4) >= 5 * 64 * 4


def _rms(lib, **kw):
    a = dict(x=1 * M, res=2 * M, w=3 * M, y=4 * M, sum=5 * M, rstd=6 * M, y8=7 * M, sc=8 * M, group=0, rows=4, D=64, xt=1,
             yt=1, eps=1e-5)
    a.update(kw)
    return lib.ret_rms_norm_fwd(*list(a.values()), None, None)


def _rms_bwd(lib, **kw):
    a = dict(dy=1 * M, x=2 * M, w=3 * M, rstd=5 * M, ds=6 * M, dx=7 * M, dw=8 * M, rows=4, D=64, xt=1, dyt=1, dxt=1,
             ws=10 * M, wsb=M)
    a.update(kw)
    return lib.ret_rms_norm_bwd(*list(a.values()), None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(y=None, y8=None, sc=None), -1), (dict(y8=None), -1), (dict(sc=None), -1), (dict(rows=-1), -1),
    (dict(D=0), -1), (dict(D=16385), -2), (dict(xt=2), -1), (dict(yt=-1), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(group=16), -1), (dict(group=256), -1),
    (dict(group=-32), -1), (dict(rows=1 << 41), -2), (dict(y8=M), -1), (dict(y8=4 * M), -1), (dict(sc=3 * M), -1),
    (dict(sc=8 * M + 2), -1), (dict(rstd=6 * M + 1), -1), (dict(y8=7 * M + 8), -1), (dict(x=M + 8), -1), (dict(y=3 * M), -1),
    (dict(y=M + 16), -1), (dict(y=2 * M, sum=2 * M), -1), (dict(rstd=M), -1), (dict(sum=3 * M), -1), (dict(y=M, yt=0), -1),
], ids=str)
def test_rms_refusals(lib, kw, status):
    assert _rms(lib, **kw) == status
    assert lib.ret_last_error() != b""


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), -1), (dict(x=None), -1), (dict(rstd=None), -1), (dict(dx=None), -1), (dict(D=20000), -2),
    (dict(rows=-2), -1), (dict(dxt=5), -1), (dict(ws=None), -3), (dict(wsb=128), -3), (dict(ws=3 * M), -1), (dict(dw=M), -1),
    (dict(dw=3 * M), -1), (dict(dx=3 * M), -1), (dict(dx=6 * M + 16), -1), (dict(ws=5 * M), -1), (dict(dx=M, dxt=0), -1),
], ids=str)
def test_rms_gradient_refusals(lib, kw, status):
    assert _rms_bwd(lib, **kw) == status


def test_rms_of_no_rows(lib):
    assert _rms(lib, rows=0, x=None, y=None, y8=None, sc=None) == 0
    assert lib.ret_rms_norm_bwd_workspace_bytes(0, 64) > 0 and lib.ret_rms_norm_bwd_workspace_bytes(4, 20000) == 0


class TestBinding:
    """What the binding refuses before it forms a pointer; the tensors are on the CPU or have no memory."""

    def _scan(self, **kw):
        import torch
        t = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="meta")  # noqa: E731
        f = lambda *s: torch.empty(s, device="meta")  # noqa: E731
        a = dict(u=t(2, 5, 32), dt=t(2, 5, 32), A=f(32, 16), b=t(2, 5, 1, 16), c=t(2, 5, 1, 16), y=t(2, 5, 32))
        return a | {k: v(t, f) if callable(v) else v for k, v in kw.items()}

    @pytest.mark.parametrize("kw", [
        dict(u=None), dict(dt=None), dict(A=None), dict(b=None), dict(c=None), dict(y=None),
        dict(u=lambda t, f: t(2, 32)), dict(dt=lambda t, f: t(2, 5, 31)), dict(dt=lambda t, f: f(2, 5, 32)),
        dict(A=lambda t, f: t(32, 16)), dict(A=lambda t, f: f(32, 8)), dict(b=lambda t, f: t(2, 5, 16)),
        dict(b=lambda t, f: t(2, 4, 1, 16)), dict(c=lambda t, f: t(2, 5, 2, 16)), dict(b=lambda t, f: t(2, 5, 3, 16)),
        dict(z=lambda t, f: t(2, 5, 16)), dict(d_skip=lambda t, f: f(31)), dict(dt_bias=lambda t, f: t(32)),
        dict(state_in=lambda t, f: f(2, 32, 8)), dict(state_out=lambda t, f: t(2, 32, 16)),
        dict(lengths=lambda t, f: f(2)), dict(y=lambda t, f: t(2, 5, 64)), dict(),  # the last: not on a GPU
    ], ids=lambda kw: "-".join(kw) or "meta")
    def test_scan(self, kw):
        from linear_recurrent_sequence_amd import retention as R
        with pytest.raises((ValueError, TypeError)):
            R.ret_selective_scan_fwd(**self._scan(**kw))

    @pytest.mark.parametrize("kw", [dict(x=(2, 5)), dict(weight=(31, 4)), dict(y=(2, 5, 31)), dict(bias=(31,)),
                                    dict(state_in=(2, 4, 32)), dict(state_out=(2, 2, 32)), dict(lengths=(3,)), dict()],
                             ids=lambda kw: "-".join(kw) or "cpu")
    def test_conv(self, kw):
        import torch

        from linear_recurrent_sequence_amd import retention as R
        a = dict(x=(2, 5, 32), weight=(32, 4), y=(2, 5, 32)) | kw
        a = {k: torch.zeros(s, dtype=torch.int32 if k == "lengths" else torch.float32) for k, s in a.items()}
        with pytest.raises(ValueError):
            R.ret_short_conv_fwd(**a)

    @pytest.mark.parametrize("kw", [dict(group=16), dict(group=1), dict(y=None), dict(scales=(3, 1)),
                                    dict(y8=(3, 64), scales=(3, 2)), dict(y8=(3, 64), scales=(3, 1), group=32),
                                    dict(y8=(3, 63), scales=(3, 1)), dict(rstd=(4,)), dict(weight=(63,)), dict()],
                             ids=lambda kw: "-".join(kw) or "cpu")
    def test_rms(self, kw):
        import torch

        from linear_recurrent_sequence_amd import retention as R
        a = dict(x=(3, 64), y=(3, 64)) | kw
        a = {k: torch.zeros(s, dtype=torch.uint8 if k == "y8" else torch.float32) if isinstance(s, tuple) else s
             for k, s in a.items()}
        with pytest.raises(ValueError):
            R.ret_rms_norm_fwd(**a)

    def test_sizes_past_31_bits(self):
        import torch

        from linear_recurrent_sequence_amd import retention as R
        big = 2 ** 32 + 16
        t = lambda *s: torch.empty(s, device="meta")  # noqa: E731
        calls = [
            lambda: R.ret_rms_norm_fwd(t(1, big), t(1, big)), lambda: R.rms_norm_bwd_workspace(t(1, big)),
            lambda: R.ret_rms_norm_bwd(t(1, big), t(1, big), t(1), t(1, big)),
            lambda: R.ret_short_conv_fwd(t(1, big, 1), t(1, 4), t(1, big, 1)),
            lambda: R.ret_short_conv_fwd(t(1, 1, big), t(big, 4), t(1, 1, big)),
            lambda: R.short_conv_bwd_workspace(t(1, big, 1), t(1, 4)),
            lambda: R.ret_short_conv_step(t(big, 1), t(1, 4), t(big, 1), t(big, 3, 1)),
            lambda: R.selective_scan_workspace(t(1, big, 1), t(1, big, 1, 16)),
            lambda: R.selective_scan_bwd_workspace(t(1, 1, big), t(1, 1, 1, 16)),
            lambda: R.ret_selective_scan_fwd(t(1, big, 1), t(1, big, 1), t(1, 16), t(1, big, 1, 16), t(1, big, 1, 16),
                                             t(1, big, 1)),
        ]
        for call in calls:
            with pytest.raises(ValueError, match="2.31"):
                call()

    def test_rows_of_slices(self):
        """The distance between rows that a slice of wider rows has, and the ones that are refused."""
        import torch

        from linear_recurrent_sequence_amd import retention as R

        class OnGpu:
            is_cuda = True

            def __init__(self, t):
                self.shape, self._t = t.shape, t

            def stride(self):
                return self._t.stride()

            def data_ptr(self):
                return self._t.data_ptr()
        wide = torch.zeros(3, 5, 100)
        rows = lambda t, inner=1: R._token_rows(OnGpu(t), "t", inner)[1]  # noqa: E731
        assert rows(wide) == 100 and rows(wide[..., 7:39]) == 100 and rows(wide[:, :1, :32]) == 500
        assert rows(wide[:1, :, :32]) == 100 and rows(wide[1:, 2:3, 4:5]) == 500 and rows(wide[:1, :1, :32]) == 32
        assert rows(wide[..., :32].unflatten(-1, (2, 16)), 2) == 100
        assert R._token_rows(None, "t", 1) == (None, 0)
        for bad in (wide[..., ::2], wide[:, :4], wide[:, ::2], wide.transpose(0, 1), wide[:, :, :1].expand(3, 5, 8),
                    wide[:1, :1].expand(3, 5, 100)):
            with pytest.raises(ValueError):
                rows(bad)
        with pytest.raises(ValueError):
            rows(wide[..., :64].unflatten(-1, (2, 32))[..., :16], 2)
