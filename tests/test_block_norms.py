"""Layer norm (forward, gradients) and the gradients of the multi-scale retention epilogue against 64-bit formulas.

Tolerances. An output of type t is off by its rounding, eps(t)/2 of the value, and by the fp32 arithmetic before it: a
statistic is at most 16 serial additions per lane and 10 levels of a tree, each value then a handful of operations, so
below 64 roundings of 2^-24 relative to the largest term. Column sums add, per column, the rows one after another in the
worst case: (rows + 64) 2^-24 of the sum of magnitudes. The hardware sigmoid adds 4 units of 2^-24.
"""
import numpy as np
import pytest

from tests.conftest import print_case

U = 2.0 ** -24


def _half_step(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


@pytest.fixture(scope="module")
def lib():
    from linear_recurrent_sequence_amd import retention
    return retention.load()


def _ln_ref(x, w, b, eps):
    mean = x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    xh = (x - mean) * rstd
    return xh * w + b, xh, mean[..., 0], rstd[..., 0]


def _close(name, got, ref, half, slack):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape
    err = np.abs(got - ref) - half * np.abs(ref)
    worst = float((err - slack).max()) if err.size else 0.0
    assert worst <= 0, "%s: off by %.3g more than its bound" % (name, worst)


DIMS = [1, 7, 8, 16, 100, 127, 128, 136, 256, 257, 512, 1000, 1001, 1024, 2048, 2056, 4096, 4097, 5000, 8192, 16383, 16384]


@pytest.mark.gpu
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("kind", ["f32", "bf16", "f32-bf16"])
def test_layer_norm(R, D, kind):
    import torch
    xt = torch.bfloat16 if kind == "bf16" else torch.float32
    yt = torch.float32 if kind == "f32" else torch.bfloat16
    for rows, residual, affine, offset in [(1, True, True, 0.0), (3, False, False, 100.0), (37, True, False, -3.0),
                                           (70, False, True, 0.5)]:
        print_case("layer_norm", D, kind, rows, residual, affine)
        g = torch.Generator().manual_seed(D * 100 + rows)
        x = (torch.randn(rows, D, generator=g) + offset).to(xt)
        res = torch.randn(rows, D, generator=g).to(xt) if residual else None
        w = 1 + 0.2 * torch.randn(D, generator=g) if affine else None
        b = 0.3 * torch.randn(D, generator=g) if affine else None
        dy = torch.randn(rows, D, generator=g).to(yt)
        dsum = torch.randn(rows, D, generator=g).to(xt) if residual else None
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        xd, y = x.cuda(), torch.empty((rows, D), dtype=yt, device="cuda")
        total = torch.empty_like(xd) if residual else None
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        R.ret_layer_norm_fwd(xd, y, dev(w), dev(b), residual=dev(res), sum_out=total, mean=mean, rstd=rstd)
        s = x if res is None else (x.float() + res.float()).to(xt)
        if residual:
            assert torch.equal(total.cpu(), s)
        s64 = s.double().numpy()
        w64, b64 = (1.0, 0.0) if w is None else (w.double().numpy(), b.double().numpy())
        ref, xh, m64, r64 = _ln_ref(s64, w64, b64, 1e-5)
        big = np.abs(s64).max() * r64.max()  # cancellation in s - mean is relative to s
        wmax = np.abs(w64).max()
        slack = 64 * U * ((1 + big + np.abs(xh).max()) * wmax + np.abs(b64).max())
        _close("y", y, ref, _half_step(yt), slack)
        _close("mean", mean, m64, U, 64 * U * np.abs(s64).max())
        _close("rstd", rstd, r64, 64 * U + 64 * U * big, 0.0)

        # gradients from the statistics as the forward left them
        dx = torch.empty((rows, D), dtype=xt, device="cuda")
        dw, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
        R.ret_layer_norm_bwd(dy.cuda(), total if residual else xd, mean, rstd, dx, weight=dev(w), dsum=dev(dsum),
                             dweight=dw, dbias=db)
        mg, rg = mean.double().cpu().numpy()[:, None], rstd.double().cpu().numpy()[:, None]
        xh = (s64 - mg) * rg
        d64 = dy.double().numpy()
        a = d64 * w64
        dref = rg * (a - a.mean(-1, keepdims=True) - xh * (a * xh).mean(-1, keepdims=True))
        scale = rg.max() * np.abs(a).max() * (1 + np.abs(xh).max() ** 2) * (1 + big)
        if residual:
            dref = dref + dsum.double().numpy()
            scale += np.abs(dsum.double().numpy()).max()
        _close("dx", dx, dref, _half_step(xt), 64 * U * scale)
        adds = rows + 64
        _close("dweight", dw, (d64 * xh).sum(0), U, adds * U * (np.abs(d64) * (np.abs(xh) + big)).sum(0).max())
        _close("dbias", db, d64.sum(0), U, adds * U * np.abs(d64).sum(0).max())


@pytest.mark.gpu
def test_layer_norm_gradient_against_differences(R):
    """dL/dx of L = sum(dy y) + sum(dsum s) against central differences of the kernel's own forward in fp32: step h
    leaves h^2 of the third derivative and 2^-24 |L| / h of rounding."""
    import torch
    g = torch.Generator().manual_seed(5)
    rows, D, h = 2, 24, 2.0 ** -6
    x, dy, ds = (torch.randn(rows, D, generator=g) for _ in range(3))
    w, b = 1 + 0.2 * torch.randn(D, generator=g), torch.randn(D, generator=g)

    def loss(xv):
        y = torch.empty_like(xv, device="cuda")
        R.ret_layer_norm_fwd(xv.cuda(), y, w.cuda(), b.cuda())
        return float((y.double().cpu() * dy.double()).sum() + (xv.double() * ds.double()).sum())

    y, m, r = torch.empty(rows, D, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    R.ret_layer_norm_fwd(x.cuda(), y, w.cuda(), b.cuda(), mean=m, rstd=r)
    dx = torch.empty(rows, D, device="cuda")
    R.ret_layer_norm_bwd(dy.cuda(), x.cuda(), m, r, dx, weight=w.cuda(), dsum=ds.cuda())
    for i, j in [(0, 0), (0, 23), (1, 7), (1, 16)]:
        e = torch.zeros_like(x)
        e[i, j] = h
        num = (loss(x + e) - loss(x - e)) / (2 * h)
        assert abs(num - float(dx[i, j])) <= 20 * h * h + 64 * U * 60 / h, (i, j, num, float(dx[i, j]))


@pytest.mark.gpu
def test_layer_norm_in_place_streams_and_empty(R):
    import torch
    g = torch.Generator().manual_seed(9)
    x, res = (torch.randn(5, 333, generator=g).cuda() for _ in range(2))
    want, total = torch.empty_like(x), torch.empty_like(x)
    R.ret_layer_norm_fwd(x, want, residual=res, sum_out=total)
    y, r2 = x.clone(), res.clone()
    R.ret_layer_norm_fwd(y, y, residual=r2, sum_out=r2)     # y over x, the sum over the residual
    assert torch.equal(y, want) and torch.equal(r2, total)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2 = torch.empty_like(x)
    R.ret_layer_norm_fwd(x, y2, residual=res, stream=s)
    m, r = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(y2, want)
    R.ret_layer_norm_fwd(x, y2, mean=m, rstd=r)
    dy = torch.randn(5, 333, generator=g).cuda()
    grads = []
    for stream in (None, s):
        s.wait_stream(torch.cuda.current_stream())
        dx, dw, db = torch.empty_like(x), torch.empty(333, device="cuda"), torch.empty(333, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        R.ret_layer_norm_bwd(dy, x, m, r, dx, dweight=dw, dbias=db, stream=stream)
        torch.cuda.synchronize()
        grads.append((dx, dw, db))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    d2 = dy.clone()
    R.ret_layer_norm_bwd(d2, x, m, r, d2)                    # dx over dy, no column sums
    assert torch.equal(d2, grads[0][0])
    e = torch.empty((0, 333), device="cuda")
    R.ret_layer_norm_fwd(e, torch.empty_like(e))
    dw, db = torch.ones(333, device="cuda"), torch.ones(333, device="cuda")
    em = torch.empty(0, device="cuda")
    R.ret_layer_norm_bwd(e, e, em, em, torch.empty_like(e), dweight=dw, dbias=db)
    assert not dw.any() and not db.any()


def _epi_ref(o, gate, w, b, dy, eps):
    mean = o.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((o - mean) ** 2).mean(-1, keepdims=True) + eps)
    xh = (o - mean) * rstd
    sg = 1 / (1 + np.exp(-gate)) if gate is not None else None
    dn = dy * gate * sg if gate is not None else dy
    dgate = dy * (xh * w + b) * sg * (1 + gate * (1 - sg)) if gate is not None else None
    a = dn * w
    do = rstd * (a - a.mean(-1, keepdims=True) - xh * (a * xh).mean(-1, keepdims=True))
    return do, dgate, dn, xh, rstd


@pytest.mark.gpu
@pytest.mark.parametrize("dv", [16, 32, 64, 128, 256, 512])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
def test_epilogue_gradients(R, dv, kind):
    import torch
    bf, f32 = torch.bfloat16, torch.float32
    types = {"f32": [f32] * 5, "bf16": [bf] * 5, "mixed": [f32, bf, bf, f32, bf]}[kind]
    for rows, H, gated, affine in [(1, 1, True, True), (33, 3, False, True), (70, 5, True, False), (600, 2, True, True)]:
        print_case("epilogue_bwd", dv, kind, rows, H, gated, affine)
        g = torch.Generator().manual_seed(dv + rows)
        dy, o = (torch.randn(rows, H, dv, generator=g).to(t) for t in types[:2])
        gate = (3 * torch.randn(rows, H, dv, generator=g)).to(types[2]) if gated else None
        w = 1 + 0.2 * torch.randn(H * dv, generator=g) if affine else None
        b = 0.3 * torch.randn(H * dv, generator=g) if affine else None
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        do = torch.empty((rows, H, dv), dtype=types[3], device="cuda")
        dgate = torch.empty((rows, H, dv), dtype=types[4], device="cuda") if gated else None
        dw, db = (torch.empty(H * dv, device="cuda") for _ in range(2))
        R.ret_msr_epilogue_bwd(dev(dy), dev(o), do, gate=dev(gate), dgate=dgate, gn_weight=dev(w), gn_bias=dev(b),
                               dweight=dw, dbias=db)
        n64 = lambda t: t.double().numpy()  # noqa: E731
        w64, b64 = (n64(w).reshape(H, dv), n64(b).reshape(H, dv)) if affine else (1.0, 0.0)
        rdo, rdg, dn, xh, rstd = _epi_ref(n64(o), n64(gate) if gated else None, w64, b64, n64(dy), 1e-5)
        big = np.abs(n64(o)).max() * rstd.max()
        xm = (np.abs(xh).max() + big) * np.abs(w64).max() + np.abs(b64).max()
        dnm = np.abs(dn).max()
        _close("do", do, rdo, _half_step(types[3]),
               64 * U * rstd.max() * dnm * np.abs(w64).max() * (1 + np.abs(xh).max() ** 2) * (1 + big))
        if gated:
            _close("dgate", dgate, rdg, _half_step(types[4]), 64 * U * np.abs(n64(dy)).max() * xm * 8)
        adds = rows + 64
        _close("dweight", dw, (dn * xh).sum(0).reshape(-1), U, adds * U * (np.abs(dn) * (np.abs(xh) + big)).sum(0).max())
        _close("dbias", db, dn.sum(0).reshape(-1), U, adds * U * np.abs(dn).sum(0).max())


@pytest.mark.gpu
def test_epilogue_gradient_follows_its_forward(R):
    """The gradients against central differences of ret_msr_epilogue in fp32 (see the layer norm's test)."""
    import torch
    g = torch.Generator().manual_seed(6)
    H, dv, h = 2, 16, 2.0 ** -6
    o, gate, dy = (torch.randn(1, H, dv, generator=g) for _ in range(3))
    w, b = 1 + 0.2 * torch.randn(H * dv, generator=g), torch.randn(H * dv, generator=g)

    def loss(ov, gv):
        y = torch.empty(1, H, dv, device="cuda")
        R.ret_msr_epilogue(ov.cuda(), y, gate=gv.cuda(), gn_weight=w.cuda(), gn_bias=b.cuda())
        return float((y.double().cpu() * dy.double()).sum())

    do, dg = (torch.empty(1, H, dv, device="cuda") for _ in range(2))
    R.ret_msr_epilogue_bwd(dy.cuda(), o.cuda(), do, gate=gate.cuda(), dgate=dg, gn_weight=w.cuda(), gn_bias=b.cuda())
    for hd, j in [(0, 0), (0, 15), (1, 3), (1, 8)]:
        e = torch.zeros_like(o)
        e[0, hd, j] = h
        tol = 20 * h * h + 64 * U * 40 / h
        assert abs((loss(o + e, gate) - loss(o - e, gate)) / (2 * h) - float(do[0, hd, j])) <= tol
        assert abs((loss(o, gate + e) - loss(o, gate - e)) / (2 * h) - float(dg[0, hd, j])) <= tol


@pytest.mark.gpu
def test_norm_gradients_replay_in_a_graph(R):
    """Layer norm forward and gradients and the epilogue's gradients captured once, replayed with new inputs and eager
    work between; every replay equals the eager call bit for bit (the sums have one order)."""
    import torch
    rows, H, dv = 300, 4, 64
    D = H * dv
    buf = {n: torch.empty(rows, D, dtype=torch.bfloat16, device="cuda") for n in ("x", "dy", "y", "dx", "do", "dg")}
    st = {n: torch.empty(rows, device="cuda") for n in ("mean", "rstd")}
    col = {n: torch.empty(D, device="cuda") for n in ("dw", "db", "ew", "eb")}
    w = torch.rand(D, device="cuda")
    ws, we = R.layer_norm_bwd_workspace(buf["x"]), R.msr_epilogue_bwd_workspace(buf["x"].view(rows, H, dv))
    v = lambda n: buf[n].view(rows, H, dv)  # noqa: E731

    def step():
        R.ret_layer_norm_fwd(buf["x"], buf["y"], weight=w, mean=st["mean"], rstd=st["rstd"])
        R.ret_layer_norm_bwd(buf["dy"], buf["x"], st["mean"], st["rstd"], buf["dx"], weight=w, dweight=col["dw"],
                             dbias=col["db"], workspace=ws)
        R.ret_msr_epilogue_bwd(v("dy"), v("x"), v("do"), gate=v("y"), dgate=v("dg"), gn_weight=w, dweight=col["ew"],
                               dbias=col["eb"], workspace=we)

    buf["x"].normal_(), buf["dy"].normal_()
    step()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        step()
    torch.cuda.synchronize()
    for i in range(3):
        buf["x"].normal_(), buf["dy"].normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in [*buf.values(), *st.values(), *col.values()]]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, [*buf.values(), *st.values(), *col.values()])), i


def _ln(lib, **kw):
    a = dict(x=1 << 20, res=None, w=None, b=None, y=2 << 20, sum=None, mean=None, rstd=None, rows=4, D=64, xt=1, yt=1,
             eps=1e-5)
    a.update(kw)
    return lib.ret_layer_norm_fwd(*list(a.values()), None, None)


def _lnb(lib, **kw):
    a = dict(dy=1 << 20, x=2 << 20, w=None, mean=3 << 20, rstd=4 << 20, ds=None, dx=5 << 20, dw=None, db=None, rows=4,
             D=64, xt=1, dyt=1, dxt=1, ws=None, wsb=0)
    a.update(kw)
    return lib.ret_layer_norm_bwd(*list(a.values()), None, None)


def _epb(lib, **kw):
    a = dict(dy=1 << 20, o=2 << 20, gate=None, w=None, b=None, do=3 << 20, dg=None, dw=None, db=None, rows=4, H=2, dv=64,
             t1=1, t2=1, t3=1, t4=1, t5=1, eps=1e-5, ws=None, wsb=0)
    a.update(kw)
    return lib.ret_msr_epilogue_bwd(*list(a.values()), None, None)


@pytest.mark.parametrize("fn,kw,status", [
    (_ln, dict(x=None), -1), (_ln, dict(y=None), -1), (_ln, dict(rows=-1), -1), (_ln, dict(D=0), -1),
    (_ln, dict(D=16385), -2), (_ln, dict(xt=2), -1), (_ln, dict(yt=-1), -1), (_ln, dict(eps=float("nan")), -1),
    (_ln, dict(eps=-1.0), -1), (_ln, dict(eps=float("inf")), -1), (_ln, dict(x=(1 << 20) + 4), -1),
    (_ln, dict(y=(1 << 20) + 16), -1),                    # y overlaps x
    (_ln, dict(y=1 << 20, yt=0), -1),                     # in place with another dtype
    (_ln, dict(sum=2 << 20), -1),                         # sum_out over y
    (_ln, dict(mean=2 << 20), -1), (_ln, dict(mean=3 << 20, rstd=3 << 20), -1), (_ln, dict(rows=1 << 50), -2),
    (_lnb, dict(dy=None), -1), (_lnb, dict(mean=None), -1), (_lnb, dict(dx=None), -1), (_lnb, dict(D=20000), -2),
    (_lnb, dict(dw=6 << 20), -3), (_lnb, dict(db=6 << 20, ws=7 << 20, wsb=8), -3), (_lnb, dict(dxt=5), -1),
    (_lnb, dict(dx=2 << 20, dxt=0), -1), (_lnb, dict(dw=6 << 20, db=6 << 20, ws=7 << 20, wsb=1 << 20), -1),
    (_lnb, dict(dw=6 << 20, ws=6 << 20, wsb=1 << 20), -1), (_lnb, dict(rows=-2), -1), (_lnb, dict(ds=(8 << 20) + 2), -1),
    (_epb, dict(dy=None), -1), (_epb, dict(do=None), -1), (_epb, dict(dg=4 << 20), -1), (_epb, dict(dv=48), -2),
    (_epb, dict(H=0), -1), (_epb, dict(rows=-1), -1), (_epb, dict(t3=7), -1), (_epb, dict(eps=-1.0), -1),
    (_epb, dict(dw=4 << 20), -3), (_epb, dict(do=(2 << 20) + 16), -1), (_epb, dict(o=(2 << 20) + 8), -1),
    (_epb, dict(gate=4 << 20, dg=3 << 20), -1),           # do over dgate
    (_epb, dict(dw=4 << 20, db=4 << 20, ws=5 << 20, wsb=1 << 20), -1), (_epb, dict(H=1 << 26), -2),
])
def test_refusals(lib, fn, kw, status):
    assert fn(lib, **kw) == status
    assert lib.ret_last_error() != b""


def test_workspace_queries(lib):
    assert lib.ret_layer_norm_bwd_workspace_bytes(-1, 64) == 0 and lib.ret_layer_norm_bwd_workspace_bytes(8, 0) == 0
    assert lib.ret_layer_norm_bwd_workspace_bytes(8, 16385) == 0 and lib.ret_layer_norm_bwd_workspace_bytes(0, 64) > 0
    assert lib.ret_msr_epilogue_bwd_workspace_bytes(8, 2, 48) == 0
    assert lib.ret_msr_epilogue_bwd_workspace_bytes(0, 2, 64) > 0
    # never more than a part of the rows: the sums of a batch stay small beside it
    assert lib.ret_layer_norm_bwd_workspace_bytes(1 << 20, 4096) <= 256 * 2 * 4096 * 4


def test_binding_checks():
    import torch
    from linear_recurrent_sequence_amd import retention as R
    x, f = torch.zeros(4, 64), torch.zeros(4)
    with pytest.raises(ValueError):
        R.ret_layer_norm_fwd(x, torch.zeros(4, 63))
    with pytest.raises(ValueError):
        R.ret_layer_norm_fwd(x, torch.zeros(4, 64), weight=torch.zeros(63))
    with pytest.raises(ValueError):
        R.ret_layer_norm_fwd(x, torch.zeros(4, 64), residual=torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        R.ret_layer_norm_fwd(x, torch.zeros(4, 64))  # not on a GPU
    with pytest.raises(ValueError):
        R.ret_layer_norm_fwd(x.half(), torch.zeros(4, 64))
    with pytest.raises(ValueError):
        R.ret_layer_norm_bwd(x, x, f, torch.zeros(5), x)
    with pytest.raises(ValueError):
        R.ret_layer_norm_bwd(x, x, f, None, x)
    o = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        R.ret_msr_epilogue_bwd(o, o, torch.zeros(4, 2, 32))
    with pytest.raises(ValueError):
        R.ret_msr_epilogue_bwd(o, o, torch.zeros_like(o), dgate=torch.zeros_like(o))
    with pytest.raises(ValueError):
        R.ret_msr_epilogue_bwd(o, o, torch.zeros_like(o), dweight=torch.zeros(64))
