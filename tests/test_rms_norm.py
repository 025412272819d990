"""RMS norm (forward, 8 bits, gradients) against 64 bits. Tolerances as in test_block_norms.py: below 64 roundings of 2^-24
of the largest term, column sums (rows + 64). In 8 bits: half a step of e4m3 (2^-4 of the value, 2^-10 of the scale below
2^-6) on top, and an ulp of the reciprocal of the scale."""
import numpy as np
import pytest

from tests.conftest import print_case
from tests.scan_ref import U, close, half_step, rand

DIMS = [1, 7, 8, 16, 31, 32, 33, 100, 128, 136, 256, 257, 300, 512, 513, 1000, 1001, 1024, 2048, 2049, 4096, 4097, 8192,
        8200, 16383, 16384]


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


def _check8(y8, scales, y, slack, group):
    """y8 scales is y; the scales are the groups' maxima over 448."""
    rows, D = y.shape
    g = group or D
    q, sc = y8.float().double().cpu().numpy(), scales.double().cpu().numpy()
    assert sc.shape == (rows, -(-D // g))
    for i in range(sc.shape[1]):
        part = slice(i * g, min(D, (i + 1) * g))
        top = np.abs(y[:, part]).max(1) / 448
        assert (np.abs(sc[:, i] - top) <= 4 * U * top + slack[:, 0] / 448 + 2.0 ** -126).all()
        want, k = y[:, part], sc[:, i:i + 1]
        bound = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * k + 4 * U * np.abs(want) + slack
        assert (np.abs(q[:, part] * k - want) <= bound).all()
        assert (np.abs(q[:, part]) <= 448).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("kind", ["f32", "bf16", "f32-bf16"])
def test_rms_norm(R, D, kind):
    import torch
    xt = torch.bfloat16 if kind == "bf16" else torch.float32
    yt = torch.float32 if kind == "f32" else torch.bfloat16
    for rows, residual, weighted, group in [(1, True, True, None), (3, False, False, 32), (37, True, False, 64),
                                            (70, False, True, 128)]:
        print_case("rms_norm", D, kind, rows, residual, weighted, group)
        gen = torch.Generator().manual_seed(D * 100 + rows)
        x = (rand(gen, rows, D) + 0.5).to(xt)
        res = rand(gen, rows, D, dtype=xt) if residual else None
        w = 1 + rand(gen, D, scale=0.2) if weighted else None
        dy, dsum = rand(gen, rows, D, dtype=yt), rand(gen, rows, D, dtype=xt) if residual else None
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        xd, y = x.cuda(), torch.empty((rows, D), dtype=yt, device="cuda")
        total = torch.empty_like(xd) if residual else None
        rstd = torch.empty(rows, device="cuda")
        y8 = torch.empty((rows, D), dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty((rows, -(-D // group) if group else 1), device="cuda")
        R.ret_rms_norm_fwd(xd, y, dev(w), residual=dev(res), sum_out=total, rstd=rstd, y8=y8, scales=scales, group=group)
        s = x if res is None else (x.float() + res.float()).to(xt)
        if residual:
            assert torch.equal(total.cpu(), s)
        s64, w64 = s.double().numpy(), 1.0 if w is None else w.double().numpy()
        r64 = 1 / np.sqrt((s64 ** 2).mean(-1) + 1e-5)
        ref = s64 * r64[:, None] * w64
        slack = 64 * U * np.abs(ref).max(1, keepdims=True)
        close("y", y, ref, half_step(yt), slack)
        close("rstd", rstd, r64, 64 * U, 0.0)
        _check8(y8, scales, ref, slack, group)
        only = torch.empty_like(y8)
        again = torch.empty_like(scales)
        R.ret_rms_norm_fwd(xd, weight=dev(w), residual=dev(res), y8=only, scales=again, group=group)
        assert torch.equal(only.view(torch.uint8), y8.view(torch.uint8)) and torch.equal(again, scales)
        y2 = torch.empty_like(y)
        R.ret_rms_norm_fwd(xd, y2, dev(w), residual=dev(res))
        assert torch.equal(y2, y)

        dx, dw = torch.empty((rows, D), dtype=xt, device="cuda"), torch.empty(D, device="cuda")
        R.ret_rms_norm_bwd(dy.cuda(), total if residual else xd, rstd, dx, weight=dev(w), dsum=dev(dsum), dweight=dw)
        rg = rstd.double().cpu().numpy()[:, None]
        xh, d64 = s64 * rg, dy.double().numpy()
        a = d64 * w64
        dref = rg * (a - xh * (a * xh).mean(-1, keepdims=True))
        scale = rg.max() * np.abs(a).max() * (1 + np.abs(xh).max() ** 2)
        if residual:
            dref = dref + dsum.double().numpy()
            scale += np.abs(dsum.double().numpy()).max()
        close("dx", dx, dref, half_step(xt), 64 * U * scale)
        close("dweight", dw, (d64 * xh).sum(0), U, (rows + 64) * U * (np.abs(d64) * np.abs(xh)).sum(0))


@pytest.mark.gpu
def test_gradient_against_differences(R):
    """dL/dx of L = sum(dy y) + sum(dsum s) against central differences of the 64-bit formula: a step of 1e-5 leaves 1e-10 of
    the third derivative (below 1e3 here) and 1e-10 of rounding; the gradient its fp32 arithmetic."""
    import torch
    gen = torch.Generator().manual_seed(5)
    rows, D = 2, 24
    x, dy, ds, w = rand(gen, rows, D), rand(gen, rows, D), rand(gen, rows, D), 1 + rand(gen, D, scale=0.2)
    y, r = torch.empty(rows, D, device="cuda"), torch.empty(rows, device="cuda")
    R.ret_rms_norm_fwd(x.cuda(), y, w.cuda(), rstd=r)
    dx, dw = torch.empty(rows, D, device="cuda"), torch.empty(D, device="cuda")
    R.ret_rms_norm_bwd(dy.cuda(), x.cuda(), r, dx, weight=w.cuda(), dsum=ds.cuda(), dweight=dw)

    def loss(xv, wv):
        out = xv * wv / (xv.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        return float((out * dy.double()).sum() + (xv * ds.double()).sum())

    for which, grad in (("x", dx), ("w", dw)):
        way = torch.randn(grad.shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        at = lambda k: (x.double() + k * way, w.double()) if which == "x" else (x.double(), w.double() + k * way)  # noqa: E731
        num = (loss(*at(h)) - loss(*at(-h))) / (2 * h)
        got = float((grad.double().cpu() * way).sum())
        assert abs(num - got) <= 1e-6 + 64 * U * 500, (which, num, got)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [24, 333, 4096])
@pytest.mark.parametrize("group", [None, 32, 128])
def test_odd_rows(R, D, group):
    """Rows of zeros, of the smallest and largest numbers, with a NaN and with an infinity; the rows around them unchanged."""
    import torch
    gen = torch.Generator().manual_seed(7)
    x = rand(gen, 9, D).cuda()
    want8, want = torch.empty((9, D), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty_like(x)
    n = -(-D // group) if group else 1
    sc = torch.empty((9, n), device="cuda")
    R.ret_rms_norm_fwd(x, want, y8=want8, scales=sc, group=group)
    bad = x.clone()
    bad[1] = 0
    bad[3] = 1e-30
    bad[5, 2] = float("nan")
    bad[7, 2] = float("inf")
    y, y8, s2 = torch.empty_like(x), torch.empty_like(want8), torch.empty_like(sc)
    R.ret_rms_norm_fwd(bad, y, y8=y8, scales=s2, group=group, eps=0.0)
    assert y[1].isnan().all() and y[5].isnan().all()
    R.ret_rms_norm_fwd(bad, y, y8=y8, scales=s2, group=group)
    same = [0, 2, 4, 6, 8]
    assert torch.equal(y[same], want[same]) and torch.equal(s2[same], sc[same])
    assert torch.equal(y8.view(torch.uint8)[same], want8.view(torch.uint8)[same])
    assert not y[1].any() and not y8[1].float().any() and (s2[1] == 2.0 ** -126).all()
    assert torch.isfinite(s2[3]).all() and torch.isfinite(y8[3].float()).all()
    assert y[5].isnan().all() and y8[5].float().isnan().all() and s2[5].isnan().all()
    assert y[7, 2].isnan() and y8[7, 2].float().isnan() and s2[7, 0].isnan()
    assert not y[7, 3:].any()


@pytest.mark.gpu
def test_in_place_streams_and_empty(R):
    import torch
    gen = torch.Generator().manual_seed(9)
    x, res = (rand(gen, 5, 333).cuda() for _ in range(2))
    want, total = torch.empty_like(x), torch.empty_like(x)
    R.ret_rms_norm_fwd(x, want, residual=res, sum_out=total)
    y, r2 = x.clone(), res.clone()
    R.ret_rms_norm_fwd(y, y, residual=r2, sum_out=r2)  # y over x, the sum over the residual
    assert torch.equal(y, want) and torch.equal(r2, total)
    s, y2, r = torch.cuda.Stream(), torch.empty_like(x), torch.empty(5, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    R.ret_rms_norm_fwd(x, y2, residual=res, rstd=r, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y2, want)
    dy = rand(gen, 5, 333).cuda()
    grads = []
    for stream in (None, s):
        dx, dw = torch.empty_like(x), torch.empty(333, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        R.ret_rms_norm_bwd(dy, total, r, dx, dweight=dw, stream=stream)
        torch.cuda.synchronize()
        grads.append((dx, dw))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    d2 = dy.clone()
    R.ret_rms_norm_bwd(d2, total, r, d2)  # dx over dy, no column sums
    assert torch.equal(d2, grads[0][0])
    e, em, dw = torch.empty((0, 333), device="cuda"), torch.empty(0, device="cuda"), torch.ones(333, device="cuda")
    R.ret_rms_norm_fwd(e, torch.empty_like(e))
    R.ret_rms_norm_bwd(e, e, em, torch.empty_like(e), dweight=dw)
    assert not dw.any()
    many = torch.randn((70000, 64), device="cuda")
    out, st = torch.empty_like(many), torch.empty(70000, device="cuda")
    R.ret_rms_norm_fwd(many, out, rstd=st)
    ref = many.double() * (many.double().square().mean(1, keepdim=True) + 1e-5).rsqrt()
    assert float((out.double() - ref).abs().max()) <= 64 * U * 8
    dw, dm = torch.empty(64, device="cuda"), torch.empty_like(many)
    R.ret_rms_norm_bwd(out, many, st, dm, dweight=dw)  # several rounds of rows a workgroup
    terms = out.double() * many.double() * st.double()[:, None]
    assert ((dw.double() - terms.sum(0)).abs() <= (70000 + 64) * U * terms.abs().sum(0)).all()
