"""RMS norm of rows whose squares leave fp32's range, above (entries past 1.8e19) or, where eps does not hide it, below (1e-19
and less): y is of the order of 1 all the same. Against 64 bits, with the tolerances of test_rms_norm.py. The reciprocal of a
root mean square above 2^126 has fewer digits, 2^-149 / 2^-128 of itself at most: 4 half steps, within the 64."""
import numpy as np
import pytest

from tests.conftest import print_case
from tests.scan_ref import U, close, half_step, rand
from tests.test_rms_norm import _check8

# a dtype's largest number, entries past the squares' range, one alone in its row, and what is just in range
LARGE = [3.3e38, 1e30, 3e19, 1.5e19]
SMALL = [1e-18, 1e-20, 1e-30, 1e-37]
# every number of lanes and values a lane
DIMS = [8, 24, 128, 100, 333, 512, 1000, 1024, 1001, 2048, 2049, 4096, 8192, 8200, 16383]


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


@pytest.mark.gpu
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [1e-5, 0.0, 1e30])
def test_rows_past_the_squares_range(R, D, kind, eps):
    import torch
    print_case("rms_norm_range", D, kind, eps)
    t = torch.float32 if kind == "f32" else torch.bfloat16
    gen = torch.Generator().manual_seed(D)
    rows = 2 * (len(LARGE) + len(SMALL) + 1) + 1
    x = rand(gen, rows, D)
    for i, top in enumerate(LARGE + SMALL):  # every second row is an ordinary one
        x[2 * i + 1] *= top / x[2 * i + 1].abs().max()
    x[-2, D // 2] = 1e25
    x, w = x.to(t), 1 + rand(gen, D, scale=0.2)
    assert torch.isfinite(x).all()
    x64, w64 = x.double().numpy(), w.double().numpy()
    r64 = 1 / np.sqrt((x64 ** 2).mean(-1) + np.float64(np.float32(eps)))
    ref = x64 * r64[:, None] * w64
    slack = 64 * U * np.abs(ref).max(1, keepdims=True)
    plain = None
    for group in (None, 32):
        y, rstd = torch.empty((rows, D), dtype=t, device="cuda"), torch.empty(rows, device="cuda")
        y8 = torch.empty((rows, D), dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty((rows, -(-D // group) if group else 1), device="cuda")
        R.ret_rms_norm_fwd(x.cuda(), y, w.cuda(), eps=eps, rstd=rstd, y8=y8, scales=scales, group=group)
        close("y", y, ref, half_step(t), slack)
        close("rstd", rstd, r64, 64 * U, 0.0)
        _check8(y8, scales, ref, slack, group)
        only = torch.empty_like(y)
        R.ret_rms_norm_fwd(x.cuda(), only, w.cuda(), eps=eps)
        assert torch.equal(only, y) and (plain is None or torch.equal(plain, y))
        plain = y
    # the rows in between are those of a call without the others
    ordinary, alone = x[::2].contiguous().cuda(), torch.empty((len(x[::2]), D), dtype=t, device="cuda")
    R.ret_rms_norm_fwd(ordinary, alone, w.cuda(), eps=eps)
    assert torch.equal(alone, plain[::2])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [24, 333, 4096])
def test_gradients_of_such_rows(R, D):
    """With the statistic of the forward call, of rows of 1e30 and (eps = 0) 1e-20, and of a residual's sum."""
    import torch
    print_case("rms_norm_range_bwd", D)
    gen = torch.Generator().manual_seed(D)
    x, res, dy, w = rand(gen, 5, D), rand(gen, 5, D), rand(gen, 5, D), 1 + rand(gen, D, scale=0.2)
    size = torch.tensor([1.0, 1e30, 1e-20, 1e35, 1e-15])[:, None]
    total, y, rstd = torch.empty(5, D, device="cuda"), torch.empty(5, D, device="cuda"), torch.empty(5, device="cuda")
    R.ret_rms_norm_fwd((x * size).cuda(), y, w.cuda(), eps=0.0, residual=(res * size).cuda(), sum_out=total, rstd=rstd)
    s64 = total.double().cpu().numpy()
    assert np.array_equal(s64, (x * size + res * size).double().numpy())
    close("rstd", rstd, 1 / np.sqrt((s64 ** 2).mean(-1)), 64 * U, 0.0)
    dx, dw = torch.empty_like(total), torch.empty(D, device="cuda")
    R.ret_rms_norm_bwd(dy.cuda(), total, rstd, dx, weight=w.cuda(), dweight=dw)
    rg, d64 = rstd.double().cpu().numpy()[:, None], dy.double().numpy()
    xh, a = s64 * rg, d64 * w.double().numpy()
    want = (a - xh * (a * xh).mean(-1, keepdims=True))
    bound = 64 * U * np.abs(a).max() * (1 + np.abs(xh).max() ** 2)
    got = dx.double().cpu().numpy() / rg
    assert (np.abs(got - want) <= bound).all()
    close("dweight", dw, (d64 * xh).sum(0), U, (5 + 64) * U * (np.abs(d64) * np.abs(xh)).sum(0))
