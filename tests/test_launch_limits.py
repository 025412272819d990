"""Sizes at the limits of a launch (2^32 work-items) and of 32-bit chunk counts."""
import pytest

T = 1 << 40  # far enough apart for any of these sizes


@pytest.fixture(scope="module")
def lib():
    from linear_recurrent_sequence_amd import retention
    return retention.load()


@pytest.mark.parametrize("H,dv", [(1 << 21, 64), (1 << 18, 512), (1 << 23, 16)])
def test_epilogue_gradients_refuse_more_channels_than_their_sums_launch(lib, H, dv):
    st = lib.ret_msr_epilogue_bwd(T, 2 * T, None, None, None, 3 * T, None, 4 * T, None, 1, H, dv, 1, 1, 1, 1, 1, 1e-5,
                                  5 * T, 1 << 32, None, None)
    assert st == -2 and lib.ret_msr_epilogue_bwd_workspace_bytes(1, H, dv) == 0
    assert lib.ret_msr_epilogue_bwd_workspace_bytes(1, H - 1, dv) == 8 * (H - 1) * dv


@pytest.mark.gpu
def test_layer_norm_of_more_rows_than_one_launch_axis_takes():
    """2^26 rows of a width whose workgroups of 256 threads hold 4 rows: 2^32 work-items. Bit for bit what calls on parts
    of the rows give, and the last rows against the formula (64 roundings of 2^-24 of the largest value and of 1)."""
    import torch

    from linear_recurrent_sequence_amd import retention as R
    from tests.conftest import print_case
    rows, D = (1 << 26) + 5, 7
    print_case("layer_norm_rows", rows, D)
    x = torch.randn(rows, D, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    y, part = torch.empty_like(x), torch.empty_like(x)
    mean = torch.empty(rows, device="cuda")
    R.ret_layer_norm_fwd(x, y, mean=mean)
    for a in range(0, rows, 1 << 24):
        R.ret_layer_norm_fwd(x[a:a + (1 << 24)], part[a:a + (1 << 24)])
    assert torch.equal(y, part)
    last = x[-9:].double().cpu()
    ref = (last - last.mean(1, keepdim=True)) / (last.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    tol = 64 * 2.0 ** -24 * (1 + last.abs().max() / last.std(1, unbiased=False).min()) * ref.abs().max()
    assert float((y[-9:].double().cpu() - ref).abs().max()) <= float(tol)
    assert float((mean[-9:].double().cpu() - last.mean(1)).abs().max()) <= 64 * 2.0 ** -24 * float(last.abs().max())
