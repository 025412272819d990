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


def _delta(lib, bwd=False, B=1, N=1, H=1, dk=32, dv=16, dt=1, segments=0, ws=None):
    """The call with buffers far apart and no workspace: -3 where all checks before that pass."""
    from linear_recurrent_sequence_amd import retention
    opts = retention._options({"segments": segments})
    shape = (B, N, H, H, dk, dv, dt, dt, 0, 0.0)
    if bwd:
        return lib.ret_gated_delta_bwd(*[T * i for i in range(1, 12)], *shape, None, None, None, None, None, 0, None, opts)
    return lib.ret_gated_delta_fwd(*[T * i for i in range(1, 7)], *shape, None, None, None, None, 0, None, opts)


@pytest.mark.parametrize("bwd", [False, True])
def test_delta_calls_refuse_what_a_launch_does_not_hold(lib, bwd):
    query = lib.ret_gated_delta_bwd_workspace_bytes if bwd else lib.ret_gated_delta_workspace_bytes
    # 60000 heads of 139 blocks of 128 columns, 512 threads each: 0.994 x 2^32 work-items; one block more
    assert _delta(lib, bwd, B=300, H=200, dv=139 * 128) == -3
    assert _delta(lib, bwd, B=300, H=200, dv=140 * 128) == -2 and b"launch" in lib.ret_last_error()
    assert query(300, 1, 200, 200, 32, 140 * 128, 1, None) == 0 < query(300, 1, 200, 200, 32, 139 * 128, 1, None)
    # the segment scan has d_v / 32 workgroups along y
    assert _delta(lib, bwd, N=512, dv=1 << 21) == -3
    assert _delta(lib, bwd, N=512, dv=1 << 21, segments=2) == -2
    assert _delta(lib, bwd, N=512, dv=(1 << 21) - 32, segments=2) == -3
    # chunks of tokens
    for N in (2 ** 31 - 1, 2 ** 31 - 64, 2 ** 30):
        assert _delta(lib, bwd, N=N) == -2 and query(1, N, 1, 1, 32, 16, 1, None) == 0


def test_delta_step_refuses_what_a_launch_does_not_hold(lib):
    step = lambda dv, state=7 * T: lib.ret_gated_delta_step(*[T * i for i in range(1, 7)], state, 1, 1, 1, 16, dv,  # noqa: E731
                                                            1, 1, 0, 0.0, None, None)
    assert step((1 << 22) - 16, None) == -1  # a missing state comes first
    assert step((1 << 22) - 16) == -2


def test_normalized_form_refuses_what_a_launch_does_not_hold(lib):
    """2^35 outputs, 68 GB in bf16: 8 a work-item."""
    import ctypes
    H = 64
    gamma = (ctypes.c_float * H)(*[0.9] * H)
    call = lambda N: lib.ret_chunkwise_normalized_fwd(T, 2 * T, 3 * T, 4 * T, 1, N, H, 64, 512, 1, 1, gamma, None, 0,  # noqa: E731
                                                      64, 7, None, None, None, None, None, 0, None, None)
    assert call((1 << 20) - 64) == -3  # nothing but the workspace is missing
    assert call(1 << 20) == -2 and b"launch" in lib.ret_last_error()
