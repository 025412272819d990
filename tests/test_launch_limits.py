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
