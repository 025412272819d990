"""Sequences of nearly 2^31 tokens in the short convolution's checks and plans (no GPU, nothing is launched: a misaligned pointer,
or no workspace, is refused after the sizes have passed)."""
import pytest

T = 1 << 40  # far enough apart for any of these sizes
MOST = 2 ** 31 - 17


@pytest.fixture(scope="module")
def lib():
    from linear_recurrent_sequence_amd import retention
    return retention.load()


def _fwd(lib, N, B=1, D=8):
    """-1 (misaligned lengths) where the sizes pass."""
    return lib.ret_short_conv_fwd(T, 0, 2 * T, None, 3 * T, B, N, D, 4, 1, 1, 1, 4 * T + 1, None, None, None, None)


def _bwd(lib, N, B=1, D=8):
    """-3 (no workspace) where the sizes pass."""
    return lib.ret_short_conv_bwd(T, 2 * T, 0, 3 * T, None, 4 * T, 5 * T, 6 * T, B, N, D, 4, 1, 1, 1, None, None, None, None,
                                  None, 0, None, None)


@pytest.mark.parametrize("N", [2 ** 30, 2 ** 31 - 200, 2 ** 31 - 128, 2 ** 31 - 64, 2 ** 31 - 32, MOST])
@pytest.mark.parametrize("B", [1, 2, 3])
def test_long_sequences_are_taken(lib, N, B):
    # a sequence has up to 2^25 strips, four to a workgroup of 256 threads: 2^31 work-items, of which two fit a launch
    fits = B * -(-N // 256) * 256 < 2 ** 32
    assert _fwd(lib, N, B) == (-1 if fits else -2) and (b"lengths" if fits else b"launch") in lib.ret_last_error()
    assert _bwd(lib, N, B) == -3
    # 1024 workgroups, each a row of (W + 1) D sums
    assert lib.ret_short_conv_bwd_workspace_bytes(B, N, 8, 4) == 1024 * 5 * 8 * 4


@pytest.mark.parametrize("N", [MOST + 1, 2 ** 31 - 1])
def test_longer_ones_are_refused(lib, N):
    assert _fwd(lib, N) == -2 and b"too large" in lib.ret_last_error()
    assert _bwd(lib, N) == -2 and b"too large" in lib.ret_last_error()
    assert lib.ret_short_conv_bwd_workspace_bytes(1, N, 8, 4) == 0


@pytest.mark.parametrize("B,N,D", [(1 << 20, (1 << 20) + 1, 8), (1, 64, (1 << 28) + 8)])
def test_no_workspace_for_sizes_that_are_refused(lib, B, N, D):
    assert _bwd(lib, N, B, D) == -2 and lib.ret_short_conv_bwd_workspace_bytes(B, N, D, 4) == 0
