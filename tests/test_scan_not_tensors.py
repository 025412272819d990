"""What is not a tensor is refused with a ValueError that names it, by the calls of the selective scan, the short convolution and
RMS norm, as by the calls before them."""
import pytest


def test_the_checks_themselves():
    import torch

    from linear_recurrent_sequence_amd import retention as R
    for bad in ([1.0], 3, "z", (torch.ones(1),)):
        with pytest.raises(ValueError, match="z must be a tensor"):
            R._rows_arg(bad, "z", (1,), (torch.float32,), 0, 1)
        with pytest.raises(ValueError, match="workspace must be a tensor"):
            R._workspace(bad, 0)
    assert R._rows_arg(None, "z", (1,), (torch.float32,), 0, 1) == (None, 0) and R._workspace(None, 0) == (None, 0)


@pytest.fixture(scope="module")
def calls():
    """{call: (function, its arguments)} that pass."""
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention as R
    R.load(build_if_missing=True)
    e = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    B, N, D, S, W = 1, 4, 16, 8, 4
    scan = dict(u=e(B, N, D), dt=e(B, N, D), A=-e(D, S), b=e(B, N, 1, S), c=e(B, N, 1, S), z=e(B, N, D))
    step = {k: v if k == "A" else v[:, 0] for k, v in scan.items()}
    grads = dict(dy=e(B, N, D), du=e(B, N, D), ddt=e(B, N, D), dA=e(D, S), db=e(B, N, 1, S), dc=e(B, N, 1, S), dz=e(B, N, D))
    return {
        "rms": (R.ret_rms_norm_fwd, dict(x=e(2, D), y=e(2, D), weight=e(D), residual=e(2, D), sum_out=e(2, D), rstd=e(2))),
        "rms gradients": (R.ret_rms_norm_bwd, dict(dy=e(2, D), x=e(2, D), rstd=e(2), dx=e(2, D), weight=e(D), dweight=e(D),
                                                   workspace=R.rms_norm_bwd_workspace(e(2, D)))),
        "conv": (R.ret_short_conv_fwd, dict(x=e(B, N, D), weight=e(D, W), y=e(B, N, D), state_out=e(B, W - 1, D))),
        "conv gradients": (R.ret_short_conv_bwd, dict(
            dy=e(B, N, D), x=e(B, N, D), weight=e(D, W), dx=e(B, N, D), dweight=e(D, W), dstate_in=e(B, W - 1, D),
            workspace=R.short_conv_bwd_workspace(e(B, N, D), e(D, W)))),
        "conv step": (R.ret_short_conv_step, dict(x=e(B, D), weight=e(D, W), y=e(B, D), state=e(B, W - 1, D))),
        "scan": (R.ret_selective_scan_fwd, dict(scan, y=e(B, N, D), workspace=R.selective_scan_workspace(scan["u"], scan["b"]))),
        "scan step": (R.ret_selective_scan_step, dict(step, y=e(B, D), state=e(B, D, S))),
        "scan gradients": (R.ret_selective_scan_bwd, dict(scan, **grads, workspace=R.selective_scan_bwd_workspace(
            scan["u"], scan["b"]))),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["rms", "rms gradients", "conv", "conv gradients", "conv step", "scan", "scan step",
                                  "scan gradients"])
def test_every_argument(calls, name):
    import numpy as np
    fn, args = calls[name]
    fn(**args)
    for key, t in args.items():
        for bad in ([1.0], np.ones(tuple(t.shape), np.float32)):
            with pytest.raises(ValueError, match="(^|[ ,])%s must be|must be .*%s" % (key, key)):
                fn(**dict(args, **{key: bad}))
