"""Sums over several rounds of a workgroup (the short convolution's strips, RMS norm's rows), the longer strips, and sizes at the
edges of the blocks that the kernels of the selective scan's block have, against 64 bits. Tolerances as in test_short_conv.py,
test_rms_norm.py and test_selective_scan.py."""
import numpy as np
import pytest

from tests import test_selective_scan as scan_tests
from tests import test_short_conv as conv_tests
from tests.conftest import print_case
from tests.scan_ref import U, close, conv, half_step, rand


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


def _rounds(B, N, D, W, lib):
    """Strips that a wave of the gradients takes one after another, by the workspace's partial rows; strips are 128 there."""
    parts = lib.ret_short_conv_bwd_workspace_bytes(B, N, D, W) // (4 * (W + 1) * D)
    return -(-B * -(-N // 128) // (4 * parts))


# more than one round of strips of 128 tokens, the last of them not full; the forward's strips are 64
@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(3, 6000, 8192, 4, "bf16"), (40, 450, 8192, 4, "f32"), (5, 1100, 8191, 4, "bf16"),
                                   (5, 1100, 8191, 3, "f32"), (40, 450, 8192, 2, "bf16-f32"), (70, 300, 8192, 3, "bf16")], ids=str)
def test_convolution_over_rounds(R, shape):
    """A sample of channels in full: each is a convolution of its own."""
    import torch
    B, N, D, W, kind = shape
    print_case("short_conv_rounds", shape)
    assert _rounds(B, N, D, W, R.load()) == 2
    tin, tout = conv_tests._types(kind)
    gen = torch.Generator(device="cuda").manual_seed(N + W)
    new = lambda *n, dtype=torch.float32: torch.randn(n, generator=gen, device="cuda").to(dtype)  # noqa: E731
    x, dy, w, b = new(B, N, D, dtype=tin), new(B, N, D, dtype=tin), new(D, W), new(D)
    s0, ds = new(B, W - 1, D, dtype=tin), new(B, W - 1, D, dtype=tout)
    lengths = [(N, N - 1, N // 2 + 1, 129, 128, 0, 65, 64)[i % 8] for i in range(B)]
    ld = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    pick = torch.tensor([0, 1, 62, 63, 64, 65, 255, 256, 257, 1000, 4095, 4096, 7935, 7936, D - 2, D - 1], device="cuda")
    take = lambda t, axis=-1: t.index_select(axis, pick).cpu()  # noqa: E731
    args = (take(x), take(w, 0), take(b), True, lengths, take(s0), take(dy), take(ds))
    want, size = conv(*args), conv(*args, absolute=True)
    for i, n in enumerate(lengths):
        x[i, n:] = dy[i, n:] = float("nan")
    y, last = torch.empty(B, N, D, dtype=tout, device="cuda"), torch.empty_like(s0)
    R.ret_short_conv_fwd(x, w, y, bias=b, lengths=ld, state_in=s0, state_out=last)
    close("y", take(y), want[0], half_step(tout), 16 * U * size[0])
    assert torch.equal(take(last).double(), torch.from_numpy(want[1]))
    dx, dw, db, d0 = torch.empty_like(y), torch.empty_like(w), torch.empty_like(b), torch.empty_like(ds)
    R.ret_short_conv_bwd(dy, x, w, dx, dw, bias=b, dbias=db, lengths=ld, state_in=s0, dstate_out=ds, dstate_in=d0)
    close("dx", take(dx), want[2], half_step(tout), 32 * U * size[2])
    close("dw", take(dw, 0), want[3], U, (32 + B * N) * U * size[3])
    close("dbias", take(db), want[4], U, (32 + B * N) * U * size[4])
    close("dstate_in", take(d0), want[5], half_step(tout), 32 * U * size[5])
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(y).all()


# strips of 8 (forward) and 16 (gradients) there; 256 channels a wave where rows move as vectors, 64 where they do not
@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 7, 256), (1, 8, 264), (3, 9, 248), (2, 15, 63), (1, 16, 256), (2, 17, 264), (1, 24, 64),
                                   (2, 25, 512), (1, 33, 252), (5, 48, 520)], ids=str)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_convolution_at_the_blocks_edges(R, shape, W, kind):
    conv_tests.test_forward_and_gradients(R, shape, W, kind)


# rounds of 4096, 1024, 256 rows and a rest: 16, 4 and one row at a time in each of 256 workgroups
@pytest.mark.gpu
@pytest.mark.parametrize("rows,D", [(5000, 512), (9001, 300), (2049, 2048), (1030, 4096), (1030, 2049), (600, 8192), (515, 8200),
                                    (300, 16383)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_norm_gradients_over_rounds(R, rows, D, kind):
    import torch
    print_case("rms_norm_rounds", rows, D, kind)
    t = torch.float32 if kind == "f32" else torch.bfloat16
    gen = torch.Generator().manual_seed(D)
    x, w = (rand(gen, rows, D) + 0.5).to(t), 1 + rand(gen, D, scale=0.2)
    dy, dsum = rand(gen, rows, D, dtype=t), rand(gen, rows, D, dtype=t)
    xd, y, rstd = x.cuda(), torch.empty((rows, D), dtype=t, device="cuda"), torch.empty(rows, device="cuda")
    R.ret_rms_norm_fwd(xd, y, w.cuda(), rstd=rstd)
    x64, w64, d64 = x.double().numpy(), w.double().numpy(), dy.double().numpy()
    r64 = 1 / np.sqrt((x64 ** 2).mean(-1) + 1e-5)
    ref = x64 * r64[:, None] * w64
    close("y", y, ref, half_step(t), 64 * U * np.abs(ref).max(1, keepdims=True))
    close("rstd", rstd, r64, 64 * U, 0.0)
    dx, dw = torch.empty_like(y), torch.empty(D, device="cuda")
    R.ret_rms_norm_bwd(dy.cuda(), xd, rstd, dx, weight=w.cuda(), dsum=dsum.cuda(), dweight=dw)
    rg = rstd.double().cpu().numpy()[:, None]
    xh, a = x64 * rg, d64 * w64
    want = rg * (a - xh * (a * xh).mean(-1, keepdims=True)) + dsum.double().numpy()
    scale = rg.max() * np.abs(a).max() * (1 + np.abs(xh).max() ** 2) + np.abs(dsum.double().numpy()).max()
    close("dx", dx, want, half_step(t), 64 * U * scale)
    close("dweight", dw, (d64 * xh).sum(0), U, (rows + 64) * U * (np.abs(d64) * np.abs(xh)).sum(0))


# a wave's block is 16, 16, 8 and 4 tokens at 8, 16, 32 and 64 states, a workgroup's chunk 128, 128, 32 and 16
SCANS = [(1, 16, 32, 8, 1, "f32"), (2, 17, 15, 8, 1, "bf16"), (1, 128, 17, 8, 1, "f32"), (2, 129, 16, 8, 1, "bf16"),
         (1, 257, 64, 8, 2, "f32"), (2, 8, 16, 32, 1, "f32"), (1, 9, 33, 32, 1, "bf16"), (2, 31, 16, 32, 1, "f32"),
         (1, 32, 17, 32, 1, "bf16-f32"), (2, 33, 32, 32, 2, "f32"), (1, 4, 16, 64, 1, "f32"), (2, 5, 17, 64, 1, "bf16"),
         (1, 15, 16, 64, 1, "f32"), (2, 16, 31, 64, 1, "f32"), (1, 16, 17, 64, 1, "bf16")]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SCANS, ids=str)
@pytest.mark.parametrize("ragged", [False, True])
def test_scan_at_the_blocks_edges(R, shape, ragged):
    scan_tests.test_forward(R, shape, ragged)
    scan_tests.test_gradients(R, shape, ragged)
