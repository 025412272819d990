"""The short causal convolution (sequences, single tokens, gradients) against 64 bits.

Tolerances, in units of 2^-24, with p the sum of the magnitudes of pre's W + 1 terms: pre is off by 8 p at most. The hardware
sigmoid s is off by |pre| + 4 of itself: its argument pre log2(e) is rounded, which moves 2^(pre log2(e)) by |pre| units, and
2^x, the sum and the reciprocal add 4. silu = pre s moves by silu' <= s (1 + p) per change of pre, so y is off by at most
8 p s (1 + p) + (p + 4) p s <= 12 p s (1 + p): 16 with its own rounding. Its derivative s (1 + pre (1 - s)) moves by
s (2 + p) per change of pre, and by (p + 4) (1 + 2 p) s from the sigmoid: together at most
8 p (2 + p) s + (p + 4) (1 + 2 p) s <= 16 s (1 + p)^2, and the sum over W and roundings make it 32. Sums over tokens add one
rounding per term at most."""
import numpy as np
import pytest

from tests.conftest import print_case
from tests.scan_ref import U, close, conv, half_step, rand


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


def _types(kind):
    import torch
    return (torch.float32 if kind == "f32" else torch.bfloat16), (torch.bfloat16 if kind == "bf16" else torch.float32)


def test_formulas_by_differentiation():
    """The 64-bit gradients are those that torch finds by differentiating the sum over taps (no GPU)."""
    import torch
    B, N, D, W, lengths = 3, 9, 4, 4, [9, 0, 2]
    gen = torch.Generator().manual_seed(1)
    x, w, b, s, dy, ds = (rand(gen, *n).double().requires_grad_() for n in
                          ((B, N, D), (D, W), (D,), (B, W - 1, D), (B, N, D), (B, W - 1, D)))
    rows = torch.cat([s, x], 1)
    pre = sum(rows[:, j:j + N] * w[:, j] for j in range(W)) + b
    y = torch.nn.functional.silu(pre)
    loss = sum((y[i, :n] * dy[i, :n]).sum() + (rows[i, n:n + W - 1] * ds[i]).sum() for i, n in enumerate(lengths))
    want = torch.autograd.grad(loss, (x, w, b, s))
    args = [t.detach() for t in (x, w, b)]
    got = conv(*args, lengths=lengths, state_in=s.detach(), dy=dy.detach(), dstate_out=ds.detach())[2:]
    for g, t in zip(got, want):
        assert np.abs(g - t.numpy()).max() <= 1e-12
    assert np.abs(conv(*args, state_in=s.detach())[0] - y.detach().numpy()).max() <= 1e-12


# tokens around the strips of 32 and 64, channels around the vectors of 8 and the workgroups of 512 and 64
SHAPES = [(1, 1, 1), (2, 1, 8), (3, 2, 5), (5, 3, 16), (2, 31, 100), (1, 32, 520), (2, 33, 64), (3, 63, 65), (1, 64, 8),
          (2, 65, 1000), (5, 128, 24), (2, 130, 513), (1, 700, 40)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16-f32"])
def test_forward_and_gradients(R, shape, W, kind):
    import torch
    B, N, D = shape
    tin, tout = _types(kind)
    for silu, full, ragged, wide in [(True, True, False, 0), (True, True, True, 1), (False, False, True, 0),
                                     (True, False, False, 8)]:
        print_case("short_conv", shape, W, kind, silu, full, ragged, wide)
        gen = torch.Generator().manual_seed(100 * D + N)
        x, w = rand(gen, B, N, D, dtype=tin), rand(gen, D, W)
        b = rand(gen, D) if full else None
        lengths = None if not ragged else [max(0, n) for n in (N, 0, N - 1, 1, 2)][:B]
        s0 = rand(gen, B, W - 1, D, dtype=tin) if full else None
        ds = rand(gen, B, W - 1, D, dtype=tout) if full else None
        dy = rand(gen, B, N, D, dtype=tin)
        want = conv(x, w, b, silu, lengths, s0, dy, ds)
        size = conv(x, w, b, silu, lengths, s0, dy, ds, absolute=True)
        if lengths is not None:
            for i, n in enumerate(lengths):
                x[i, n:] = dy[i, n:] = float("nan")
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        xd = dev(x)
        if wide:
            rows = torch.full((B, N, D + 2 * wide), float("nan"), dtype=tin, device="cuda")
            rows[..., wide:wide + D] = xd
            xd = rows[..., wide:wide + D]
        ld = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        new = lambda t, *n: torch.full(n, 7.0, dtype=t, device="cuda")  # noqa: E731
        y, last = new(tout, B, N, D), new(tin, B, W - 1, D)
        R.ret_short_conv_fwd(xd, dev(w), y, bias=dev(b), silu=silu, lengths=ld, state_in=dev(s0), state_out=last)
        close("y", y, want[0], half_step(tout), 16 * U * size[0])
        assert torch.equal(last.cpu().double(), torch.from_numpy(want[1]))
        dx, dw, db = new(tout, B, N, D), new(torch.float32, D, W), new(torch.float32, D)
        d0 = new(tout, B, W - 1, D) if full else None
        R.ret_short_conv_bwd(dev(dy), xd, dev(w), dx, dw, bias=dev(b), dbias=db, silu=silu, lengths=ld, state_in=dev(s0),
                             dstate_out=dev(ds), dstate_in=d0)
        close("dx", dx, want[2], half_step(tout), 32 * U * size[2])
        close("dw", dw, want[3], U, (32 + B * N) * U * size[3])
        close("dbias", db, want[4], U, (32 + B * N) * U * size[4])
        if full:
            close("dstate_in", d0, want[5], half_step(tout), 32 * U * size[5])
        dx2 = torch.empty_like(dx)
        R.ret_short_conv_bwd(dev(dy), xd, dev(w), dx2, bias=dev(b), silu=silu, lengths=ld, state_in=dev(s0),
                             dstate_out=dev(ds))
        assert torch.equal(dx, dx2)  # without the sums, and the same bits again


@pytest.mark.gpu
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16-f32"])
def test_step_is_the_sequence_token_by_token(R, W, kind):
    import torch
    tin, tout = _types(kind)
    for B, D, silu, wide in [(1, 1, True, 0), (3, 24, True, 8), (2, 2056, False, 0), (5, 77, True, 3)]:
        N = 6
        print_case("short_conv_step", W, kind, B, D)
        gen = torch.Generator().manual_seed(D)
        x, w, b = rand(gen, B, N, D, dtype=tin), rand(gen, D, W), rand(gen, D)
        state = rand(gen, B, W - 1, D, dtype=tin)
        want, size = (conv(x, w, b, silu, None, state, absolute=a) for a in (False, True))
        rows = torch.zeros((B, N, D + 2 * wide), dtype=tin, device="cuda")
        rows[..., wide:wide + D] = x.cuda()
        y, s = torch.empty((B, N, D), dtype=tout, device="cuda"), state.cuda()
        for t in range(N):
            yt = torch.empty((B, D), dtype=tout, device="cuda")
            R.ret_short_conv_step(rows[:, t, wide:wide + D], w.cuda(), yt, s, bias=b.cuda(), silu=silu)
            y[:, t] = yt
        close("y", y, want[0], half_step(tout), 16 * U * size[0])
        assert torch.equal(s.cpu().double(), torch.from_numpy(want[1]))


@pytest.mark.gpu
def test_state_in_place_streams_and_nan(R):
    import torch
    gen = torch.Generator().manual_seed(3)
    x, w, s = rand(gen, 2, 50, 64, dtype=torch.bfloat16).cuda(), rand(gen, 64, 4).cuda(), \
        rand(gen, 2, 3, 64, dtype=torch.bfloat16).cuda()
    y, out = torch.empty_like(x), torch.empty_like(s)
    for lengths in (None, torch.tensor([1, 0], dtype=torch.int32, device="cuda")):
        R.ret_short_conv_fwd(x, w, y, state_in=s, state_out=out, lengths=lengths)
        s2, y2, stream = s.clone(), torch.empty_like(x), torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        R.ret_short_conv_fwd(x, w, y2, state_in=s2, state_out=s2, lengths=lengths, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(out, s2)
    R.ret_short_conv_fwd(x, w, y)
    bad, y2 = x.clone(), torch.empty_like(x)
    bad[0, 20, 3] = float("nan")
    R.ret_short_conv_fwd(bad, w, y2)
    assert y2[0, 20:24, 3].isnan().all() and int(y2.isnan().sum()) == 4


@pytest.mark.gpu
def test_offsets_past_32_bits(R):
    import torch
    N, D = 70000, 32768
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((1, N, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    w, y = torch.randn((D, 4), generator=gen, device="cuda"), torch.empty_like(x)
    R.ret_short_conv_fwd(x, w, y)
    cut = N - 200
    tail = torch.empty_like(x[:, cut:])
    R.ret_short_conv_fwd(x[:, cut:].contiguous(), w, tail, state_in=x[:, cut - 3:cut].contiguous())
    assert torch.equal(y[:, cut:], tail)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    R.ret_short_conv_bwd(x, x, w, dx, dw)
    dtail = torch.empty_like(tail)
    R.ret_short_conv_bwd(x[:, cut:].contiguous(), x[:, cut:].contiguous(), w, dtail,
                         state_in=x[:, cut - 3:cut].contiguous())
    assert torch.equal(dx[:, cut:], dtail) and torch.isfinite(dw).all()
