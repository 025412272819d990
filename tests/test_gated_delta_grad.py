"""Gradients of the gated delta rule against the token-by-token recurrence's in 64 bits, against differences of the
forward call, and in a run of the whole block.

Tolerances. F32: fp32 sums of a few hundred terms in two chains and three products: below 1e-5 in the 2-norm. BF16: dv and
dstate_in come from split products, 1e-5 (dv adds its rounding); dq, dk, dg and dbeta multiply two to four values stored
in bf16, each off by 2^-9 of itself at most and 2^-9/sqrt(3) on the average over a binade, 2^-9 at worst: up to four of
them, independent, and the output's own rounding make at most sqrt(5) 2^-8 / sqrt(3) = 5.1e-3 in the 2-norm. dg is a sum
over a chunk of differences of such terms, which do not cancel on the average: twice that.
"""
import numpy as np
import pytest

from tests.conftest import print_case
from tests.delta_ref import gradients, inputs, np64

pytestmark = pytest.mark.gpu
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dstate_in")


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


def bound(name, dtype, got):
    if dtype == "f32" or name == "dstate_in":
        return 1e-5
    if name == "dv":
        return 1e-5 if str(got.dtype) == "torch.float32" else 2.0 ** -8 / np.sqrt(3)
    return 1.1e-2 if name == "dg" else 5.1e-3


def run(R, x, dout, state=None, dstate=None, lengths=None, out=None, options=None, workspace=None):
    import torch
    d = {n: t.cuda() for n, t in x.items()}
    B, N, H, dv = x["v"].shape
    out = out or x["q"].dtype
    gr = [torch.full(x[n].shape, 7.0, dtype=t, device="cuda")
          for n, t in (("q", out), ("k", out), ("v", out), ("g", x["g"].dtype), ("beta", x["g"].dtype))]
    ds = torch.full((B, H, x["q"].shape[3], dv), 7.0, device="cuda")
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    R.ret_gated_delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], dout.cuda(), *gr, state_in=dev(state),
                          lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                          dstate_out=dev(dstate), dstate_in=ds, options=options, workspace=workspace)
    return gr + [ds]


def check(got, ref, dtype):
    for name, a, b in zip(NAMES, got, ref):
        g = a.double().cpu().numpy()
        assert g.shape == b.shape and np.isfinite(g).all(), name
        norm, off = np.sqrt((b ** 2).sum()), np.sqrt(((g - b) ** 2).sum())
        print("   %-9s %.2e" % (name, off / norm if norm else off))
        assert off <= bound(name, dtype, a) * norm, (name, off / norm if norm else off)


SHAPES = [("f32", 1, 1, 1, 1, 16, 16), ("f32", 2, 64, 2, 1, 16, 48), ("f32", 1, 65, 4, 2, 32, 80),
          ("f32", 2, 200, 3, 3, 64, 64), ("f32", 1, 150, 2, 1, 128, 144), ("bf16", 1, 1, 2, 1, 32, 16),
          ("bf16", 2, 63, 2, 2, 64, 64), ("bf16", 1, 64, 4, 1, 128, 128), ("bf16", 3, 129, 2, 1, 32, 208),
          ("bf16", 1, 300, 3, 3, 64, 48), ("bf16", 2, 260, 4, 2, 128, 160), ("bf16", 1, 257, 2, 1, 256, 96),
          ("bf16", 1, 330, 1, 1, 256, 272)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("segments", [1, 3])
def test_gradients(R, shape, segments):
    import torch
    dtype, B, N, H, Hk, dk, dv = shape
    for variant in range(2):
        print_case("gated_delta_bwd", shape, segments, variant)
        gates = "bf16" if dtype == "bf16" and variant else "f32"
        x = inputs(N + dk + 1, B, N, H, Hk, dk, dv, dtype, gates, strong=variant == 1)
        gen = torch.Generator().manual_seed(1)
        dout = torch.randn(B, N, H, dv, generator=gen).to(x["q"].dtype)
        state = 0.5 * torch.randn(B, H, dk, dv, generator=gen) if variant else None
        dstate = torch.randn(B, H, dk, dv, generator=gen) if variant else None
        lengths = [N - 1] + [N // 3] * (B - 1) if variant and N > 1 else None
        out = torch.float32 if variant == 0 else None
        got = run(R, x, dout, state, dstate, lengths, out, {"segments": segments})
        ref = gradients(*[np64(x[n]) for n in ("q", "k", "v", "g", "beta")], dk ** -0.5, np64(dout), np64(state),
                        np64(dstate), None if lengths is None else np.array(lengths))
        check(got, ref, dtype)
        if lengths is not None:
            for b, n in enumerate(lengths):
                assert not any(t[b, n:].any() for t in got[:5])


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 32, 16), ("bf16", 64, 32)])
def test_extremes(R, dtype, dk, dv):
    """Decays that clear the state, writes of strength zero, and padding of NaN: finite gradients, zero on the padding,
    and those of the recurrence."""
    import torch
    B, N, H = 2, 150, 2
    print_case("gated_delta_bwd_extremes", dtype, dk, dv)
    x = inputs(3, B, N, H, H, dk, dv, dtype)
    x["g"][:, 40] = -float("inf")
    x["g"][:, 100:110] = -150.0
    x["beta"][:, 20:30] = 0.0
    x["beta"][:, 60:70] = 1.0
    dout = torch.randn(B, N, H, dv, generator=torch.Generator().manual_seed(4)).to(x["q"].dtype)
    lengths = [0, 145]
    ref = {n: np64(t).copy() for n, t in x.items()}
    rd = np64(dout).copy()
    ref["g"] = np.maximum(ref["g"], -1e4)
    for t, r in [(x[n], ref[n]) for n in x] + [(dout, rd)]:
        t[0] = float("nan")
        t[1, 145:] = float("nan")
        r[0] = 0.0
        r[1, 145:] = 0.0
    dstate = torch.randn(B, H, dk, dv, generator=torch.Generator().manual_seed(2))
    want = gradients(ref["q"], ref["k"], ref["v"], ref["g"], ref["beta"], dk ** -0.5, rd, None, np64(dstate),
                     np.array(lengths))
    for segments in (1, 2):
        got = run(R, x, dout, None, dstate, lengths, options={"segments": segments})
        check(got, want, dtype)
        assert torch.equal(got[5][0].cpu(), dstate[0])
        assert not any(t[0].any() or t[1, 145:].any() for t in got[:5])


def test_against_differences(R):
    """Central differences of L = sum(dout o) + sum(dstate state) over the forward call in fp32: h^2 of the third
    derivative (bounded by 10 here) and the loss's own rounding, 3e-6 |L| / h."""
    import torch
    B, N, H, Hk, dk, dv, h = 1, 70, 2, 1, 16, 16, 2.0 ** -5
    x = inputs(7, B, N, H, Hk, dk, dv, "f32")
    gen = torch.Generator().manual_seed(8)
    dout, dstate = torch.randn(B, N, H, dv, generator=gen) / 8, torch.randn(B, H, dk, dv, generator=gen) / 8
    state = torch.randn(B, H, dk, dv, generator=gen)

    def loss(y, s):
        d = {n: t.cuda() for n, t in y.items()}
        o, so = torch.empty(B, N, H, dv, device="cuda"), torch.empty(B, H, dk, dv, device="cuda")
        R.ret_gated_delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], o, state_in=s.cuda(), state_out=so)
        return float((o.cpu().double() * dout.double()).sum() + (so.cpu().double() * dstate.double()).sum())

    got = dict(zip(NAMES, run(R, x, dout, state, dstate)))
    L = abs(loss(x, state)) + 10
    for name, at in [("q", (0, 3, 0, 5)), ("k", (0, 0, 0, 1)), ("k", (0, 66, 0, 9)), ("v", (0, 20, 1, 4)),
                     ("g", (0, 33, 0)), ("g", (0, 69, 1)), ("g", (0, 2, 1)), ("beta", (0, 10, 0)), ("beta", (0, 64, 1))]:
        lo, hi = ({n: t.clone() for n, t in x.items()} for _ in range(2))
        hi[name][at] += h
        lo[name][at] -= h
        num = (loss(hi, state) - loss(lo, state)) / (2 * h)
        assert abs(num - float(got["d" + name][at])) <= 10 * h * h + 3e-6 * L / h, (name, at)
    e = torch.zeros_like(state)
    e[0, 1, 3, 7] = h
    num = (loss(x, state + e) - loss(x, state - e)) / (2 * h)
    assert abs(num - float(got["dstate_in"][0, 1, 3, 7])) <= 10 * h * h + 3e-6 * L / h


def test_graph_replays_and_same_bits(R):
    """The gradients captured and replayed with new inputs, eager work of the same leaves between; every replay has the
    eager call's bits, and two eager calls the same ones."""
    import torch
    B, N, H, Hk, dk, dv = 2, 200, 4, 2, 64, 64
    x = inputs(1, B, N, H, Hk, dk, dv, "bf16", "bf16")
    d = {n: t.cuda() for n, t in x.items()}
    dout = torch.randn(B, N, H, dv, device="cuda").bfloat16()
    gr = [torch.empty_like(d[n]) for n in ("q", "k", "v", "g", "beta")]
    ws = R.gated_delta_bwd_workspace(d["q"], d["v"], {"segments": 2})

    def step():
        R.ret_gated_delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], dout, *gr, workspace=ws, options={"segments": 2})

    step()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        step()
    torch.cuda.synchronize()
    for i in range(3):
        y = inputs(30 + i, B, N, H, Hk, dk, dv, "bf16", "bf16")
        for n in d:
            d[n].copy_(y[n])
        dout.normal_()
        graph.replay()
        torch.cuda.synchronize()
        a = [t.clone() for t in gr]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, gr)), i
        ref = gradients(*[np64(y[n]) for n in ("q", "k", "v", "g", "beta")], dk ** -0.5, np64(dout.cpu()))
        check(a, ref[:5], "bf16")
