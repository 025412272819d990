"""Gradients of the gated delta rule in fp32 from bf16 input: as precise as their type asks, not as the input's.

Tolerances in the 2-norm. What the two chains hand over is within 1e-5 of itself (test_gated_delta_grad.py) and is stored
in two bf16 parts, off by 2^-17 at most and 2^-17 / sqrt(3) = 4.4e-6 on the average, like X and Z; a product of two such
operands leaves out that of the low parts, (2^-8 / sqrt(3))^2 = 5.1e-6 of it on the average. A term has two stored
operands, one of X and Z and up to two such products: sqrt(2 (1e-5)^2 + 3 (4.4e-6)^2 + 2 (5.1e-6)^2) = 1.8e-5, taken as 2e-5.
dg is a difference of sums of such terms: four times that. A bf16 output adds its rounding, 2^-8 / sqrt(3).

A token's own term beta_i scale (q_i.k_i) (dO_i.e_i) cancels in dg; the kernel leaves it out there, so that dg of a single
token without states is 0, as it should be."""
import numpy as np
import pytest

import tests.test_gated_delta_grad as bwd
from tests.conftest import print_case
from tests.delta_ref import gradients, inputs, np64

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dstate_in")


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


def check(got, ref):
    for name, a, b in zip(NAMES, got, ref):
        g = a.double().cpu().numpy()
        assert g.shape == b.shape and np.isfinite(g).all(), name
        lim = 8e-5 if name == "dg" else 1e-5 if name == "dstate_in" else 2e-5
        if str(a.dtype) == "torch.bfloat16":
            lim += 2.0 ** -8 / np.sqrt(3)
        norm, off = np.sqrt((b ** 2).sum()), np.sqrt(((g - b) ** 2).sum())
        print("   %-9s %.2e" % (name, off / norm if norm else off))
        assert off <= lim * norm, (name, off / norm if norm else off)


SHAPES = [(1, 1, 2, 1, 32, 16), (2, 63, 2, 2, 64, 64), (1, 64, 4, 1, 128, 128), (3, 129, 2, 1, 32, 208),
          (1, 300, 3, 3, 64, 48), (2, 260, 4, 2, 128, 160), (1, 257, 2, 1, 256, 96), (1, 330, 1, 1, 256, 272),
          (1, 140, 6, 2, 64, 96), (2, 70, 3, 3, 32, 32), (1, 200, 2, 2, 128, 64), (1, 70, 2, 2, 256, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("gates,out", [("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_gradients(R, shape, gates, out):
    import torch
    B, N, H, Hk, dk, dv = shape
    for variant in range(2):
        print_case("gated_delta_precision", shape, gates, out, variant)
        x = inputs(N + dk, B, N, H, Hk, dk, dv, "bf16", gates, strong=variant == 1)
        gen = torch.Generator().manual_seed(1)
        dout = torch.randn(B, N, H, dv, generator=gen).bfloat16()
        state = 0.5 * torch.randn(B, H, dk, dv, generator=gen) if variant else None
        dstate = torch.randn(B, H, dk, dv, generator=gen) if variant else None
        lengths = [N - 1] + [N // 3] * (B - 1) if variant and N > 1 else None
        got = bwd.run(R, x, dout, state, dstate, lengths, torch.float32 if out == "f32" else torch.bfloat16,
                      {"segments": 1 + 2 * variant})
        ref = gradients(*[np64(x[n]) for n in ("q", "k", "v", "g", "beta")], dk ** -0.5, np64(dout), np64(state),
                        np64(dstate), None if lengths is None else np.array(lengths))
        check(got, ref)
        if lengths is not None:
            for b, n in enumerate(lengths):
                assert not any(t[b, n:].any() for t in got[:5])


@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv", [(64, 32), (256, 48)])
def test_extremes(R, dk, dv):
    """Decays that clear the state, writes of strength zero, padding of NaN, one sequence without tokens."""
    import torch
    B, N, H = 2, 150, 2
    print_case("gated_delta_precision_extremes", dk, dv)
    x = inputs(3, B, N, H, H, dk, dv, "bf16")
    x["g"][:, 40] = -float("inf")
    x["g"][:, 100:110] = -150.0
    x["beta"][:, 20:30] = 0.0
    dout = torch.randn(B, N, H, dv, generator=torch.Generator().manual_seed(4)).bfloat16()
    ref, rd = {n: np64(t).copy() for n, t in x.items()}, np64(dout).copy()
    ref["g"] = np.maximum(ref["g"], -1e4)
    for t, r in [(x[n], ref[n]) for n in x] + [(dout, rd)]:
        t[0] = float("nan")
        t[1, 145:] = float("nan")
        r[0] = 0.0
        r[1, 145:] = 0.0
    dstate = torch.randn(B, H, dk, dv, generator=torch.Generator().manual_seed(2))
    lengths = [0, 145]
    want = gradients(ref["q"], ref["k"], ref["v"], ref["g"], ref["beta"], dk ** -0.5, rd, None, np64(dstate),
                     np.array(lengths))
    for segments in (1, 2):
        got = bwd.run(R, x, dout, None, dstate, lengths, torch.float32, {"segments": segments})
        check(got, want)
        assert torch.equal(got[5][0].cpu(), dstate[0])
        assert not any(t[0].any() or t[1, 145:].any() for t in got[:5])


@pytest.mark.gpu
def test_same_bits_in_a_graph_and_a_dirty_workspace(R):
    import torch
    B, N, H, Hk, dk, dv = 2, 200, 4, 2, 64, 80
    x = inputs(1, B, N, H, Hk, dk, dv, "bf16", "f32")
    d = {n: t.cuda() for n, t in x.items()}
    dout = torch.randn(B, N, H, dv, device="cuda").bfloat16()
    ws = R.gated_delta_bwd_workspace(d["q"], d["v"], {"segments": 2}).fill_(255)
    gr = [torch.empty_like(d[n]) for n in ("q", "k", "v", "g", "beta")]

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
        y = inputs(30 + i, B, N, H, Hk, dk, dv, "bf16", "f32")
        for n in d:
            d[n].copy_(y[n])
        graph.replay()
        torch.cuda.synchronize()
        a = [t.clone() for t in gr]
        ws.fill_(255)
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, gr)), i
        check(a, gradients(*[np64(y[n]) for n in ("q", "k", "v", "g", "beta")], dk ** -0.5, np64(dout.cpu()))[:5])


def test_the_workspace_holds_both_forms():
    from linear_recurrent_sequence_amd import retention
    from tests.test_gated_delta_checks import _bwd
    lib = retention.load()
    need = lib.ret_gated_delta_bwd_workspace_bytes(1, 64, 2, 2, 64, 64, 1, None)
    state, rows = 2 * 64 * 64 * 2, 2 * 64 * 64 * 2  # one part of each of two states, and of E and dU
    assert _bwd(lib, gd=1, wsb=need - 2 * (state + rows) - 1) == -3
    assert _bwd(lib, gd=0, wsb=need - 1) == -3 and _bwd(lib, gd=1, outd=0, wsb=need - 1) == -3
