"""The gated delta rule: whole sequences and single tokens against the token-by-token recurrence in 64 bits.

Tolerances. On BF16 input everything computed is split in two bf16 parts: each value carries an error of at most 2^-18 of
itself, 2^-18/sqrt(3) on the average, and the product of the two low parts that is left out another 2^-18 at most. About
six such errors stand between the inputs and an output (S, R, U, T or P, twice over), which are independent: below 1e-5
in the 2-norm. On F32 input the sums of d_k + 64 products in fp32 leave less than 3e-6. Single values are held to 20 times the 2-norm's bound relative to the tensor's rms.
A bf16 output adds its own rounding, 2^-8 of the value; a whole sequence's is also allowed 2^-16 of the sum of its terms'
magnitudes (2^-17 for each of a term's two split operands), which can be far above the value. A single token's output is
fp32 arithmetic and its rounding.
"""
import numpy as np
import pytest

from tests.conftest import print_case
from tests.delta_ref import forward, inputs, np64, term_sums

pytestmark = pytest.mark.gpu
NORM = {"f32": 3e-6, "bf16": 1e-5}


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


def check(name, got, ref, dtype, terms=0.0):
    """terms: the sums of magnitudes of a whole sequence's outputs (used where they are bf16)."""
    half = 2.0 ** -8 if str(got.dtype) == "torch.bfloat16" else 2.0 ** -24
    if half < 1e-6:
        terms = 0.0
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    rms = np.sqrt((ref ** 2).mean()) if ref.size else 0.0
    d = np.abs(got - ref)
    assert (d <= half * np.abs(ref) + 2.0 ** -16 * terms + 20 * NORM[dtype] * rms).all(), (name, float(d.max()), float(rms))
    if half < 1e-6 and rms > 0:
        assert np.sqrt((d ** 2).mean()) <= NORM[dtype] * rms, (name, float(np.sqrt((d ** 2).mean()) / rms))


def run(R, x, H, dv, state=None, lengths=None, out="same", options=None, workspace=None, scale=None):
    import torch
    B, N = x["v"].shape[:2]
    d = {n: t.cuda() for n, t in x.items()}
    o = torch.full((B, N, H, dv), 7.0, dtype=x["v"].dtype if out == "same" else torch.float32, device="cuda")
    s = torch.full((B, H, x["q"].shape[3], dv), 7.0, device="cuda")
    R.ret_gated_delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], o, scale=scale,
                          lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                          state_in=None if state is None else state.cuda(), state_out=s, options=options,
                          workspace=workspace)
    return o, s


# (dtype, B, N, H, Hk, dk, dv)
SHAPES = [("f32", 1, 1, 1, 1, 16, 16), ("f32", 2, 64, 2, 1, 16, 48), ("f32", 1, 65, 4, 2, 32, 80),
          ("f32", 2, 333, 3, 3, 64, 64), ("f32", 1, 200, 2, 2, 128, 144), ("bf16", 1, 1, 2, 1, 32, 16),
          ("bf16", 2, 63, 2, 2, 64, 64), ("bf16", 1, 64, 4, 1, 128, 128), ("bf16", 3, 129, 2, 1, 32, 208),
          ("bf16", 1, 500, 3, 3, 64, 48), ("bf16", 2, 300, 2, 2, 128, 160), ("bf16", 1, 257, 2, 1, 256, 96),
          ("bf16", 1, 700, 1, 1, 256, 512)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("segments", [1, 3])
def test_forward(R, shape, segments):
    import torch
    dtype, B, N, H, Hk, dk, dv = shape
    for variant in range(2):
        print_case("gated_delta_fwd", shape, segments, variant)
        gates = "bf16" if dtype == "bf16" and variant else "f32"
        x = inputs(N + dk, B, N, H, Hk, dk, dv, dtype, gates, strong=variant == 1)
        state = 0.5 * torch.randn(B, H, dk, dv, generator=torch.Generator().manual_seed(1)) if variant else None
        lengths = [N - 1] + [N // 3] * (B - 1) if variant else None
        out = "f32" if dtype == "bf16" and variant == 0 else "same"
        o, s = run(R, x, H, dv, state, lengths, out, {"segments": segments})
        a = [np64(x[n]) for n in ("q", "k", "v", "g", "beta")]
        ro, rs, before = forward(*a, dk ** -0.5, np64(state), None if lengths is None else np.array(lengths))
        check("o", o, ro, dtype, term_sums(*a, dk ** -0.5, before))
        check("state", s, rs, dtype)
        if lengths is not None:
            for b, n in enumerate(lengths):
                assert not o[b, n:].any()


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 32, 16), ("bf16", 64, 32), ("bf16", 128, 144)])
def test_extremes(R, dtype, dk, dv):
    """Decays that clear the state (g = -inf and far below the range of exp), writes of strength 0 and 1, the same key at
    every token, and padding that holds NaN and infinities."""
    import torch
    B, N, H = 2, 210, 2
    print_case("gated_delta_extremes", dtype, dk, dv)
    x = inputs(3, B, N, H, H, dk, dv, dtype)
    x["g"][:, 40] = -float("inf")
    x["g"][:, 41] = -1e30
    x["g"][:, 100:140] = -150.0
    x["g"][:, 150:170] = 0.0
    x["beta"][:, 20:30] = 0.0
    x["beta"][:, 60:90] = 1.0
    x["k"][:, 60:130] = x["k"][:, 60:61]
    lengths = [0, 205]
    ref = {n: np64(t) for n, t in x.items()}
    ref["g"] = np.maximum(ref["g"], -1e4)
    for n in ("q", "k", "v", "g", "beta"):
        x[n][0, :] = float("nan")
        x[n][1, 205:] = float("inf")
        ref[n][0] = 0.0
        ref[n][1, 205:] = 0.0
    state = torch.randn(B, H, dk, dv, generator=torch.Generator().manual_seed(2))
    for segments in (1, 2, 4):
        o, s = run(R, x, H, dv, state, lengths, options={"segments": segments})
        a = [ref[n] for n in ("q", "k", "v", "g", "beta")]
        ro, rs, before = forward(*a, dk ** -0.5, np64(state), np.array(lengths))
        check("o", o, ro, dtype, term_sums(*a, dk ** -0.5, before))
        check("state", s, rs, dtype)
        assert torch.equal(s[0].cpu(), state[0])


def test_lengths_out_of_range_and_scale(R):
    import torch
    x = inputs(4, 3, 70, 2, 2, 64, 32, "bf16")
    o, s = run(R, x, 2, 32, lengths=[-5, 1000, 70], scale=0.7)
    a = [np64(x[n]) for n in ("q", "k", "v", "g", "beta")]
    ro, rs, before = forward(*a, 0.7, None, np.array([0, 70, 70]))
    check("o", o, ro, "bf16", term_sums(*a, 0.7, before))
    check("state", s, rs, "bf16")
    assert not s[0].any() and not torch.isnan(o).any()


def test_resumed_sequence_then_steps(R):
    """Two calls (the state in place), then single tokens, against one run over all tokens."""
    import torch
    B, N, H, Hk, dk, dv, extra = 2, 300, 4, 2, 64, 80, 5
    for dtype in ("bf16", "f32"):
        x = inputs(8, B, N + extra, H, Hk, dk, dv, dtype)
        d = {n: t.cuda() for n, t in x.items()}
        cut = lambda a, b: {n: t[:, a:b].contiguous() for n, t in d.items()}  # noqa: E731
        state, outs = torch.zeros(B, H, dk, dv, device="cuda"), []
        for a, b in ((0, 130), (130, N)):
            p = cut(a, b)
            o = torch.empty_like(p["v"])
            R.ret_gated_delta_fwd(p["q"], p["k"], p["v"], p["g"], p["beta"], o, state_in=state, state_out=state,
                                  options={"segments": 2})
            outs.append(o)
        for t in range(N, N + extra):
            p = {n: y[:, t].contiguous() for n, y in d.items()}
            o = torch.empty_like(p["v"])
            R.ret_gated_delta_step(p["q"], p["k"], p["v"], p["g"], p["beta"], o, state)
            outs.append(o[:, None])
        a = [np64(x[n]) for n in ("q", "k", "v", "g", "beta")]
        ro, rs, before = forward(*a, dk ** -0.5)
        # the second call's chunks begin at token 130
        first = term_sums(*[y[:, :130] for y in a], dk ** -0.5, before)
        second = term_sums(*[y[:, 130:N] for y in a], dk ** -0.5, before[130:])
        check("o", torch.cat(outs, 1), ro, dtype, np.concatenate([first, second, np.zeros_like(ro[:, N:])], 1))
        check("state", state, rs, dtype)


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 48), (64, 64), (128, 208), (256, 80), (256, 512)])
def test_step(R, dtype, out, dk, dv):
    import torch
    tt = {"f32": torch.float32, "bf16": torch.bfloat16}
    for B, H, Hk in [(1, 1, 1), (3, 6, 2), (40, 2, 2)]:
        print_case("gated_delta_step", dtype, out, dk, dv, B, H, Hk)
        gates = "bf16" if out == "bf16" else "f32"
        x = inputs(dk + B, B, 1, H, Hk, dk, dv, dtype, gates)
        state = torch.randn(B, H, dk, dv, generator=torch.Generator().manual_seed(3))
        d = {n: t[:, 0].contiguous().cuda() for n, t in x.items()}
        s, o = state.cuda(), torch.empty(B, H, dv, dtype=tt[out], device="cuda")
        R.ret_gated_delta_step(d["q"], d["k"], d["v"], d["g"], d["beta"], o, s)
        ro, rs, _ = forward(*[np64(x[n]) for n in ("q", "k", "v", "g", "beta")], dk ** -0.5, np64(state))
        check("o", o, ro[:, 0], "f32")   # fp32 arithmetic whatever the inputs
        check("state", s, rs, "f32")


def test_streams_shared_workspace_and_graph(R):
    """A captured forward and step replayed with new inputs, other shapes in the same workspace between the replays, each
    replay against the recurrence; a call on another stream."""
    import torch
    B, N, H, dk, dv = 1, 260, 2, 64, 64
    x = inputs(11, B, N, H, H, dk, dv, "bf16")
    d = {n: t.cuda() for n, t in x.items()}
    big = inputs(12, 2, 400, H, H, dk, dv, "bf16")
    bd = {n: t.cuda() for n, t in big.items()}
    ws = R.gated_delta_workspace(bd["q"], bd["v"], {"segments": 3})
    o, s = torch.empty_like(d["v"]), torch.empty(B, H, dk, dv, device="cuda")
    so, first = torch.empty_like(d["v"][:, 0]), {n: t[:, 0].clone() for n, t in d.items()}

    def step():
        R.ret_gated_delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], o, state_out=s, workspace=ws,
                              options={"segments": 2})
        R.ret_gated_delta_step(first["q"], first["k"], first["v"], first["g"], first["beta"], so, s)

    step()
    torch.cuda.synchronize()
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st), torch.cuda.graph(graph, stream=st):
        step()
    torch.cuda.synchronize()
    bo = torch.empty_like(bd["v"])
    for i in range(3):
        x = inputs(20 + i, B, N, H, H, dk, dv, "bf16")
        for n in d:
            d[n].copy_(x[n])
            first[n].copy_(x[n][:, 0])
        graph.replay()
        R.ret_gated_delta_fwd(bd["q"], bd["k"], bd["v"], bd["g"], bd["beta"], bo, workspace=ws, options={"segments": 3})
        torch.cuda.synchronize()
        a = [np64(x[n]) for n in ("q", "k", "v", "g", "beta")]
        ro, rs, before = forward(*a, dk ** -0.5)
        check("o", o, ro, "bf16", term_sums(*a, dk ** -0.5, before))
        ro, rs, _ = forward(*[y[:, :1] for y in a], dk ** -0.5, rs)
        check("step", so, ro[:, 0], "bf16")
        check("state", s, rs, "bf16")
    other = torch.empty_like(bd["v"])
    st.wait_stream(torch.cuda.current_stream())
    R.ret_gated_delta_fwd(bd["q"], bd["k"], bd["v"], bd["g"], bd["beta"], other, stream=st, options={"segments": 3})
    torch.cuda.synchronize()
    assert torch.equal(other, bo)
