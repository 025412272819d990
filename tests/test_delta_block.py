"""The operators of a gated delta block together: layer norm, the delta rule, GroupNorm and gate, and back, against the
same block in 64 bits under autograd; the prefill, then single tokens; and the shapes of the delta rule that
test_gated_delta.py and test_gated_delta_grad.py leave out (each d_k with d_v on both sides of 64, grouped and not).

Tolerances of the block. F32: the stages' own bounds in the 2-norm (norms 1e-6, delta rule 3e-6, its gradients 1e-5) add
up to 2e-5; a norm's Jacobian passes an error on by the ratio of the rows' deviations, below 5 for these inputs: 1e-4.
BF16: the reference rounds where the block stores (the sum, the norm's output, o), so that what differs forward is the output's
rounding; backward dO's rounding (2^-8 / sqrt(3)), the delta gradients' bounds (5.1e-3, dg 1.1e-2) and the result's own
rounding (2^-8 / sqrt(3)) add up to 1e-2 (dg 1.6e-2): twice that.
"""
import numpy as np
import pytest

import tests.test_gated_delta as fwd
import tests.test_gated_delta_grad as bwd
from tests.conftest import print_case
from tests.delta_ref import forward, gradients, inputs, np64, term_sums

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


SHAPES = [("f32", 2, 130, 2, 1, 16, 96), ("f32", 1, 140, 4, 2, 64, 80), ("f32", 1, 131, 1, 1, 128, 64),
          ("f32", 1, 70, 2, 2, 32, 64), ("bf16", 2, 200, 2, 1, 64, 112), ("bf16", 1, 190, 2, 2, 128, 64),
          ("bf16", 1, 200, 2, 1, 256, 64), ("bf16", 1, 70, 1, 1, 256, 16), ("bf16", 1, 129, 3, 1, 32, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("segments", [1, 2])
@pytest.mark.parametrize("variant", [0, 1])
def test_shapes(R, shape, segments, variant):
    import torch
    dtype, B, N, H, Hk, dk, dv = shape
    print_case("gated_delta_shapes", shape, segments, variant)
    x = inputs(N + dk, B, N, H, Hk, dk, dv, dtype, "bf16" if dtype == "bf16" and variant else "f32", strong=variant == 1)
    gen = torch.Generator().manual_seed(1)
    state = 0.5 * torch.randn(B, H, dk, dv, generator=gen)
    dout = torch.randn(B, N, H, dv, generator=gen).to(x["q"].dtype)
    dstate = torch.randn(B, H, dk, dv, generator=gen)
    lengths = [N - 1] + [N // 3] * (B - 1) if variant else None
    ln = None if lengths is None else np.array(lengths)
    a = [np64(x[n]) for n in ("q", "k", "v", "g", "beta")]
    o, s = fwd.run(R, x, H, dv, state, lengths, "same" if variant else "f32", {"segments": segments})
    ro, rs, before = forward(*a, dk ** -0.5, np64(state), ln)
    fwd.check("o", o, ro, dtype, term_sums(*a, dk ** -0.5, before))
    fwd.check("state", s, rs, dtype)
    got = bwd.run(R, x, dout, state, dstate, lengths, None if variant else torch.float32, {"segments": segments})
    bwd.check(got, gradients(*a, dk ** -0.5, np64(dout), np64(state), np64(dstate), ln), dtype)


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 32, 48), ("bf16", 64, 64), ("bf16", 128, 96)])
def test_segments_of_the_default_plan(R, dtype, dk, dv):
    """A sequence long enough that the call splits it by itself; the same bits from a call into a larger workspace."""
    import torch
    B, N, H = 1, 13 * 64 + 5, 2
    print_case("gated_delta_default_plan", dtype, dk, dv)
    x = inputs(5, B, N, H, 1, dk, dv, dtype)
    a = [np64(x[n]) for n in ("q", "k", "v", "g", "beta")]
    o, s = fwd.run(R, x, H, dv)
    ro, rs, before = forward(*a, dk ** -0.5)
    fwd.check("o", o, ro, dtype, term_sums(*a, dk ** -0.5, before))
    fwd.check("state", s, rs, dtype)
    dout = torch.randn(B, N, H, dv, generator=torch.Generator().manual_seed(2)).to(x["q"].dtype)
    got = bwd.run(R, x, dout)
    bwd.check(got, gradients(*a, dk ** -0.5, np64(dout)), dtype)
    d = {n: t.cuda() for n, t in x.items()}
    ws = torch.full((R.gated_delta_bwd_workspace(d["q"], d["v"]).numel() + 4096,), 255, dtype=torch.uint8, device="cuda")
    again = bwd.run(R, x, dout, workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


def block64(t, B, N, H, Hk, dk, dv, stored):
    """The block in 64 bits: -> (s, out); stored(x): x as it is stored, with the gradient passed through."""
    import torch
    s = stored(t["x"] + t["res"])
    mu, var = s.mean(-1, keepdim=True), s.var(-1, unbiased=False, keepdim=True)
    y = stored((s - mu) / torch.sqrt(var + 1e-5) * t["w"] + t["b"])
    q, k, v = y.split([Hk * dk, Hk * dk, H * dv], -1)
    q, k = (z.view(B, N, Hk, dk).repeat_interleave(H // Hk, 2) for z in (q, k))
    v, S, o = v.view(B, N, H, dv), t["state"], []
    for i in range(N):
        S = S * torch.exp(t["g"][:, i])[..., None, None]
        u = t["beta"][:, i][..., None] * (v[:, i] - (k[:, i][..., None] * S).sum(2))
        S = S + k[:, i][..., None] * u[:, :, None]
        o.append(dk ** -0.5 * (q[:, i][..., None] * S).sum(2))
    o = stored(torch.stack(o, 1))
    mu, var = o.mean(-1, keepdim=True), o.var(-1, unbiased=False, keepdim=True)
    z = (o - mu) / torch.sqrt(var + 1e-5) * t["gw"].view(H, dv) + t["gb"].view(H, dv)
    return s, z * torch.nn.functional.silu(t["gate"]), S


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_block(R, dtype):
    import torch
    B, N, extra, H, Hk, dk, dv = 2, 150, 4, 4, 2, 32, 64  # d_v: one that ret_msr_epilogue takes
    print_case("gated_delta_block", dtype)
    tt, D = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype], 2 * Hk * dk + H * dv
    gen = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    M = N + extra
    t = dict(x=rn(B, M, D).to(tt), res=rn(B, M, D).to(tt), gate=rn(B, M, H, dv).to(tt), b=0.02 * rn(D),
             w=torch.cat([torch.full((2 * Hk * dk,), dk ** -0.5), torch.ones(H * dv)]) * (1 + 0.1 * rn(D)),
             gw=1 + 0.2 * rn(H * dv), gb=0.2 * rn(H * dv), g=-torch.exp(0.5 * rn(B, M, H) - 3),
             beta=torch.sigmoid(rn(B, M, H)), state=rn(B, H, dk, dv))
    dout, dsum, dstate = rn(B, N, H, dv).to(tt), rn(B, N, D).to(tt), rn(B, H, dk, dv)
    stored = (lambda z: z) if dtype == "f32" else (lambda z: z + (z.detach().bfloat16().double() - z.detach()))

    # 64 bits: all tokens for the values, the first N for the gradients
    ref = {n: z.double().requires_grad_() for n, z in t.items()}
    cut = {n: z[:, :N].detach().clone().requires_grad_() if n in ("x", "res", "gate", "g", "beta") else z
           for n, z in ref.items()}
    _, rout, rend = block64(ref, B, M, H, Hk, dk, dv, stored)
    s, out, end = block64(cut, B, N, H, Hk, dk, dv, stored)
    ((out * dout.double()).sum() + (s * dsum.double()).sum() + (end * dstate.double()).sum()).backward()

    # the operators
    d = {n: z.cuda() for n, z in t.items()}
    p = {n: d[n][:, :N].contiguous() for n in ("x", "res", "gate", "g", "beta")}
    new = lambda *s, dt=tt: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    f32 = torch.float32

    def parts(y):
        return [z.reshape(*y.shape[:-1], *hd).contiguous()
                for z, hd in zip(y.split([Hk * dk, Hk * dk, H * dv], -1), ((Hk, dk), (Hk, dk), (H, dv)))]

    y, sm, mean, rstd = new(B, N, D), new(B, N, D), new(B, N, dt=f32), new(B, N, dt=f32)
    R.ret_layer_norm_fwd(p["x"], y, weight=d["w"], bias=d["b"], residual=p["res"], sum_out=sm, mean=mean, rstd=rstd)
    q, k, v = parts(y)
    o, S, z = new(B, N, H, dv), new(B, H, dk, dv, dt=f32), new(B, N, H, dv)
    R.ret_gated_delta_fwd(q, k, v, p["g"], p["beta"], o, state_in=d["state"], state_out=S, options={"segments": 2})
    R.ret_msr_epilogue(o, z, gate=p["gate"], gn_weight=d["gw"], gn_bias=d["gb"])
    outs = [z.clone()]
    # single tokens from the state the prefill left
    Sd = S.clone()
    for i in range(N, M):
        c = {n: d[n][:, i].contiguous() for n in p}
        y1, o1 = new(B, D), new(B, H, dv)
        R.ret_layer_norm_fwd(c["x"], y1, weight=d["w"], bias=d["b"], residual=c["res"])
        q1, k1, v1 = parts(y1)
        R.ret_gated_delta_step(q1, k1, v1, c["g"], c["beta"], o1, Sd)
        R.ret_msr_epilogue(o1, o1, gate=c["gate"], gn_weight=d["gw"], gn_bias=d["gb"])
        outs.append(o1[:, None])
    # back
    do, dgate, dgw, dgb = new(B, N, H, dv), new(B, N, H, dv), new(H * dv, dt=f32), new(H * dv, dt=f32)
    R.ret_msr_epilogue_bwd(dout.cuda(), o, do, gate=p["gate"], dgate=dgate, gn_weight=d["gw"], gn_bias=d["gb"],
                           dweight=dgw, dbias=dgb)
    dq, dkk, dvv, dg, dbeta, dS = (torch.empty_like(n) for n in (q, k, v, p["g"], p["beta"], S))
    R.ret_gated_delta_bwd(q, k, v, p["g"], p["beta"], do, dq, dkk, dvv, dg, dbeta, state_in=d["state"],
                          dstate_out=dstate.cuda(), dstate_in=dS, options={"segments": 2})
    dy = torch.cat([n.reshape(B, N, -1) for n in (dq, dkk, dvv)], -1)
    dx, dw, db = new(B, N, D), new(D, dt=f32), new(D, dt=f32)
    R.ret_layer_norm_bwd(dy, sm, mean, rstd, dx, weight=d["w"], dsum=dsum.cuda(), dweight=dw, dbias=db)

    tol = 1e-4 if dtype == "f32" else 2e-2
    for name, got, want, lim in [("out", torch.cat(outs, 1), rout, tol), ("state", Sd, rend, tol), ("dx", dx, cut["x"].grad, tol),
                                 ("dw", dw, ref["w"].grad, tol), ("db", db, ref["b"].grad, tol),
                                 ("dgate", dgate, cut["gate"].grad, tol), ("dgw", dgw, ref["gw"].grad, tol),
                                 ("dgb", dgb, ref["gb"].grad, tol), ("dg", dg, cut["g"].grad, 1.6 * tol),
                                 ("dbeta", dbeta, cut["beta"].grad, tol), ("dS", dS, ref["state"].grad, tol)]:
        want = want.detach()
        assert got.shape == want.shape, name
        off = float((got.double().cpu() - want).norm() / want.norm())
        print("   %-6s %.2e" % (name, off))
        assert off <= lim, (name, off)


def test_two_graphs_share_a_workspace(R):
    """A captured forward of one shape and captured gradients of another in one workspace, replayed in turn with eager
    calls in the same workspace between: every replay has the eager call's bits. The gradients on another stream, their
    workspace made by the call, too."""
    import torch
    def operands(seed, B, N, H, Hk, dk, dv):
        return {n: t.cuda() for n, t in inputs(seed, B, N, H, Hk, dk, dv, "bf16").items()}
    a, b = operands(1, 1, 400, 2, 2, 64, 96), operands(2, 2, 150, 4, 2, 128, 64)
    names = ("q", "k", "v", "g", "beta")
    opt = {"segments": 3}
    ws = torch.empty(max(R.gated_delta_workspace(a["q"], a["v"], opt).numel(),
                         R.gated_delta_bwd_workspace(b["q"], b["v"]).numel()), dtype=torch.uint8, device="cuda")
    o, dout = torch.empty_like(a["v"]), torch.randn(b["v"].shape, device="cuda").bfloat16()
    grads = [torch.empty_like(b[n]) for n in names]

    def first():
        R.ret_gated_delta_fwd(*[a[n] for n in names], o, workspace=ws, options=opt)

    def second():
        R.ret_gated_delta_bwd(*[b[n] for n in names], dout, *grads, workspace=ws)

    first()
    second()
    torch.cuda.synchronize()
    want_o, want_g = o.clone(), [t.clone() for t in grads]
    graphs, s = [], torch.cuda.Stream()
    for fn in (first, second):
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            fn()
        graphs.append(g)
    torch.cuda.synchronize()
    for i in range(3):
        for t in [o] + grads:
            t.fill_(3.0)
        for g in graphs if i % 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want_o) and all(torch.equal(p, q) for p, q in zip(grads, want_g)), i
        first()
        second()
        torch.cuda.synchronize()
    other = [torch.empty_like(t) for t in grads]
    s.wait_stream(torch.cuda.current_stream())
    R.ret_gated_delta_bwd(*[b[n] for n in names], dout, *other, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(other, want_g))


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 16, 32), ("bf16", 32, 80), ("bf16", 256, 128)])
def test_more_segments_than_chunks_and_one_tensor_for_q_and_k(R, dtype, dk, dv):
    """Every chunk a segment (the option asks for more than there are), some of them past a sequence's end; q is k."""
    import torch
    B, N, H = 2, 330, 2
    print_case("gated_delta_single_chunk_segments", dtype, dk, dv)
    x = inputs(9, B, N, H, H, dk, dv, dtype)
    x["q"] = x["k"]
    lengths = [70, 330]
    gen = torch.Generator().manual_seed(4)
    state, dstate = torch.randn(B, H, dk, dv, generator=gen), torch.randn(B, H, dk, dv, generator=gen)
    dout = torch.randn(B, N, H, dv, generator=gen).to(x["q"].dtype)
    a = [np64(x[n]) for n in ("q", "k", "v", "g", "beta")]
    o, s = fwd.run(R, x, H, dv, state, lengths, "same", {"segments": 50})
    ro, rs, before = forward(*a, dk ** -0.5, np64(state), np.array(lengths))
    fwd.check("o", o, ro, dtype, term_sums(*a, dk ** -0.5, before))
    fwd.check("state", s, rs, dtype)
    got = bwd.run(R, x, dout, state, dstate, lengths, None, {"segments": 50})
    bwd.check(got, gradients(*a, dk ** -0.5, np64(dout), np64(state), np64(dstate), np.array(lengths)), dtype)
