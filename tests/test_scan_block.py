"""A pre-norm selective-scan block from the library's operators: RMS norm with the residual's addition, the projections (torch),
the short convolution, the scan, gated. Sequences, single tokens, gradients, 8 bits, captured graphs; and the plans of larger
calls, held against each other."""
import pytest

from tests.conftest import print_case
from tests.scan_ref import U, rand, units

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


class Block:
    """Weights of a block of width M, inner width D, S states, W taps, step lengths of rank K."""

    def __init__(self, M, D, S, W, K, dtype, seed):
        import torch
        gen = torch.Generator().manual_seed(seed)
        self.sizes, self.dtype = (M, D, S, W, K), dtype
        self.norm = 1 + rand(gen, M, scale=0.1)
        self.w_in = rand(gen, M, 2 * D, scale=M ** -0.5)
        self.conv, self.conv_b = rand(gen, D, W, scale=W ** -0.5), rand(gen, D, scale=0.1)
        self.w_x = rand(gen, D, K + 2 * S, scale=D ** -0.5)
        self.w_dt, self.dt_bias = rand(gen, K, D, scale=K ** -0.5), torch.empty(D).uniform_(-5.0, -2.0, generator=gen)
        self.A, self.skip = -torch.arange(1, S + 1).float() * torch.exp(rand(gen, D, S, scale=0.1)), 1 + rand(gen, D, scale=0.1)
        self.w_out = rand(gen, D, M, scale=D ** -0.5)
        self.names = ("norm", "w_in", "conv", "conv_b", "w_x", "w_dt", "dt_bias", "A", "skip", "w_out")

    def to(self, device):
        for n in self.names:
            t = getattr(self, n).to(device)
            setattr(self, n, t.to(self.dtype) if n.startswith("w_") else t)
        return self


def forward(R, m, x, res, conv_in=None, scan_in=None, options=None):
    """The block over [B, N, M] on the GPU: (out, the residual stream, what the gradients need, the states after it)."""
    import torch
    M, D, S, W, K = m.sizes
    B, N, _ = x.shape
    e = lambda *s, t=m.dtype: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    k = dict(normed=e(B, N, M), stream=e(B, N, M), rstd=e(B, N, t=torch.float32), u=e(B, N, D), y=e(B, N, D),
             conv_out=e(B, W - 1, D), scan_out=e(B, D, S, t=torch.float32), conv_in=conv_in, scan_in=scan_in)
    R.ret_rms_norm_fwd(x, k["normed"], m.norm, residual=res, sum_out=k["stream"], rstd=k["rstd"])
    k["xz"] = k["normed"] @ m.w_in
    k["x"], k["z"] = k["xz"][..., :D], k["xz"][..., D:]
    R.ret_short_conv_fwd(k["x"], m.conv, k["u"], bias=m.conv_b, state_in=conv_in, state_out=k["conv_out"])
    k["proj"] = k["u"] @ m.w_x
    k["b"], k["c"] = (k["proj"][..., K + i * S:K + (i + 1) * S].unflatten(-1, (1, S)) for i in (0, 1))
    k["dt"] = k["proj"][..., :K] @ m.w_dt
    R.ret_selective_scan_fwd(k["u"], k["dt"], m.A, k["b"], k["c"], k["y"], d_skip=m.skip, z=k["z"], dt_bias=m.dt_bias,
                             state_in=scan_in, state_out=k["scan_out"], options=options)
    return k["y"] @ m.w_out, k["stream"], k


def step(R, m, x, res, conv, scan):
    """One token of the block: [B, M]; the states in place."""
    import torch
    M, D, S, W, K = m.sizes
    B = x.shape[0]
    e = lambda *s: torch.empty(s, dtype=m.dtype, device="cuda")  # noqa: E731
    normed, stream, u, y = e(B, M), e(B, M), e(B, D), e(B, D)
    R.ret_rms_norm_fwd(x, normed, m.norm, residual=res, sum_out=stream)
    xz = normed @ m.w_in
    R.ret_short_conv_step(xz[:, :D], m.conv, u, conv, bias=m.conv_b)
    proj = u @ m.w_x
    b, c = (proj[:, K + i * S:K + (i + 1) * S].unflatten(-1, (1, S)) for i in (0, 1))
    R.ret_selective_scan_step(u, proj[:, :K] @ m.w_dt, m.A, b, c, y, scan, d_skip=m.skip, z=xz[:, D:], dt_bias=m.dt_bias)
    return y @ m.w_out, stream


def reference(m, x, res):
    """(out, stream) in the weights' type on the CPU, differentiable; the recurrence token by token."""
    import torch
    F = torch.nn.functional
    M, D, S, W, K = m.sizes
    stream = x + res
    normed = stream * (stream.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * m.norm
    xz = normed @ m.w_in
    rows = torch.cat([torch.zeros_like(xz[:, :W - 1, :D]), xz[..., :D]], 1)
    u = F.silu((rows.unfold(1, W, 1) * m.conv).sum(-1) + m.conv_b)
    proj = u @ m.w_x
    dt = F.softplus(proj[..., :K] @ m.w_dt + m.dt_bias)
    h, ys = x.new_zeros((x.shape[0], D, S)), []
    for t in range(x.shape[1]):
        h = torch.exp(dt[:, t, :, None] * m.A) * h + (dt * u)[:, t, :, None] * proj[:, t, None, K:K + S]
        ys.append((h * proj[:, t, None, K + S:]).sum(-1) + m.skip * u[:, t])
    return (torch.stack(ys, 1) * F.silu(xz[..., D:])) @ m.w_out, stream


def test_sequence_steps_and_gradients(R):
    """In fp32, against 64 bits. Every operator is within its own bound, and the projections add M, D and K terms in torch's
    order; what is asked of the whole is 2^-24 times 3000 (the scan's units, once and a half) of the largest value."""
    import torch
    B, N, M, D, S, W, K = 2, 70, 48, 64, 16, 4, 8
    m = Block(M, D, S, W, K, torch.float64, 1).to("cpu")
    gen = torch.Generator().manual_seed(2)
    x, res, dout, dstream = (rand(gen, B, N, M) for _ in range(4))
    leaves = [getattr(m, n).requires_grad_() for n in m.names]
    x64, r64 = x.double().requires_grad_(), res.double().requires_grad_()
    for n in m.names:
        setattr(m, n, getattr(m, n).double())
    want, stream = reference(m, x64, r64)
    loss = (want * dout.double()).sum() + (stream * dstream.double()).sum()
    grads = dict(zip(m.names + ("x",), torch.autograd.grad(loss, leaves + [x64])))
    g = Block(M, D, S, W, K, torch.float32, 1).to("cuda")
    print_case("scan block", B, N, M, D)
    xd, rd = x.cuda(), res.cuda()
    out, got_stream, k = forward(R, g, xd, rd)

    def near(name, got, ref):
        off, top = float((got.double().cpu() - ref).abs().max()), float(ref.abs().max())
        assert off <= 3000 * U * top, (name, off / top / U)
    near("out", out, want.detach())
    near("stream", got_stream, stream.detach())
    # the first 60 tokens at once, the rest one by one, from the states
    head, _, kh = forward(R, g, xd[:, :60].contiguous(), rd[:, :60].contiguous())
    conv, scan, rest = kh["conv_out"], kh["scan_out"], []
    for t in range(60, N):
        y, _ = step(R, g, xd[:, t].contiguous(), rd[:, t].contiguous(), conv, scan)
        rest.append(y[:, None])
    near("steps", torch.cat([head] + rest, 1), want.detach())
    # gradients, operator by operator
    dd = dout.cuda()
    e = torch.empty_like
    dy, dw_out = dd @ g.w_out.t(), (k["y"].flatten(0, 1).t() @ dd.flatten(0, 1))
    du, ddt, dA, db, dc = e(k["u"]), e(k["dt"]), e(g.A), torch.empty_like(k["b"].contiguous()), \
        torch.empty_like(k["c"].contiguous())
    dskip, dz, dbias = e(g.skip), torch.empty_like(k["u"]), e(g.dt_bias)
    R.ret_selective_scan_bwd(k["u"], k["dt"], g.A, k["b"], k["c"], dy, du, ddt, dA, db, dc, d_skip=g.skip, dd_skip=dskip,
                             z=k["z"], dz=dz, dt_bias=g.dt_bias, ddt_bias=dbias)
    dw_dt = k["proj"][..., :K].flatten(0, 1).t() @ ddt.flatten(0, 1)
    dproj = torch.cat([ddt @ g.w_dt.t(), db.flatten(-2), dc.flatten(-2)], -1)
    dw_x, du = k["u"].flatten(0, 1).t() @ dproj.flatten(0, 1), du + dproj @ g.w_x.t()
    dx, dconv, dconv_b = torch.empty_like(k["u"]), e(g.conv), e(g.conv_b)
    R.ret_short_conv_bwd(du, k["x"], g.conv, dx, dconv, bias=g.conv_b, dbias=dconv_b)
    dxz = torch.cat([dx, dz], -1)
    dw_in, dnormed = k["normed"].flatten(0, 1).t() @ dxz.flatten(0, 1), dxz @ g.w_in.t()
    dstr, dnorm = torch.empty_like(xd), e(g.norm)
    R.ret_rms_norm_bwd(dnormed, k["stream"], k["rstd"], dstr, weight=g.norm, dsum=dstream.cuda(), dweight=dnorm)
    for name, got in (("norm", dnorm), ("w_in", dw_in), ("conv", dconv), ("conv_b", dconv_b), ("w_x", dw_x), ("w_dt", dw_dt),
                      ("dt_bias", dbias), ("A", dA), ("skip", dskip), ("w_out", dw_out), ("x", dstr)):
        near("d " + name, got, grads[name])


def test_8_bits_stand_for_the_norm(R):
    """What a projection in 8 bits multiplies is the bf16 norm but for half a step of each format."""
    import torch
    x = torch.randn((5, 7, 256), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    y, y8 = torch.empty_like(x), torch.empty_like(x, dtype=torch.float8_e4m3fn)
    for group, n in ((None, 1), (64, 4)):
        scales = torch.empty((5, 7, n), device="cuda")
        R.ret_rms_norm_fwd(x, y, y8=y8, scales=scales, group=group)
        k = scales.repeat_interleave(256 // n, -1)
        off = (y8.float() * k - y.float()).abs()
        assert (off <= (2 ** -4 + 2 ** -8) * y.float().abs() + 2 ** -10 * k).all()


def test_8_bits_are_the_quotients(R):
    """Without a weight the values are exact but for their last rounding: the quotient comes in two parts, off by 2^-46 of itself
    before fp32 and e4m3 round it, so that 64 bits lead elsewhere only where it is that near to a border of both."""
    import torch
    for dtype, rows, D, group in ((torch.bfloat16, 256, 4096, None), (torch.float32, 64, 1001, 32), (torch.float32, 999, 256, 64)):
        gen = torch.Generator(device="cuda").manual_seed(D)
        x = torch.randn((rows, D), generator=gen, device="cuda").to(dtype)
        g = group or D
        y8, scales = torch.empty_like(x, dtype=torch.float8_e4m3fn), torch.empty((rows, -(-D // g)), device="cuda")
        print_case("quotients", rows, D, group)
        R.ret_rms_norm_fwd(x, y8=y8, scales=scales, group=group)
        for i, part in enumerate(x.double().split(g, 1)):
            want = (448 * part / part.abs().amax(1, keepdim=True)).float().to(torch.float8_e4m3fn)
            assert torch.equal(y8[:, i * g:(i + 1) * g].float(), want.float()), (D, i)


def test_captured_graphs(R):
    """A prompt, a step and the gradients, captured, replayed several times with eager work between, bit for bit the eager
    results; two graphs that share a workspace, in turn."""
    import torch
    B, N, D, S, W = 2, 300, 96, 16, 4
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s, t=torch.bfloat16: torch.randn(s, generator=gen, device="cuda").to(t)  # noqa: E731
    f32 = torch.float32
    x, res, w, cw = r(B, N, D), r(B, N, D), 1 + 0.1 * r(D, t=f32), r(D, W, t=f32)
    dt, b, c, z, A = r(B, N, D), r(B, N, 1, S), r(B, N, 1, S), r(B, N, D), -torch.rand((D, S), generator=gen, device="cuda") - 0.1
    opt = {"segments": 3}
    ws = R.selective_scan_workspace(x, b, opt)
    wsb = torch.empty((max(R.selective_scan_bwd_workspace(x, b).numel(), R.short_conv_bwd_workspace(x, cw).numel(),
                           R.rms_norm_bwd_workspace(x).numel()),), dtype=torch.uint8, device="cuda")
    e = torch.empty_like
    o = dict(n=e(x), s=e(x), rs=torch.empty((B, N), device="cuda"), y8=e(x, dtype=torch.float8_e4m3fn),
             sc=torch.empty((B, N, 1), device="cuda"), u=e(x), y=e(x), h=torch.empty((B, D, S), device="cuda"),
             cs=torch.empty((B, W - 1, D), dtype=x.dtype, device="cuda"), ys=torch.empty((B, D), dtype=x.dtype, device="cuda"),
             us=torch.empty((B, D), dtype=x.dtype, device="cuda"))
    first = [t[:, 0].contiguous() for t in (x, dt, b, c, z)]

    def prompt():
        R.ret_rms_norm_fwd(x, o["n"], w, residual=res, sum_out=o["s"], rstd=o["rs"], y8=o["y8"], scales=o["sc"])
        R.ret_short_conv_fwd(o["n"], cw, o["u"], state_out=o["cs"])
        R.ret_selective_scan_fwd(o["u"], dt, A, b, c, o["y"], z=z, state_out=o["h"], workspace=ws, options=opt)
        R.ret_short_conv_step(first[0], cw, o["us"], o["cs"])
        R.ret_selective_scan_step(o["us"], first[1], A, first[2], first[3], o["ys"], o["h"], z=first[4])

    d = dict(du=e(x), ddt=e(x), dA=e(A), db=e(b), dc=e(c), dz=e(x), dx=e(x), dcw=e(cw), dn=e(x), dw=e(w))

    def back():
        R.ret_selective_scan_bwd(o["u"], dt, A, b, c, x, d["du"], d["ddt"], d["dA"], d["db"], d["dc"], z=z, dz=d["dz"],
                                 workspace=wsb)
        R.ret_short_conv_bwd(d["du"], o["n"], cw, d["dx"], d["dcw"], workspace=wsb)
        R.ret_rms_norm_bwd(d["dx"], o["s"], o["rs"], d["dn"], weight=w, dweight=d["dw"], workspace=wsb)

    print_case("scan block graphs")
    prompt(), back()
    want = {k: v.clone() for k, v in {**o, **d}.items()}
    side = torch.cuda.Stream()
    graphs = []
    for call in (prompt, back):
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            call()
        graphs.append(g)
    torch.cuda.synchronize()
    for i in range(4):
        for v in list(o.values()) + list(d.values()):
            v.view(torch.uint8).fill_(i)
        ws.fill_(255), wsb.fill_(17 * i)
        graphs[0].replay()
        if i % 2:
            torch.cuda.synchronize()
        graphs[1].replay()
        back() if i == 2 else None
        torch.cuda.synchronize()
        for k, v in {**o, **d}.items():
            assert torch.equal(v.view(torch.uint8), want[k].view(torch.uint8)), (i, k)


# each of the three ways to cut a sequence up is some shape's own choice
@pytest.mark.parametrize("shape,kernels", [
    ((4, 130, 8192, 16), ("ret_scan_walk",)), ((1, 600, 4096, 16), ("ret_scan_chunks",)), ((1, 40, 64, 8), ("ret_scan_chunks",)),
    ((1, 5000, 512, 16), ("ret_scan_local", "ret_scan_join", "ret_scan_walk")), ((2, 300, 8192, 64), ("ret_scan_walk",)),
    ((1, 9000, 100, 32), ("ret_scan_local", "ret_scan_join", "ret_scan_walk")),
], ids=str)
def test_plans_agree(R, shape, kernels):
    """The call's own plan, the walk, the chunks and segments: each within units() of the same numbers. Decays of exp(-0.03) and
    less: no more than 900 tokens count."""
    import torch
    B, N, D, S = shape
    gen = torch.Generator(device="cuda").manual_seed(N)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    u, dt, z, b, c = r(B, N, D), r(B, N, D), r(B, N, D), r(B, N, 1, S), r(B, N, 1, S)
    A, bias, h0 = -1 - torch.rand((D, S), generator=gen, device="cuda"), torch.full((D,), -3.0, device="cuda"), r(B, D, S)
    lengths = torch.tensor([N] + [max(1, N // 3)] * (B - 1), dtype=torch.int32, device="cuda")
    outs = []
    for opt in ({}, {"variant": 1, "segments": 1}, {"variant": 2, "segments": 1}, {"segments": 7}, {"variant": 2, "segments": 2}):
        t = R.Timer()
        y, h = torch.full_like(u, 7.0), torch.empty_like(h0)
        R.ret_selective_scan_fwd(u, dt, A, b, c, y, z=z, dt_bias=bias, lengths=lengths, state_in=h0, state_out=h,
                                 options={**opt, "timer": t})
        if not opt:
            ran = [k for k in ("ret_scan_local", "ret_scan_join", "ret_scan_walk", "ret_scan_chunks") if t.query(k)[1]]
            assert tuple(ran) == kernels
        outs.append((y, h))
    # magnitudes: the same scan of magnitudes
    size, hs = torch.empty_like(u), torch.empty_like(h0)
    R.ret_selective_scan_fwd(u.abs(), dt, A, b.abs(), c.abs(), size, dt_bias=bias, lengths=lengths, state_in=h0.abs(),
                             state_out=hs)
    k = 2 * units(900, S) * U
    gate = torch.nn.functional.silu(z).abs()
    for y, h in outs[1:]:
        assert ((y - outs[0][0]).abs() <= k * size * gate + 1e-30).all()
        assert ((h - outs[0][1]).abs() <= k * hs + 1e-30).all()


@pytest.mark.parametrize("shape", [(3, 200, 512, 16), (2, 700, 1024, 16), (1, 5000, 512, 16), (5, 1000, 48, 8), (40, 20, 256, 32)],
                         ids=str)
def test_lengths_of_whole_sequences(R, shape):
    """Lengths change which part of the card does what, and nothing else: with those of whole sequences every output is that of
    the call without, bit for bit, and with others each sequence's is the same wherever in the batch it stands."""
    import torch
    B, N, D, S = shape
    gen = torch.Generator(device="cuda").manual_seed(13)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    t = dict(u=r(B, N, D), dt=r(B, N, D), b=r(B, N, 1, S), c=r(B, N, 1, S), z=r(B, N, D), dy=r(B, N, D),
             h0=r(B, D, S).float(), dh=r(B, D, S).float())
    A, bias = -1 - torch.rand((D, S), generator=gen, device="cuda"), torch.full((D,), -3.0, device="cuda")

    def call(t, lengths):
        e = torch.empty_like
        o = {k: e(t[k]) for k in ("u", "dt", "b", "c", "z", "dy", "h0", "dh")}
        dA, db = e(A), e(bias)
        R.ret_selective_scan_fwd(t["u"], t["dt"], A, t["b"], t["c"], o["dy"], z=t["z"], dt_bias=bias, lengths=lengths,
                                 state_in=t["h0"], state_out=o["h0"])
        R.ret_selective_scan_bwd(t["u"], t["dt"], A, t["b"], t["c"], t["dy"], o["u"], o["dt"], dA, o["b"], o["c"], z=t["z"],
                                 dz=o["z"], dt_bias=bias, ddt_bias=db, lengths=lengths, state_in=t["h0"],
                                 dstate_out=t["dh"], dstate_in=o["dh"])
        return o, (dA, db)
    print_case("lengths", B, N, D, S)
    want, sums = call(t, None)
    got, sums2 = call(t, torch.full((B,), N, dtype=torch.int32, device="cuda"))
    for k in want:
        assert torch.equal(got[k], want[k]), k
    assert torch.equal(sums[0], sums2[0]) and torch.equal(sums[1], sums2[1])
    lengths = torch.tensor([[0, 1, N, N // 3, 17][i % 5] for i in range(B)], dtype=torch.int32, device="cuda")
    one, _ = call(t, lengths)
    two, _ = call({k: v.flip(0) for k, v in t.items()}, lengths.flip(0))
    for k in want:
        assert torch.equal(one[k], two[k].flip(0)), k


def test_channels_apart(R):
    """A call's channels are those of calls on parts of them, bit for bit, and db and dc the parts' sums: each adds its channels
    in an order of its own, at most D roundings apart."""
    import torch
    B, N, D, S = 1, 4100, 1024, 16  # two blocks of channels a workgroup of the gradients; the parts one
    gen = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    u, dt, z, dy, b, c = r(B, N, D), r(B, N, D), r(B, N, D), r(B, N, D), r(B, N, 1, S), r(B, N, 1, S)
    A, bias = -1 - torch.rand((D, S), generator=gen, device="cuda"), torch.full((D,), -3.0, device="cuda")

    def call(s):
        cut = lambda t: t[..., s].contiguous()  # noqa: E731
        n = s.stop - s.start
        e = lambda *m: torch.empty(m, device="cuda")  # noqa: E731
        o = dict(du=e(B, N, n), ddt=e(B, N, n), dz=e(B, N, n), dA=e(n, S), dbias=e(n), db=e(B, N, 1, S), dc=e(B, N, 1, S))
        R.ret_selective_scan_bwd(cut(u), cut(dt), A[s].contiguous(), b, c, cut(dy), o["du"], o["ddt"], o["dA"], o["db"], o["dc"],
                                 z=cut(z), dz=o["dz"], dt_bias=bias[s].contiguous(), ddt_bias=o["dbias"])
        return o
    whole, parts = call(slice(0, D)), [call(slice(0, 400)), call(slice(400, D))]
    for k in ("du", "ddt", "dz"):
        assert torch.equal(whole[k], torch.cat([p[k] for p in parts], -1)), k
    for k in ("dA", "dbias"):
        assert torch.equal(whole[k], torch.cat([p[k] for p in parts], 0)), k
    for k in ("db", "dc"):
        both = parts[0][k].double() + parts[1][k].double()
        # the sum of magnitudes of 1024 terms is below sqrt(1024) times their root mean square
        size = 32 * float(both.square().mean().sqrt()) + both.abs()
        assert ((whole[k].double() - both).abs() <= 2 * D * U * size).all(), k


def test_many_sequences_and_rows(R):
    """More sequences than a launch axis other than x takes, and more rows than one x axis is given: the last ones right."""
    import torch
    B, D, S, W = 70001, 16, 8, 2
    gen = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    print_case("many sequences", B)
    x, cw, st = r(B, 3, D), r(D, W), r(B, 1, D)
    y, y1, s1 = torch.empty_like(x), torch.empty((B, D), device="cuda"), st.clone()
    R.ret_short_conv_fwd(x, cw, y, state_in=st)
    R.ret_short_conv_step(x[:, 0].contiguous(), cw, y1, s1)
    tail = slice(B - 3, B)
    t = torch.empty_like(x[tail])
    R.ret_short_conv_fwd(x[tail].contiguous(), cw, t, state_in=st[tail].contiguous())
    assert torch.equal(y[tail], t) and torch.equal(s1[:, 0], x[:, 0])
    # two taps of at most 6 x 6 in magnitude, each with a few roundings in one order or another
    assert float((y1 - y[:, 0]).abs().max()) <= 16 * U * 72
    dt, b, c, A = r(B, 3, D), r(B, 3, 1, S), r(B, 3, 1, S), -torch.rand((D, S), generator=gen, device="cuda") - 0.1
    h = torch.empty((B, D, S), device="cuda")
    R.ret_selective_scan_fwd(x, dt, A, b, c, y, state_out=h)
    ht, hb = torch.empty((3, D, S), device="cuda"), torch.zeros((B, D, S), device="cuda")
    cut = lambda v: v[tail].contiguous()  # noqa: E731
    R.ret_selective_scan_fwd(cut(x), cut(dt), A, cut(b), cut(c), t, state_out=ht, options={"variant": 1})
    for i in range(3):
        R.ret_selective_scan_step(*(v[:, i].contiguous() for v in (x, dt)), A, *(v[:, i].contiguous() for v in (b, c)), y1, hb)
    # a state is at most three terms of step length, u and b, each up to 6; both sides may be off by units() of that
    k = units(3, S) * U
    assert float((h[tail] - ht).abs().max()) <= 2 * k * 648 and float((h - hb).abs().max()) <= 2 * k * 648
    rows = (1 << 22) + 5
    v = r(rows, 7)
    out, part = torch.empty_like(v), torch.empty_like(v)
    R.ret_rms_norm_fwd(v, out)
    for a in range(0, rows, 1 << 21):
        R.ret_rms_norm_fwd(v[a:a + (1 << 21)], part[a:a + (1 << 21)])
    assert torch.equal(out, part)
