"""The selective scan (sequences, single tokens, gradients) against 64 bits, token by token. Tolerances: scan_ref.py."""
import numpy as np
import pytest

from tests.conftest import print_case
from tests.scan_ref import Scan, U, close, cuda, half_step, rand, scan_inputs, units


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


def _call(R, x, y, **kw):
    d = cuda(x)
    return R.ret_selective_scan_fwd(d["u"], d["dt"], d["A"], d["b"], d["c"], y, d_skip=d["d_skip"], z=d["z"],
                                    dt_bias=d["dt_bias"], **kw)


def test_formulas_by_differentiation():
    """The 64-bit gradients are those that torch finds by differentiating the recurrence (no GPU)."""
    import torch
    B, N, D, S, G = 2, 7, 6, 8, 2
    x = scan_inputs(B, N, D, S, G, torch.float32, 3)
    lengths = [7, 4]
    gen = torch.Generator().manual_seed(4)
    h0, dS, dy = rand(gen, B, D, S), rand(gen, B, D, S), rand(gen, B, N, D)
    leaf = {k: v.double().requires_grad_() for k, v in x.items()}
    leaf["h0"] = h0.double().requires_grad_()
    h, loss = leaf["h0"], 0
    for t in range(N):
        live = torch.tensor([[t < n] for n in lengths])
        dt = torch.nn.functional.softplus(leaf["dt"][:, t] + leaf["dt_bias"]) * live
        b, c = (leaf[k][:, t].repeat_interleave(D // G, 1) for k in ("b", "c"))
        h = torch.exp(dt[..., None] * leaf["A"]) * h + (dt * leaf["u"][:, t])[..., None] * b
        y = ((c * h).sum(-1) + leaf["d_skip"] * leaf["u"][:, t]) * torch.nn.functional.silu(leaf["z"][:, t])
        loss = loss + (y * dy[:, t].double() * live).sum()
    loss = loss + (h * dS.double()).sum()
    want = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    got = Scan(**x, lengths=lengths, state_in=h0).backward(dy, dS)
    for name, g in zip(("u", "dt", "A", "b", "c", "d_skip", "z", "dt_bias", "h0"), got):
        assert np.abs(g - want[name].numpy()).max() <= 1e-12 * (1 + np.abs(g).max()), name


# (B, N, D, S, G, kind, options): one token, odd lengths around the blocks of 256 / S and chunks of 2048 / S tokens (1024 / S
# where S > 16), channels around the blocks of 16, every number of states and type, one and two groups
SHAPES = [
    (1, 1, 1, 16, 1, "f32"), (2, 2, 16, 8, 1, "bf16"), (1, 15, 17, 16, 1, "f32"), (3, 16, 5, 32, 1, "bf16"),
    (2, 17, 33, 64, 1, "f32"), (1, 31, 48, 8, 1, "bf16-f32"), (2, 33, 20, 8, 1, "f32"), (2, 127, 32, 16, 2, "bf16"),
    (1, 128, 100, 16, 1, "f32"), (2, 129, 64, 16, 2, "bf16-f32"), (1, 333, 250, 8, 1, "f32"), (2, 300, 40, 32, 1, "f32"),
    (1, 257, 96, 64, 2, "bf16"), (2, 700, 18, 16, 1, "f32"), (1, 1100, 16, 8, 1, "bf16"), (5, 64, 7, 16, 1, "bf16"),
]


def _lengths(B, N, ragged):
    return None if not ragged else [N, 0, N // 2 + 1, 1, N - 1][:B] if B > 1 else [max(1, N - 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("ragged", [False, True])
def test_forward(R, shape, ragged):
    import torch
    B, N, D, S, G, kind = shape
    tin, tout = _types(kind)
    for segments, full in ((0, True), (3, True), (1, False)):
        print_case("selective_scan", shape, ragged, segments, full)
        x = scan_inputs(B, N, D, S, G, tin, N + D)
        lengths = _lengths(B, N, ragged)
        h0 = rand(torch.Generator().manual_seed(1), B, D, S) if full else None
        if not full:
            x.update(d_skip=None, z=None, dt_bias=None)
        ref = Scan(**x, lengths=lengths, state_in=h0)
        want, state, _ = ref.forward()
        size, ssize, _ = ref.forward(absolute=True)
        if lengths is not None:  # inputs past a length are not read into anything
            for i, n in enumerate(lengths):
                for k in ("u", "dt", "z", "b", "c"):
                    if x[k] is not None:
                        x[k][i, n:] = float("nan")
        y = torch.full((B, N, D), 7.0, dtype=tout, device="cuda")
        out = torch.full((B, D, S), 7.0, device="cuda")
        ld = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        _call(R, x, y, lengths=ld, state_in=None if h0 is None else h0.cuda(), state_out=out,
              options={"segments": segments})
        k = units(N, S) * U
        close("y", y, want, half_step(tout), k * size)
        close("state", out, state, U, k * ssize)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("ragged", [False, True])
def test_gradients(R, shape, ragged):
    import torch
    B, N, D, S, G, kind = shape
    tin, tout = _types(kind)
    gen = torch.Generator().manual_seed(N)
    for full in (True, False):
        print_case("selective_scan_bwd", shape, ragged, full)
        x = scan_inputs(B, N, D, S, G, tin, N + D + 1)
        lengths = _lengths(B, N, ragged)
        h0, dS = (rand(gen, B, D, S) for _ in range(2)) if full else (None, None)
        dy = rand(gen, B, N, D, dtype=tin)
        if not full:
            x.update(d_skip=None, z=None, dt_bias=None)
        ref = Scan(**x, lengths=lengths, state_in=h0)
        want, size = ref.backward(dy, dS), ref.backward(dy, dS, absolute=True)
        if lengths is not None:
            for i, n in enumerate(lengths):
                for k in ("u", "dt", "z", "b", "c"):
                    if x[k] is not None:
                        x[k][i, n:] = float("nan")
                dy[i, n:] = float("nan")
        d, new = cuda(x), lambda t, *s: torch.full(s, 7.0, dtype=t, device="cuda")  # noqa: E731
        du, ddt, dz = (new(tout, B, N, D) for _ in range(3))
        db, dc = (new(tout, B, N, G, S) for _ in range(2))
        dA, dskip, dbias = new(torch.float32, D, S), new(torch.float32, D), new(torch.float32, D)
        dS0 = new(torch.float32, B, D, S) if full else None
        ld = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        R.ret_selective_scan_bwd(d["u"], d["dt"], d["A"], d["b"], d["c"], dy.cuda(), du, ddt, dA, db, dc,
                                 d_skip=d["d_skip"], dd_skip=dskip if full else None, z=d["z"], dz=dz if full else None,
                                 dt_bias=d["dt_bias"], ddt_bias=dbias, lengths=ld,
                                 state_in=None if h0 is None else h0.cuda(),
                                 dstate_out=None if dS is None else dS.cuda(), dstate_in=dS0)
        k, half = units(N, S, grad=True) * U, half_step(tout)
        chans, toks = D // G * U, B * N * U
        names = ("du", "ddt", "dA", "db", "dc", "dskip", "dz", "dbias", "dstate_in")
        got = (du, ddt, dA, db, dc, dskip if full else None, dz if full else None, dbias, dS0)
        halves = (half, half, U, half, half, U, half, U, U)
        more = (0, 0, toks, chans, chans, toks, 0, toks, 0)
        for name, g, r, s, h, m in zip(names, got, want, size, halves, more):
            if g is not None:
                close(name, g, r, h, (k + m) * s)


@pytest.mark.gpu
def test_gradients_against_differences(R):
    """Along a random direction, against the 64-bit forward: a step of 1e-4 leaves 1e-8 of the third derivative (below 1e3
    here) and 1e-12 of rounding; the gradients their fp32 arithmetic."""
    import torch
    B, N, D, S, G = 1, 40, 24, 16, 1
    x = scan_inputs(B, N, D, S, G, torch.float32, 11)
    gen = torch.Generator().manual_seed(12)
    h0, dS, dy = rand(gen, B, D, S), rand(gen, B, D, S), rand(gen, B, N, D)
    d, e = cuda(x), lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    g = dict(u=e(B, N, D), dt=e(B, N, D), A=e(D, S), b=e(B, N, G, S), c=e(B, N, G, S), d_skip=e(D), z=e(B, N, D),
             dt_bias=e(D), state_in=e(B, D, S))
    R.ret_selective_scan_bwd(d["u"], d["dt"], d["A"], d["b"], d["c"], dy.cuda(), g["u"], g["dt"], g["A"], g["b"], g["c"],
                             d_skip=d["d_skip"], dd_skip=g["d_skip"], z=d["z"], dz=g["z"], dt_bias=d["dt_bias"],
                             ddt_bias=g["dt_bias"], state_in=h0.cuda(), dstate_out=dS.cuda(), dstate_in=g["state_in"])

    def loss(v):
        y, h, _ = Scan(**{k: t for k, t in v.items() if k != "state_in"}, state_in=v["state_in"]).forward()
        return float((y * dy.double().numpy()).sum() + (h * dS.double().numpy()).sum())

    at = {k: v.double() for k, v in x.items()} | {"state_in": h0.double()}
    sizes = dict(zip(("u", "dt", "A", "b", "c", "d_skip", "z", "dt_bias", "state_in"),
                     Scan(**x, state_in=h0).backward(dy, dS, absolute=True)))
    for name in at:
        way = torch.randn(at[name].shape, generator=gen, dtype=torch.float64)
        step = 1e-4
        num = (loss(at | {name: at[name] + step * way}) - loss(at | {name: at[name] - step * way})) / (2 * step)
        got = float((g[name].double().cpu() * way).sum())
        arith = units(N, S, grad=True) * U * float((sizes[name] * way.abs().numpy()).sum())
        assert abs(num - got) <= arith + 1e-8 * 1e3, (name, num, got)


@pytest.mark.gpu
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16-f32"])
def test_step(R, S, kind):
    import torch
    tin, tout = _types(kind)
    for B, D, G, full in [(1, 1, 1, True), (3, 100, 1, False), (2, 96, 2, True), (5, 33, 1, True)]:
        print_case("selective_scan_step", S, kind, B, D, G)
        x = scan_inputs(B, 1, D, S, G, tin, D + S)
        if not full:
            x.update(d_skip=None, z=None, dt_bias=None)
        h0 = rand(torch.Generator().manual_seed(B), B, D, S)
        ref = Scan(**x, state_in=h0)
        want, state, _ = ref.forward()
        size, ssize, _ = ref.forward(absolute=True)
        d = cuda({k: v if v is None or k in ("A", "d_skip", "dt_bias") else v[:, 0] for k, v in x.items()})
        y, h = torch.empty((B, D), dtype=tout, device="cuda"), h0.cuda()
        R.ret_selective_scan_step(d["u"], d["dt"], d["A"], d["b"], d["c"], y, h, d_skip=d["d_skip"], z=d["z"],
                                  dt_bias=d["dt_bias"])
        k = units(1, S) * U
        close("y", y, want[:, 0], half_step(tout), k * size[:, 0])
        close("state", h, state, U, k * ssize)


@pytest.mark.gpu
def test_resumed_and_stepped(R):
    """A sequence in one call, in two with the state in between, and its last tokens one by one; the state in place."""
    import torch
    B, N, D, S, G = 2, 301, 40, 16, 1
    x = scan_inputs(B, N, D, S, G, torch.float32, 21)
    ref = Scan(**x)
    want, state, _ = ref.forward()
    size, ssize, _ = ref.forward(absolute=True)
    k = units(N, S) * U
    d = cuda(x)
    cut = lambda s: {n: v[:, s].contiguous() if n in ("u", "dt", "z", "b", "c") else v for n, v in x.items()}  # noqa: E731
    h = torch.empty((B, D, S), device="cuda")
    first, second = torch.empty((B, 200, D), device="cuda"), torch.empty((B, 95, D), device="cuda")
    _call(R, cut(slice(0, 200)), first, state_out=h)
    _call(R, cut(slice(200, 295)), second, state_in=h, state_out=h)
    ys = [first, second]
    for t in range(295, N):
        y = torch.empty((B, D), device="cuda")
        p = {n: d[n][:, t].contiguous() for n in ("u", "dt", "z", "b", "c")}
        R.ret_selective_scan_step(p["u"], p["dt"], d["A"], p["b"], p["c"], y, h, d_skip=d["d_skip"], z=p["z"],
                                  dt_bias=d["dt_bias"])
        ys.append(y[:, None])
    close("y", torch.cat(ys, 1), want, U, k * size)
    close("state", h, state, U, k * ssize)
    # state in place where the sequence is in several segments
    h2, y2, y3, h3 = rand(torch.Generator().manual_seed(5), B, D, S).cuda(), torch.empty((B, N, D), device="cuda"), \
        torch.empty((B, N, D), device="cuda"), torch.empty((B, D, S), device="cuda")
    _call(R, x, y3, state_in=h2, state_out=h3, options={"segments": 3})
    _call(R, x, y2, state_in=h2, state_out=h2, options={"segments": 3})
    assert torch.equal(y2, y3) and torch.equal(h2, h3)


@pytest.mark.gpu
def test_extreme_values(R):
    """Step lengths from softplus over its whole range; a channel without memory (A = -inf, -1e30), one that keeps all
    (A = 0), one that grows; a NaN and an infinity reach later tokens only."""
    import torch
    B, N, D, S = 1, 150, 16, 16
    x = scan_inputs(B, N, D, S, 1, torch.float32, 31)
    raw = torch.linspace(-100, 40, N)
    x["dt"][0, :, 0], x["dt_bias"][0], x["A"][0] = raw, 0.0, 0.0
    x["A"][1], x["A"][2] = -1e30, 0.0
    x["A"][3] = 0.01
    ref = Scan(**x)
    want, state, _ = ref.forward()
    size, ssize, _ = ref.forward(absolute=True)
    y, h = torch.empty((B, N, D), device="cuda"), torch.empty((B, D, S), device="cuda")
    _call(R, x, y, state_out=h)
    k = units(N, S) * U
    close("y", y, want, U, k * size + 1e-37)
    close("state", h, state, U, k * ssize + 1e-37)
    x["A"][1] = float("-inf")
    y2 = torch.empty_like(y)
    ld = torch.tensor([N - 5], dtype=torch.int32, device="cuda")
    _call(R, x, y2, lengths=ld, state_out=h)
    assert torch.equal(y2[:, :N - 5], y[:, :N - 5]) and torch.isfinite(h).all() and not y2[:, N - 5:].any()
    for bad, t in ((float("nan"), 70), (float("inf"), 17)):
        p = {n: None if v is None else v.clone() for n, v in x.items()}
        p["u"][0, t, 5] = bad
        y3 = torch.empty_like(y)
        _call(R, p, y3)
        _call(R, x, y2)
        others = [c for c in range(D) if c != 5]
        assert torch.equal(y3[:, :t], y2[:, :t]) and torch.equal(y3[..., others], y2[..., others])
        assert not torch.isfinite(y3[0, t, 5])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices(R, dtype):
    """z, b and c as slices of wider rows, at offsets that the vectors do not take, give the bits of whole tensors."""
    import torch
    tin, _ = _types(dtype)
    B, N, D, S, G = 2, 70, 32, 16, 2
    x = cuda(scan_inputs(B, N, D, S, G, tin, 41))
    base = torch.empty((B, N, D), dtype=tin, device="cuda")
    put = lambda y, z, b, c: R.ret_selective_scan_fwd(x["u"], x["dt"], x["A"], b, c, y, z=z)  # noqa: E731
    put(base, x["z"], x["b"], x["c"])
    for pad in (1, 4, 8):
        wide = torch.full((B, N, pad + D + 2 * G * S + 3), float("nan"), dtype=tin, device="cuda")
        if pad != 1:
            wide = torch.full((B, N, pad + D + 2 * G * S + 4), float("nan"), dtype=tin, device="cuda")
        z, b, c = wide[..., pad:pad + D], wide[..., pad + D:pad + D + G * S].unflatten(-1, (G, S)), \
            wide[..., pad + D + G * S:pad + D + 2 * G * S].unflatten(-1, (G, S))
        z.copy_(x["z"]), b.copy_(x["b"]), c.copy_(x["c"])
        y = torch.empty_like(base)
        put(y, z, b, c)
        assert torch.equal(y, base), pad
        p = lambda t: t[:, 0]  # noqa: E731
        h, h2 = torch.ones((B, D, S), device="cuda"), torch.ones((B, D, S), device="cuda")
        y1, y2 = torch.empty((B, D), dtype=tin, device="cuda"), torch.empty((B, D), dtype=tin, device="cuda")
        R.ret_selective_scan_step(p(x["u"]).contiguous(), p(x["dt"]).contiguous(), x["A"], p(b), p(c), y1, h, z=p(z))
        R.ret_selective_scan_step(p(x["u"]).contiguous(), p(x["dt"]).contiguous(), x["A"], p(x["b"]).contiguous(),
                                  p(x["c"]).contiguous(), y2, h2, z=p(x["z"]).contiguous())
        assert torch.equal(y1, y2) and torch.equal(h, h2)
        g1, g2 = [], []
        for out, (zz, bb, cc) in ((g1, (x["z"], x["b"], x["c"])), (g2, (z, b, c))):
            e = lambda *s, t=tin: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
            o = [e(B, N, D), e(B, N, D), e(D, S, t=torch.float32), e(B, N, G, S), e(B, N, G, S), e(B, N, D)]
            R.ret_selective_scan_bwd(x["u"], x["dt"], x["A"], bb, cc, base, *o[:5], z=zz, dz=o[5])
            out += o
        assert all(torch.equal(a, b2) for a, b2 in zip(g1, g2))


@pytest.mark.gpu
def test_streams_and_repeats(R):
    """The same bits on another stream, twice in a row, from a workspace of other content, and from two calls at once."""
    import torch
    B, N, D, S, G = 2, 400, 48, 16, 1
    x = cuda(scan_inputs(B, N, D, S, G, torch.bfloat16, 51))
    opt = {"segments": 2}

    def both(stream=None, ws=None, wsb=None):
        e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        o = [e(B, N, D), e(B, N, D), e(B, N, D), e(D, S, t=torch.float32), e(B, N, G, S), e(B, N, G, S), e(B, N, D)]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        R.ret_selective_scan_fwd(x["u"], x["dt"], x["A"], x["b"], x["c"], o[0], z=x["z"], workspace=ws, stream=stream,
                                 options=opt)
        R.ret_selective_scan_bwd(x["u"], x["dt"], x["A"], x["b"], x["c"], x["z"], *o[1:6], z=x["z"], dz=o[6],
                                 workspace=wsb, stream=stream)
        return o
    want = both()
    dirty = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in
             (R.selective_scan_workspace(x["u"], x["b"], opt).numel(), R.selective_scan_bwd_workspace(x["u"], x["b"]).numel())]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [both(), both(ws=dirty[0], wsb=dirty[1]), both(stream=s1), both(stream=s2)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.gpu
def test_offsets_past_32_bits(R):
    """A tensor of more than 2^31 elements: its last tokens, against the same tokens from the state before them."""
    import torch
    N, D, S = 70000, 32768, 8
    gen = torch.Generator(device="cuda").manual_seed(61)
    u, dt = (torch.randn((1, N, D), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    b, c = (torch.randn((1, N, 1, S), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    A, bias = -torch.rand((D, S), generator=gen, device="cuda") - 0.5, torch.full((D,), -3.0, device="cuda")
    y, h = torch.empty_like(u), torch.empty((1, D, S), device="cuda")
    R.ret_selective_scan_fwd(u, dt, A, b, c, y, dt_bias=bias, state_out=h)
    cut = N - 400
    part = [t[:, :cut] for t in (u, dt, b, c)]
    mid, y0, y1, h1 = torch.empty_like(h), torch.empty_like(u[:, :cut]), torch.empty_like(u[:, cut:]), torch.empty_like(h)
    R.ret_selective_scan_fwd(part[0], part[1], A, part[2], part[3], y0, dt_bias=bias, state_out=mid)
    R.ret_selective_scan_fwd(u[:, cut:].contiguous(), dt[:, cut:].contiguous(), A, b[:, cut:].contiguous(),
                             c[:, cut:].contiguous(), y1, dt_bias=bias, state_in=mid, state_out=h1)
    # both sides are within units() of the same numbers; decays of exp(-0.02) and less keep no more than 1500 tokens of them
    size = float(h.abs().max())
    assert float((h - h1).abs().max()) <= 2 * units(1500, S) * U * 40 * size
    off = (y[:, cut:].float() - y1.float()).abs().max()
    assert float(off) <= 2 ** -7 * float(y1.abs().max())
    assert torch.equal(y[:, :cut], y0)
