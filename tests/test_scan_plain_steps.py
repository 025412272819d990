"""The selective scan with steps as they are given (softplus=False): sequences by every plan, gradients, single tokens, against 64
bits. Tolerances: scan_ref.py, whose softplus and its slope are then exact. Steps of 0 among them: such a token leaves the
state as it is, and its gradient is that of the decay alone."""
import pytest

from tests.conftest import print_case
from tests.scan_ref import Scan, U, close, cuda, half_step, rand, scan_inputs, units

# (B, N, D, S, G, kind)
SHAPES = [(2, 150, 40, 8, 1, "f32"), (1, 300, 33, 16, 1, "bf16"), (3, 70, 32, 16, 2, "bf16-f32"), (2, 100, 20, 32, 1, "f32"),
          (1, 90, 48, 64, 1, "bf16")]


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


def _inputs(B, N, D, S, G, tin, seed):
    import torch
    x = scan_inputs(B, N, D, S, G, tin, seed)
    gen = torch.Generator().manual_seed(seed + 1)
    x["dt"] = torch.empty(B, N, D).uniform_(0.0, 0.4, generator=gen).to(tin)
    x["dt_bias"] = torch.empty(D).uniform_(0.0, 0.1, generator=gen)
    x["dt_bias"][::3] = 0.0
    x["dt"][:, N // 3:N // 3 + 5, ::3] = 0.0
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("bias", [True, False])
def test_sequences_and_gradients(R, shape, bias):
    import torch
    B, N, D, S, G, kind = shape
    tin, tout = _types(kind)
    x = _inputs(B, N, D, S, G, tin, N + D)
    if not bias:
        x["dt_bias"] = None
    lengths = [N, N - 7, 0][:B]
    gen = torch.Generator().manual_seed(N)
    h0, dS, dy = rand(gen, B, D, S), rand(gen, B, D, S), rand(gen, B, N, D, dtype=tin)
    ref = Scan(**x, softplus=False, lengths=lengths, state_in=h0)
    want, state, _ = ref.forward()
    size, ssize, _ = ref.forward(absolute=True)
    grads, gsize = ref.backward(dy, dS), ref.backward(dy, dS, absolute=True)
    d, ld = cuda(x), torch.tensor(lengths, dtype=torch.int32, device="cuda")
    new = lambda t, *s: torch.full(s, 7.0, dtype=t, device="cuda")  # noqa: E731
    k = units(N, S) * U
    for options in ({}, {"variant": 1}, {"variant": 2}, {"segments": 3}):
        print_case("plain_steps", shape, bias, options)
        y, out = new(tout, B, N, D), new(torch.float32, B, D, S)
        R.ret_selective_scan_fwd(d["u"], d["dt"], d["A"], d["b"], d["c"], y, d_skip=d["d_skip"], z=d["z"],
                                 dt_bias=d["dt_bias"], softplus=False, lengths=ld, state_in=h0.cuda(), state_out=out,
                                 options=options)
        close("y", y, want, half_step(tout), k * size)
        close("state", out, state, U, k * ssize)
    print_case("plain_steps gradients", shape, bias)
    f = torch.float32
    o = [new(tout, B, N, D), new(tout, B, N, D), new(f, D, S), new(tout, B, N, G, S), new(tout, B, N, G, S), new(f, D),
         new(tout, B, N, D), new(f, D), new(f, B, D, S)]
    R.ret_selective_scan_bwd(d["u"], d["dt"], d["A"], d["b"], d["c"], dy.cuda(), *o[:5], d_skip=d["d_skip"], dd_skip=o[5],
                             z=d["z"], dz=o[6], dt_bias=d["dt_bias"], ddt_bias=o[7], softplus=False, lengths=ld,
                             state_in=h0.cuda(), dstate_out=dS.cuda(), dstate_in=o[8])
    k, toks, chans = units(N, S, grad=True) * U, B * N * U, D // G * U
    more = (0, 0, toks, chans, chans, toks, 0, toks, 0)
    for name, g, r, s, m in zip(("du", "ddt", "dA", "db", "dc", "dskip", "dz", "dbias", "dstate_in"), o, grads, gsize, more):
        close(name, g, r, half_step(g.dtype), (k + m) * s)


@pytest.mark.gpu
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16-f32"])
def test_step(R, S, kind):
    import torch
    tin, tout = _types(kind)
    B, D, G = 3, 96, 2
    print_case("plain_steps step", S, kind)
    x = _inputs(B, 1, D, S, G, tin, S)
    h0 = rand(torch.Generator().manual_seed(B), B, D, S)
    ref = Scan(**x, softplus=False, state_in=h0)
    want, state, _ = ref.forward()
    size, ssize, _ = ref.forward(absolute=True)
    d = cuda({k: v if k in ("A", "d_skip", "dt_bias") else v[:, 0].contiguous() for k, v in x.items()})
    y, h = torch.empty((B, D), dtype=tout, device="cuda"), h0.cuda()
    R.ret_selective_scan_step(d["u"], d["dt"], d["A"], d["b"], d["c"], y, h, d_skip=d["d_skip"], z=d["z"],
                              dt_bias=d["dt_bias"], softplus=False)
    k = units(1, S) * U
    close("y", y, want[:, 0], half_step(tout), k * size[:, 0])
    close("state", h, state, U, k * ssize)
