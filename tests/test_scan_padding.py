"""Gradients of the selective scan where a token past its sequence's end would count if its factors of zero met something that is
not finite: a decay rate at the end of fp32's range (or minus infinity), a state or a state's gradient that is infinite or
NaN. Against 64 bits; tolerances: scan_ref.py."""
import numpy as np
import pytest

from tests.conftest import print_case
from tests.scan_ref import Scan, U, close, cuda, half_step, rand, scan_inputs, units

NAMES = ("du", "ddt", "dA", "db", "dc", "dskip", "dz", "dbias", "dstate_in")


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


def _gradients(R, x, dy, dS, h0, lengths, tout):
    """The gradients by NAMES; x, dy, dS, h0 on the CPU."""
    import torch
    B, N, D = x["u"].shape
    S, G = x["A"].shape[1], x["b"].shape[2]
    d, new = cuda(x), lambda t, *s: torch.full(s, 7.0, dtype=t, device="cuda")  # noqa: E731
    f = torch.float32
    o = dict(zip(NAMES, (new(tout, B, N, D), new(tout, B, N, D), new(f, D, S), new(tout, B, N, G, S), new(tout, B, N, G, S),
                         new(f, D), new(tout, B, N, D), new(f, D), new(f, B, D, S))))
    ld = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    R.ret_selective_scan_bwd(d["u"], d["dt"], d["A"], d["b"], d["c"], dy.cuda(), o["du"], o["ddt"], o["dA"], o["db"], o["dc"],
                             d_skip=d["d_skip"], dd_skip=o["dskip"], z=d["z"], dz=o["dz"], dt_bias=d["dt_bias"],
                             ddt_bias=o["dbias"], lengths=ld, state_in=h0.cuda(), dstate_out=dS.cuda(),
                             dstate_in=o["dstate_in"])
    return o


def _reference(x, dy, dS, h0, lengths, absolute=False):
    """The 64-bit gradients of each sequence cut to its length, by NAMES; zeros behind it."""
    B, N, D = x["u"].shape
    S, G = x["A"].shape[1], x["b"].shape[2]
    w = {k: np.zeros((B, N, G, S) if k in ("db", "dc") else (D, S) if k == "dA" else (D,) if k in ("dskip", "dbias") else
                     (B, D, S) if k == "dstate_in" else (B, N, D)) for k in NAMES}
    for i, n in enumerate(lengths):
        one = {k: v[i:i + 1, :n] if k in ("u", "dt", "b", "c", "z") else v for k, v in x.items()}
        with np.errstate(invalid="ignore"):
            got = dict(zip(NAMES, Scan(**one, state_in=h0[i:i + 1]).backward(dy[i:i + 1, :n], dS[i:i + 1], absolute=absolute)))
        for k in NAMES:
            if k in ("dA", "dskip", "dbias"):
                w[k] += got[k]
            elif k == "dstate_in":
                w[k][i] = got[k][0]
            else:
                w[k][i, :n] = got[k][0]
    return w


def _padding(o, lengths):
    for i, n in enumerate(lengths):
        for name in ("du", "ddt", "db", "dc", "dz"):
            assert not o[name][i, n:].any(), (name, i)  # NaN counts as any


def _compare(o, x, dy, dS, h0, lengths, tout):
    """What 64 bits give as finite is finite and right; the rest is not finite."""
    import torch
    B, N, D = x["u"].shape
    S, G = x["A"].shape[1], x["b"].shape[2]
    want, size = (_reference(x, dy, dS, h0, lengths, absolute=a) for a in (False, True))
    k, half = units(N, S, grad=True) * U, half_step(tout)
    more = dict(dA=B * N * U, db=D // G * U, dc=D // G * U, dskip=B * N * U, dbias=B * N * U)
    for name in NAMES:
        fine = np.isfinite(want[name])
        at, got = torch.from_numpy(fine), o[name].cpu()
        assert fine.any() and not torch.isfinite(got[~at]).any(), name
        close(name, got[at], want[name][fine], half if got.dtype == tout else U, (k + more.get(name, 0)) * size[name][fine])


# every number of states; N = 150 ends within a chunk (128, 32 or 16 tokens) and within a wave's block of 16, 8 or 4
@pytest.mark.gpu
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [None, [145, 70]], ids=str)
def test_states_without_memory(R, S, kind, lengths):
    """Decay rates from -1e30 to minus infinity: no state outlives a token, and the padding's steps of 0 leave the last one
    where it is. Its product with the rate is outside of fp32 and has no part in any gradient."""
    import torch
    print_case("states_without_memory", S, kind, lengths)
    tin = torch.float32 if kind == "f32" else torch.bfloat16
    B, N, D, G = 2, 150, 20, 1
    gen = torch.Generator().manual_seed(S)
    x = scan_inputs(B, N, D, S, G, tin, 71)
    x["A"][1], x["A"][4, ::3], x["A"][7], x["A"][19] = -1e30, -1e38, -3e38, -1e37
    h0, dS, dy = rand(gen, B, D, S), rand(gen, B, D, S, scale=10.0), rand(gen, B, N, D, dtype=tin)
    o = _gradients(R, x, dy, dS, h0, lengths, tin)
    _padding(o, lengths or [N, N])
    assert torch.isfinite(o["dbias"]).all()
    _compare(o, x, dy, dS, h0, lengths or [N, N], tin)
    x["A"][7] = float("-inf")
    same = _gradients(R, x, dy, dS, h0, lengths, tin)
    assert all(torch.equal(o[k], same[k]) for k in NAMES)


@pytest.mark.gpu
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("bad", ["u", "state_in", "dstate_out"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")], ids=str)
def test_states_that_are_not_finite(R, S, bad, value):
    """An infinity or NaN in channel 5 of the first sequence: in the input of its last token (the state that the padding
    keeps), in the entering state, in the last state's gradient. The padding is zero all the same."""
    import torch
    print_case("states_that_are_not_finite", S, bad, value)
    B, N, D, G, lengths = 2, 150, 20, 1, [133, 70]
    gen = torch.Generator().manual_seed(S)
    x = scan_inputs(B, N, D, S, G, torch.float32, 72)
    h0, dS, dy = rand(gen, B, D, S), rand(gen, B, D, S), rand(gen, B, N, D)
    if bad == "u":
        x["u"][0, lengths[0] - 1, 5] = value
    elif bad == "state_in":
        h0[0, 5, S // 2] = value
    else:
        dS[0, 5, S // 2] = value
    o = _gradients(R, x, dy, dS, h0, lengths, torch.float32)
    _padding(o, lengths)
    _compare(o, x, dy, dS, h0, lengths, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_steps_that_underflow(R, S, kind):
    """Steps of exp(-200) and exp(-180), 0 in fp32 as their derivatives, of channels without memory: the state stays as it is,
    and its product with the rate, which is outside of fp32, has no part in the step's gradient. In 64 bits that is
    3e38 exp(-180) = 2e-40 times a state and its gradient: nothing beside what close() allows for fp32's range."""
    import torch
    print_case("steps_that_underflow", S, kind)
    tin = torch.float32 if kind == "f32" else torch.bfloat16
    B, N, D, G, lengths = 2, 150, 20, 1, [150, 90]
    gen = torch.Generator().manual_seed(S)
    x = scan_inputs(B, N, D, S, G, tin, 73)
    x["A"][1], x["A"][7], x["A"][19, ::2] = -1e38, -3e38, -2e38
    for d in (1, 7, 19):
        x["dt_bias"][d] = 0.0
        x["dt"][:, 20:45, d], x["dt"][:, 80:, d] = -200.0, -180.0
    h0, dS, dy = rand(gen, B, D, S), rand(gen, B, D, S, scale=10.0), rand(gen, B, N, D, dtype=tin)
    o = _gradients(R, x, dy, dS, h0, lengths, tin)
    _padding(o, lengths)
    assert torch.isfinite(o["ddt"]).all() and torch.isfinite(o["dbias"]).all()
    _compare(o, x, dy, dS, h0, lengths, tin)
    x["A"][7] = float("-inf")
    same = _gradients(R, x, dy, dS, h0, lengths, tin)
    assert all(torch.equal(o[k], same[k]) for k in NAMES)
