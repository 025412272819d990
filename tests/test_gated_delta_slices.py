"""Gates and lengths that are slices of larger tensors: the kernels read them one element at a time, so an element's
alignment is all they need. Tolerances as in test_gated_delta.py and test_gated_delta_grad.py."""
import numpy as np
import pytest

import tests.test_gated_delta as fwd
import tests.test_gated_delta_grad as bwd
from tests.conftest import print_case
from tests.delta_ref import forward, gradients, inputs, np64, term_sums
from tests.test_gated_delta_checks import _bwd, _fwd

M = 1 << 24


@pytest.fixture(scope="module")
def lib():
    from linear_recurrent_sequence_amd import retention
    return retention.load()


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


@pytest.mark.parametrize("kw", [dict(g=4 * M + 4), dict(beta=5 * M + 12), dict(g=4 * M + 2, beta=5 * M + 6, gd=1),
                                dict(lengths=15 * M + 4)], ids=str)
def test_element_alignment_is_taken(lib, kw):
    """The call goes on to the next check (a missing workspace); nothing is launched."""
    assert _fwd(lib, **kw, ws=None) == -3
    assert _bwd(lib, **kw, ws=None) == -3


def test_gradient_gates_too(lib):
    assert _bwd(lib, dg=10 * M + 4, dbeta=11 * M + 8, ws=None) == -3
    assert _bwd(lib, dg=10 * M + 2, dbeta=11 * M + 2, gd=1, ws=None) == -3


@pytest.mark.parametrize("kw", [dict(g=4 * M + 2), dict(beta=5 * M + 1, gd=1), dict(lengths=15 * M + 2)], ids=str)
def test_less_than_an_element_is_refused(lib, kw):
    assert _fwd(lib, **kw, ws=None) == -1
    assert _bwd(lib, **kw, ws=None) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("gates", ["f32", "bf16"])
def test_single_sequence_decodes_from_slices(R, gates):
    """B = 1: g[:, t] of a [1, N, H] tensor is contiguous where it lies, at any multiple of H elements."""
    import torch
    N, H, Hk, dk, dv = 9, 6, 2, 32, 48
    print_case("gated_delta_step_slices", gates)
    x = inputs(2, 1, N, H, Hk, dk, dv, "bf16", gates)
    d = {n: t.cuda() for n, t in x.items()}
    state, outs, odd = torch.zeros(1, H, dk, dv, device="cuda"), [], 0
    for t in range(N):
        g, beta = d["g"][:, t].contiguous(), d["beta"][:, t].contiguous()
        odd += g.data_ptr() % 16 != 0
        o = torch.empty(1, H, dv, device="cuda")
        R.ret_gated_delta_step(d["q"][:, t].clone(), d["k"][:, t].clone(), d["v"][:, t].clone(), g, beta, o, state)
        outs.append(o[:, None])
    assert odd
    ro, rs, _ = forward(*[np64(x[n]) for n in ("q", "k", "v", "g", "beta")], dk ** -0.5)
    fwd.check("o", torch.cat(outs, 1), ro, "f32")
    fwd.check("state", state, rs, "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("gates", ["f32", "bf16"])
def test_sequences_from_slices(R, gates):
    """Gates, their gradients and lengths of the last sequences of a batch: views that start at an odd element."""
    import torch
    B, N, H, Hk, dk, dv = 2, 70, 3, 3, 32, 32
    print_case("gated_delta_slices", gates)
    x = inputs(5, B + 1, N + 1, H, Hk, dk, dv, "bf16", gates)
    flat = {n: x[n].cuda().reshape(-1)[1:1 + B * N * H].view(B, N, H) for n in ("g", "beta")}
    x = {n: x[n][1:, 1:].contiguous() if n in ("q", "k", "v") else flat[n].cpu() for n in x}
    lens = torch.tensor([3, 70, 33], dtype=torch.int32, device="cuda")[1:]
    d = {n: x[n].cuda() if n in ("q", "k", "v") else flat[n] for n in x}
    assert d["g"].data_ptr() % 16 and lens.data_ptr() % 16
    o, s = torch.empty_like(d["v"]), torch.empty(B, H, dk, dv, device="cuda")
    R.ret_gated_delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], o, lengths=lens, state_out=s)
    a, n = [np64(x[m]) for m in ("q", "k", "v", "g", "beta")], np.array([70, 33])
    ro, rs, before = forward(*a, dk ** -0.5, None, n)
    fwd.check("o", o, ro, "bf16", term_sums(*a, dk ** -0.5, before))
    fwd.check("state", s, rs, "bf16")
    dout = torch.randn(B, N, H, dv, generator=torch.Generator().manual_seed(6)).bfloat16()
    gr = [torch.empty_like(d[m]) for m in ("q", "k", "v")]
    buf = torch.full((2, B * N * H + 2), 7.0, dtype=d["g"].dtype, device="cuda")
    dg, db = (b[1:-1].view(B, N, H) for b in buf)
    R.ret_gated_delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], dout.cuda(), *gr, dg, db, lengths=lens)
    bwd.check(gr + [dg, db], gradients(*a, dk ** -0.5, np64(dout), lengths=n)[:5], "bf16")
    assert (buf[:, 0] == 7).all() and (buf[:, -1] == 7).all()
