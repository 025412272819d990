"""Single tokens of more sequences than a sequence call takes at once: 4096 and 8192 of 16 heads."""
import pytest

import tests.test_gated_delta as fwd
from tests.conftest import print_case
from tests.delta_ref import forward, inputs, np64
from tests.test_gated_delta_checks import _fwd, _step


def test_refusals():
    from linear_recurrent_sequence_amd import retention
    lib = retention.load()
    assert _step(lib, B=8193, H=16, Hk=16, dk=16, dv=16) == -2 and b"131072" in lib.ret_last_error()
    assert _fwd(lib, B=4096, H=16, Hk=16) == -2 and b"65535" in lib.ret_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("B,dtype", [(4096, "bf16"), (8192, "f32")])
def test_step_of_many_sequences(B, dtype):
    """Against the recurrence at both ends and around 65536 heads, and bit for bit against calls on parts of the batch."""
    import torch
    from linear_recurrent_sequence_amd import retention as R
    H, dk, dv = 16, 16, 16
    print_case("gated_delta_step_many", B, dtype)
    x = {n: t[:, 0].contiguous() for n, t in inputs(1, B, 1, H, H, dk, dv, dtype).items()}
    d = {n: t.cuda() for n, t in x.items()}
    start = torch.randn(B, H, dk, dv, generator=torch.Generator().manual_seed(2))
    names, outs = ("q", "k", "v", "g", "beta"), []
    for step in (B, 1024):
        o, s = torch.full((B, H, dv), 7.0, device="cuda"), start.cuda()
        for b in range(0, B, step):
            R.ret_gated_delta_step(*[d[n][b:b + step] for n in names], o[b:b + step], s[b:b + step])
        outs.append((o, s))
    assert all(torch.equal(p, q) for p, q in zip(*outs))
    for at in (0, 4095, B - 1):
        ro, rs, _ = forward(*[np64(x[n][at:at + 1])[:, None] for n in names], dk ** -0.5, np64(start[at:at + 1]))
        fwd.check("o", outs[0][0][at:at + 1], ro[:, 0], "f32")
        fwd.check("state", outs[0][1][at:at + 1], rs, "f32")
