"""Sizes at which the block's kernels loop more than once: several value heads per workgroup of the chunk matrices,
rows and partial sums past one pass of the grid, default plans of many segments. Tolerances as derived in
test_block_norms.py, test_gated_delta.py and test_gated_delta_grad.py."""
import numpy as np
import pytest

import tests.test_gated_delta as fwd
import tests.test_gated_delta_grad as bwd
from tests.conftest import print_case
from tests.delta_ref import forward, gradients, inputs, np64, term_sums
from tests.test_block_norms import U, _close, _epi_ref, _half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_recurrent_sequence_amd import retention
    retention.load(build_if_missing=True)
    return retention


# 4 sequences of 18 chunks and 8 value heads: 576 workgroups, more than delta_prep starts one by one, so that one of them
# has the 4 value heads of a key head; and few heads of many chunks, which the default plan cuts in 10 and 11 segments
@pytest.mark.parametrize("dtype,gates,B,N,H,Hk,dk,dv", [
    ("f32", "f32", 4, 1100, 8, 2, 32, 16), ("bf16", "f32", 4, 1100, 8, 2, 32, 16), ("bf16", "bf16", 4, 1100, 8, 2, 32, 16),
    ("f32", "f32", 1, 2500, 2, 1, 32, 48), ("bf16", "f32", 1, 2500, 1, 1, 64, 64), ("bf16", "f32", 1, 2777, 2, 2, 128, 80)])
def test_delta_rule(R, dtype, gates, B, N, H, Hk, dk, dv):
    import torch
    print_case("gated_delta_loops", dtype, gates, B, N, H, Hk, dk, dv)
    x = inputs(N, B, N, H, Hk, dk, dv, dtype, gates)
    gen = torch.Generator().manual_seed(1)
    dout = torch.randn(B, N, H, dv, generator=gen).to(x["q"].dtype)
    lengths = None if B == 1 else [N, 1030, N - 1, 700]
    ln = None if lengths is None else np.array(lengths)
    a = [np64(x[n]) for n in ("q", "k", "v", "g", "beta")]
    o, s = fwd.run(R, x, H, dv, None, lengths)
    ro, rs, before = forward(*a, dk ** -0.5, None, ln)
    fwd.check("o", o, ro, dtype, term_sums(*a, dk ** -0.5, before))
    fwd.check("state", s, rs, dtype)
    got = bwd.run(R, x, dout, None, None, lengths)
    bwd.check(got, gradients(*a, dk ** -0.5, np64(dout), None, None, ln), dtype)


# workgroups: 256 at most, of 1, 1, 16 and 64 rows
@pytest.mark.parametrize("rows,D", [(600, 8192), (600, 16383), (4500, 257), (16700, 104)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_layer_norm_gradients(R, rows, D, kind):
    import torch
    print_case("layer_norm_loops", rows, D, kind)
    t = torch.float32 if kind == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(D)
    x, dy = (torch.randn(rows, D, generator=g) + 0.5).to(t), torch.randn(rows, D, generator=g).to(t)
    w = 1 + 0.2 * torch.randn(D, generator=g)
    y, dx = (torch.empty(rows, D, dtype=t, device="cuda") for _ in range(2))
    mean, rstd, dw, db = (torch.empty(n, device="cuda") for n in (rows, rows, D, D))
    xd = x.cuda()
    R.ret_layer_norm_fwd(xd, y, w.cuda(), mean=mean, rstd=rstd)
    R.ret_layer_norm_bwd(dy.cuda(), xd, mean, rstd, dx, weight=w.cuda(), dweight=dw, dbias=db)
    x64, d64, w64 = x.double().numpy(), dy.double().numpy(), w.double().numpy()
    m, r = mean.double().cpu().numpy()[:, None], rstd.double().cpu().numpy()[:, None]
    m64 = x64.mean(-1, keepdims=True)
    r64 = 1 / np.sqrt(((x64 - m64) ** 2).mean(-1, keepdims=True) + 1e-5)
    big = np.abs(x64).max() * r64.max()
    _close("mean", mean, m64[:, 0], U, 64 * U * np.abs(x64).max())
    _close("rstd", rstd, r64[:, 0], 64 * U + 64 * U * big, 0.0)
    xh, a = (x64 - m) * r, d64 * w64
    _close("y", y, xh * w64, _half_step(t), 64 * U * (1 + big + np.abs(xh).max()) * np.abs(w64).max())
    ref = r * (a - a.mean(-1, keepdims=True) - xh * (a * xh).mean(-1, keepdims=True))
    _close("dx", dx, ref, _half_step(t), 64 * U * r.max() * np.abs(a).max() * (1 + np.abs(xh).max() ** 2) * (1 + big))
    adds = rows + 64
    _close("dweight", dw, (d64 * xh).sum(0), U, adds * U * (np.abs(d64) * (np.abs(xh) + big)).sum(0).max())
    _close("dbias", db, d64.sum(0), U, adds * U * np.abs(d64).sum(0).max())


# strips: 512 of 16 rows for one block of channels, 171 for three
@pytest.mark.parametrize("rows,H,dv", [(9000, 1, 16), (3000, 3, 512)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_epilogue_gradients(R, rows, H, dv, kind):
    import torch
    print_case("epilogue_loops", rows, H, dv, kind)
    t = torch.float32 if kind == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(dv)
    dy, o = (torch.randn(rows, H, dv, generator=g).to(t) for _ in range(2))
    gate = (2 * torch.randn(rows, H, dv, generator=g)).to(t)
    w, b = 1 + 0.2 * torch.randn(H * dv, generator=g), 0.3 * torch.randn(H * dv, generator=g)
    do, dgate = (torch.empty(rows, H, dv, dtype=t, device="cuda") for _ in range(2))
    dw, db = (torch.empty(H * dv, device="cuda") for _ in range(2))
    R.ret_msr_epilogue_bwd(dy.cuda(), o.cuda(), do, gate=gate.cuda(), dgate=dgate, gn_weight=w.cuda(), gn_bias=b.cuda(),
                           dweight=dw, dbias=db)
    n64 = lambda z: z.double().numpy()  # noqa: E731
    w64, b64 = n64(w).reshape(H, dv), n64(b).reshape(H, dv)
    rdo, rdg, dn, xh, rstd = _epi_ref(n64(o), n64(gate), w64, b64, n64(dy), 1e-5)
    big, wmax, dnm = np.abs(n64(o)).max() * rstd.max(), np.abs(w64).max(), np.abs(dn).max()
    _close("do", do, rdo, _half_step(t), 64 * U * rstd.max() * dnm * wmax * (1 + np.abs(xh).max() ** 2) * (1 + big))
    _close("dgate", dgate, rdg, _half_step(t),
           64 * U * np.abs(n64(dy)).max() * ((np.abs(xh).max() + big) * wmax + np.abs(b64).max()) * 8)
    adds = rows + 64
    _close("dweight", dw, (dn * xh).sum(0).reshape(-1), U, adds * U * (np.abs(dn) * (np.abs(xh) + big)).sum(0).max())
    _close("dbias", db, dn.sum(0).reshape(-1), U, adds * U * np.abs(dn).sum(0).max())
