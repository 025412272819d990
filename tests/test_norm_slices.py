"""Layer norm whose statistics are slices of those of more rows. Tolerances as in test_block_norms.py: the same call on
whole tensors has to give the same bits."""
import pytest

from tests.conftest import print_case
from tests.test_norm_overlaps import M, _ln, _lnb


@pytest.mark.parametrize("fn", ["_ln", "_lnb"])
@pytest.mark.parametrize("kw", [dict(mean=12 * M + 2), dict(rstd=13 * M + 1)], ids=str)
def test_less_than_a_float_is_refused(fn, kw):
    from linear_recurrent_sequence_amd import retention
    lib = retention.load()
    assert {"_ln": _ln, "_lnb": _lnb}[fn](lib, **kw) == -1
    assert b"4-byte aligned" in lib.ret_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 1001])
def test_statistics_from_slices(D):
    import torch
    from linear_recurrent_sequence_amd import retention as R
    rows = 6
    print_case("layer_norm_slices", D)
    gen = torch.Generator().manual_seed(D)
    x, dy = (torch.randn(rows, D, generator=gen).cuda() for _ in range(2))
    got, want = [], []
    for at, out in ((0, want), (1, got), (3, got)):
        stats = torch.full((2, rows + 5), 7.0, device="cuda")
        mean, rstd = stats[0, at:at + rows], stats[1, at:at + rows]
        y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(D, device="cuda")
        if at == 0:
            mean, rstd = mean.clone(), rstd.clone()
        R.ret_layer_norm_fwd(x, y, mean=mean, rstd=rstd)
        R.ret_layer_norm_bwd(dy, x, mean, rstd, dx, dweight=dw)
        out.append([t.clone() for t in (y, dx, dw, mean, rstd)])
        if at:
            assert (stats[:, :at] == 7).all() and (stats[:, at + rows:] == 7).all()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want[0]))
