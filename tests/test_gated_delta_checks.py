"""The gated delta rule's refusals and workspace queries (no GPU, nothing is launched)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from linear_recurrent_sequence_amd import retention
    return retention.load()


def _fwd(lib, **kw):
    M = 1 << 24
    a = dict(q=1 * M, k=2 * M, v=3 * M, g=4 * M, beta=5 * M, o=6 * M, B=1, N=64, H=2, Hk=2, dk=64, dv=64, ind=1, outd=1,
             gd=0, scale=0.0, lengths=None, sin=None, sout=None, ws=8 * M, wsb=1 << 24)
    a.update(kw)
    return lib.ret_gated_delta_fwd(*list(a.values()), None, None)


def _step(lib, **kw):
    M = 1 << 24
    a = dict(q=1 * M, k=2 * M, v=3 * M, g=4 * M, beta=5 * M, o=6 * M, state=7 * M, B=1, H=2, Hk=2, dk=64, dv=64, ind=1,
             outd=1, gd=0, scale=0.0)
    a.update(kw)
    return lib.ret_gated_delta_step(*list(a.values()), None, None)


@pytest.mark.parametrize("fn", [_fwd, _step])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(g=None), -1), (dict(o=None), -1), (dict(B=0), -1), (dict(H=3), -1), (dict(Hk=0), -1),
    (dict(dk=0), -1), (dict(dk=48), -2), (dict(dk=512), -2), (dict(dv=24), -2), (dict(dv=-16), -1), (dict(ind=2), -1),
    (dict(ind=0, outd=1), -1), (dict(ind=0, outd=0, gd=1), -1), (dict(gd=3), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(q=(1 << 24) + 8), -1), (dict(o=3 << 24), -1), (dict(o=(1 << 24) + 64), -1),
    (dict(B=70000), -2), (dict(H=1 << 16, Hk=1, dv=64), -2),
])
def test_refusals(lib, fn, kw, status):
    assert fn(lib, **kw) == status
    assert lib.ret_last_error() != b""


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), -1), (dict(N=-3), -1), (dict(ws=None), -3), (dict(wsb=1000), -3), (dict(ws=(8 << 24) + 4), -1),
    (dict(ws=3 << 24), -1), (dict(sin=9 << 24, sout=(9 << 24) + 64), -1), (dict(sout=6 << 24), -1),
    (dict(lengths=(9 << 24) + 2), -1), (dict(dk=16), -2), (dict(ind=0, outd=0, dk=256), -2),
])
def test_sequence_refusals(lib, kw, status):
    assert _fwd(lib, **kw) == status


def test_step_needs_a_state_of_its_own(lib):
    assert _step(lib, state=None) == -1
    assert _step(lib, state=3 << 24) == -1


def test_workspace_queries(lib):
    q = lambda *a: lib.ret_gated_delta_workspace_bytes(*a, None)  # noqa: E731
    assert q(1, 64, 2, 2, 48, 64, 1) == 0 and q(1, 0, 2, 2, 64, 64, 1) == 0 and q(1, 64, 3, 2, 64, 64, 1) == 0
    assert q(1, 64, 2, 2, 64, 24, 1) == 0 and q(1, 64, 2, 2, 64, 64, 5) == 0
    assert 0 < q(1, 64, 2, 2, 64, 64, 1) < q(1, 128, 2, 2, 64, 64, 1)


def test_binding_checks():
    import torch
    from linear_recurrent_sequence_amd import retention as R
    q, v, g = torch.zeros(1, 8, 2, 64), torch.zeros(1, 8, 4, 32), torch.zeros(1, 8, 4)
    bad = [dict(k=torch.zeros(1, 8, 2, 32)), dict(v=torch.zeros(1, 8, 3, 32)), dict(g=torch.zeros(1, 8, 2)),
           dict(beta=g.bfloat16()), dict(o=torch.zeros(1, 8, 4, 16)), dict(o=None), dict(g=None), dict(scale=0.0),
           dict(lengths=torch.zeros(1, dtype=torch.int64)), dict(state_in=torch.zeros(1, 4, 64, 16)),
           dict(state_out=torch.zeros(1, 4, 64, 32, dtype=torch.bfloat16)), dict(q=q.half(), k=q.half()), dict()]
    for kw in bad:  # the last: everything fits but nothing is on a GPU
        a = dict(q=q, k=q, v=v, g=g, beta=g, o=torch.zeros_like(v)) | kw
        with pytest.raises(ValueError):
            R.ret_gated_delta_fwd(**a)
    s = torch.zeros(1, 4, 64, 32)
    for kw in (dict(state=None), dict(state=s[:, :2]), dict(q=torch.zeros(1, 3, 64)), dict()):
        a = dict(q=q[:, 0], k=q[:, 0], v=v[:, 0], g=g[:, 0], beta=g[:, 0], o=v[:, 0], state=s) | kw
        with pytest.raises(ValueError):
            R.ret_gated_delta_step(**a)


def _bwd(lib, **kw):
    M = 1 << 24
    a = dict(q=1 * M, k=2 * M, v=3 * M, g=4 * M, beta=5 * M, dout=6 * M, dq=7 * M, dk_out=8 * M, dv_out=9 * M, dg=10 * M,
             dbeta=11 * M, B=1, N=64, H=2, Hk=2, dk=64, dv=64, ind=1, outd=1, gd=0, scale=0.0, lengths=None, sin=None,
             dsout=None, dsin=None, ws=12 * M, wsb=1 << 24)
    a.update(kw)
    return lib.ret_gated_delta_bwd(*list(a.values()), None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(dout=None), -1), (dict(dq=None), -1), (dict(dbeta=None), -1), (dict(B=0), -1),
    (dict(N=0), -1), (dict(H=3), -1), (dict(Hk=0), -1), (dict(dk=48), -2), (dict(dk=512), -2), (dict(dv=24), -2),
    (dict(ind=2), -1), (dict(ind=0, outd=1), -1), (dict(ind=0, outd=0, gd=1), -1), (dict(gd=3), -1),
    (dict(scale=float("nan")), -1), (dict(q=(1 << 24) + 8), -1), (dict(dout=(6 << 24) + 8), -1),
    (dict(dq=3 << 24), -1), (dict(dk_out=7 << 24), -1), (dict(dg=11 << 24), -1), (dict(dsin=6 << 24), -1),
    (dict(sin=13 << 24, dsin=(13 << 24) + 64), -1), (dict(dsout=13 << 24, dsin=13 << 24), -1),
    (dict(lengths=(13 << 24) + 2), -1), (dict(ws=None), -3), (dict(wsb=1000), -3), (dict(ws=(12 << 24) + 4), -1),
    (dict(ws=3 << 24), -1), (dict(B=70000), -2), (dict(H=1 << 16, Hk=1), -2), (dict(dk=16), -2),
    (dict(ind=0, outd=0, dk=256), -2), (dict(H=1, Hk=1, dk=256, dv=1 << 21), -2),
])
def test_gradient_refusals(lib, kw, status):
    assert _bwd(lib, **kw) == status
    assert lib.ret_last_error() != b""


def test_states_past_32_bit_offsets_are_refused(lib):
    for fn in (_fwd, _step):
        assert fn(lib, H=1, Hk=1, dk=256, dv=1 << 20) == -2
    assert lib.ret_gated_delta_workspace_bytes(1, 64, 1, 1, 256, 1 << 20, 1, None) == 0


def test_gradient_workspace_query(lib):
    q = lambda *a: lib.ret_gated_delta_bwd_workspace_bytes(*a, None)  # noqa: E731
    assert q(1, 64, 2, 2, 48, 64, 1) == 0 and q(1, 0, 2, 2, 64, 64, 1) == 0 and q(1, 64, 3, 2, 64, 64, 1) == 0
    assert lib.ret_gated_delta_workspace_bytes(1, 64, 2, 2, 64, 64, 1, None) < q(1, 64, 2, 2, 64, 64, 1)
    assert q(1, 64, 2, 2, 64, 64, 1) < q(1, 128, 2, 2, 64, 64, 1)


def test_gradient_binding_checks():
    import torch
    from linear_recurrent_sequence_amd import retention as R
    q, v, g = torch.zeros(1, 8, 2, 64), torch.zeros(1, 8, 4, 32), torch.zeros(1, 8, 4)
    base = dict(q=q, k=q, v=v, g=g, beta=g, dout=v, dq=torch.zeros_like(q), dk=torch.zeros_like(q),
                dv=torch.zeros_like(v), dg=torch.zeros_like(g), dbeta=torch.zeros_like(g))
    bad = [dict(dout=None), dict(dout=v.bfloat16()), dict(dq=None), dict(dq=v), dict(dv=q), dict(dk=base["dk"].bfloat16()),
           dict(dg=torch.zeros(1, 8, 2)), dict(dbeta=g.bfloat16()), dict(scale=0.0),
           dict(lengths=torch.zeros(2, dtype=torch.int32)), dict(state_in=torch.zeros(1, 4, 64, 16)),
           dict(dstate_out=torch.zeros(1, 4, 64, 32).bfloat16()), dict(dstate_in=torch.zeros(4, 64, 32)), dict()]
    for kw in bad:  # the last: everything fits but nothing is on a GPU
        with pytest.raises(ValueError):
            R.ret_gated_delta_bwd(**(base | kw))
