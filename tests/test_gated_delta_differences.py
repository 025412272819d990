"""Gradients of the gated delta rule against differences of its forward.

Moving one entry of one token, the loss L = sum(dout o) + sum(dstate state) is a polynomial: of degree one in q, v, beta
and the entering state, of degree two in k, which stands in the read and in the write; and A + B exp(g) in g. Central
differences are exact for the first four and for k, and for g once they are multiplied by h / sinh(h). Nothing is left but
rounding: the forward is within 3e-6 of the recurrence in the 2-norm (test_gated_delta.py), so that a loss is off by at
most 3e-6 (|dout| |o| + |dstate| |state|), a difference by that over h, and the gradient itself by 1e-5 of its tensor's
2-norm (test_gated_delta_grad.py). Each gradient tested is more than ten times the sum of both."""
import numpy as np
import pytest

from tests.conftest import print_case
from tests.delta_ref import forward, gradients, inputs, np64

NAMES = ("q", "k", "v", "g", "beta", "state")
STEP = dict(q=1.0, k=0.5, v=1.0, g=0.5, beta=0.5, state=1.0)
B, N, H, Hk, DK, DV = 1, 70, 2, 1, 16, 16


def case():
    import torch
    x = inputs(7, B, N, H, Hk, DK, DV, "f32")
    gen = torch.Generator().manual_seed(8)
    dout, dstate, state = (torch.randn(*s, generator=gen) for s in ((B, N, H, DV), (B, H, DK, DV), (B, H, DK, DV)))
    return dict(x, state=state), dout, dstate


def entries(name, ref):
    """The largest gradients of the whole tensor, of its first 20 tokens and of those after the first chunk."""
    a, out = np.abs(ref), []
    for lo, hi in ((0, None),) if name == "state" else ((0, None), (0, 20), (64, None)):
        part = a if name == "state" else a[:, lo:hi]
        for flat in np.argsort(part.reshape(-1))[-3:]:
            at = list(np.unravel_index(flat, part.shape))
            if name != "state":
                at[1] += lo
            out.append(tuple(int(i) for i in at))
    return sorted(set(out))


def compare(x, dout, dstate, run, noise, got):
    """run(inputs) -> (o, state) in 64-bit arrays; got: the gradients to test; noise: of an output, of a gradient."""
    a = {n: np64(x[n]) for n in NAMES}
    d, ds = np64(dout), np64(dstate)
    ref = dict(zip(NAMES, gradients(*[a[n] for n in NAMES[:5]], DK ** -0.5, d, a["state"], ds)))
    loss = lambda o, s: (o * d).sum() + (s * ds).sum()  # noqa: E731
    norm = lambda z: np.sqrt((z ** 2).sum())  # noqa: E731
    for name in NAMES:
        for at in entries(name, ref[name]):
            h, sides, size = STEP[name], [], 0.0
            for sign in (1, -1):
                y = {n: t.clone() for n, t in x.items()}
                y[name][at] += sign * h
                o, s = run(y)
                size = max(size, norm(d) * norm(o) + norm(ds) * norm(s))
                sides.append((loss(o, s), float(y[name][at].double())))
            num = (sides[0][0] - sides[1][0]) / (sides[0][1] - sides[1][1])
            if name == "g":
                num *= h / np.sinh(h)
            tol = noise[0] * size / h + noise[1] * norm(ref[name])
            assert abs(ref[name][at]) > 10 * tol, ("too small to tell", name, at, ref[name][at], tol)
            assert abs(num - got[name][at]) <= tol, (name, at, num, got[name][at], tol)


def test_reference():
    """The 64-bit gradients against differences of the 64-bit forward: the polynomials are what they are said to be."""
    x, dout, dstate = case()
    x = {n: t.double() for n, t in x.items()}
    a = [np64(x[n]) for n in NAMES]
    got = dict(zip(NAMES, gradients(*a[:5], DK ** -0.5, np64(dout), a[5], np64(dstate))))

    def run(y):
        o, s, _ = forward(*[np64(y[n]) for n in NAMES[:5]], DK ** -0.5, np64(y["state"]))
        return o, s

    compare(x, dout, dstate, run, (1e-12, 1e-12), got)


@pytest.mark.gpu
def test_kernels():
    import torch
    from linear_recurrent_sequence_amd import retention as R
    print_case("gated_delta_differences")
    x, dout, dstate = case()
    dev = {n: t.cuda() for n, t in x.items()}
    grads = [torch.empty_like(dev[n]) for n in NAMES]
    R.ret_gated_delta_bwd(*[dev[n] for n in NAMES[:5]], dout.cuda(), *grads[:5], state_in=dev["state"],
                          dstate_out=dstate.cuda(), dstate_in=grads[5])
    got = {n: t.double().cpu().numpy() for n, t in zip(NAMES, grads)}

    def run(y):
        y = {n: t.cuda() for n, t in y.items()}
        o, s = torch.empty(B, N, H, DV, device="cuda"), torch.empty(B, H, DK, DV, device="cuda")
        R.ret_gated_delta_fwd(*[y[n] for n in NAMES[:5]], o, state_in=y["state"], state_out=s)
        return o.double().cpu().numpy(), s.double().cpu().numpy()

    compare(x, dout, dstate, run, (3e-6, 1e-5), got)
