"""The selective scan, the short convolution and RMS norm in 64 bits, token by token on the CPU, and how far fp32 arithmetic
may be off.

absolute=True runs the same sums over the terms' magnitudes. A contribution to a state passes, per token, one product and one
sum (2 roundings of 2^-24) and a decay exp2(dt A log2 e) with its own error of one unit and, from its argument, (|raw| + 4)
units times |dt A| (raw: the softplus's argument, below 16 in these tests). The |dt A| of its way add up to the logarithm of
its decay; where that is over 20 the contribution is below 2^-28 of what it was, so at most 20 * 20 units come from
arguments. Up to S + 30 more come from the sum over the states, the gate (the hardware sigmoid's argument and itself, |z| + 4
with |z| below 16) and the step. Back through the gradient the way is gone twice. So an output of N tokens is off by at most
    units(N, S) = 400 + 3 N + S  (forward),  800 + 6 N + S  (gradients)  times 2^-24 of the sum of magnitudes,
and sums over tokens or channels add one unit per term that they add one after another."""
import numpy as np

U = 2.0 ** -24


def units(N, S, grad=False):
    return (800 + 6 * N if grad else 400 + 3 * N) + S


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def sigmoid(x):
    return 1 / (1 + np.exp(-x))


class Scan:
    """One call's inputs (torch tensors of any type and device, b and c [B, N, G, S]) in 64 bits."""

    def __init__(self, u, dt, A, b, c, d_skip=None, z=None, dt_bias=None, softplus=True, lengths=None, state_in=None):
        self.u, self.A = _np(u), _np(A)
        B, N, D = self.u.shape
        S, G = self.A.shape[1], b.shape[2]
        self.size = B, N, D, S, G
        raw = _np(dt) + (0 if dt_bias is None else _np(dt_bias))
        self.dt = np.logaddexp(raw, 0) if softplus else raw
        self.slope = sigmoid(raw) if softplus else np.ones_like(raw)
        self.b, self.c = (np.repeat(_np(t), D // G, axis=2) for t in (b, c))
        self.skip = 0 * self.A[:, 0] if d_skip is None else _np(d_skip)
        zz = _np(z)
        self.gate = np.ones_like(raw) if z is None else zz * sigmoid(zz)
        self.dgate = np.zeros_like(raw) if z is None else sigmoid(zz) * (1 + zz * (1 - sigmoid(zz)))
        n = [N] * B if lengths is None else [min(max(int(x), 0), N) for x in lengths]
        # its terms' magnitudes: silu' is 0 at z = -1.28, where they cancel
        self.mgate = np.zeros_like(raw) if z is None else sigmoid(zz) * (1 + np.abs(zz) * (1 - sigmoid(zz)))
        self.live = (np.arange(N)[None] < np.array(n)[:, None])[..., None]
        keep = lambda x: np.where(self.live, x, 0)  # noqa: E731
        for name in ("u", "dt", "slope", "gate", "dgate", "mgate"):
            setattr(self, name, keep(getattr(self, name)))
        self.b, self.c = (np.where(self.live[..., None], x, 0) for x in (self.b, self.c))
        self.h0 = np.zeros((B, D, S)) if state_in is None else _np(state_in)

    def forward(self, absolute=False):
        """(y, state after the last token, states before and after every token)."""
        f = np.abs if absolute else (lambda x: x)
        B, N, D, S, G = self.size
        h, states = f(self.h0), [f(self.h0)]
        y = np.zeros((B, N, D))
        for t in range(N):
            a = np.exp(self.dt[:, t, :, None] * self.A)
            h = a * h + f((self.dt * self.u)[:, t, :, None] * self.b[:, t])
            states.append(h)
            y[:, t] = (f(self.c[:, t]) * h).sum(-1) + f(self.skip * self.u[:, t])
        self.plain = y
        return y * f(self.gate), h, states

    def backward(self, dy, dstate_out=None, absolute=False):
        """du, ddt, dA, db, dc, dskip, dz, dbias, dstate_in."""
        f = np.abs if absolute else (lambda x: x)
        B, N, D, S, G = self.size
        _, _, states = self.forward(absolute)
        dy = np.where(self.live, f(_np(dy)), 0)
        dp, dz = dy * f(self.gate), dy * self.plain * (self.mgate if absolute else self.dgate)
        g = np.zeros((B, D, S)) if dstate_out is None else f(_np(dstate_out))
        du, dd = np.zeros((B, N, D)), np.zeros((B, N, D))
        db, dc, dA = np.zeros((B, N, G, S)), np.zeros((B, N, G, S)), np.zeros((D, S))
        for t in reversed(range(N)):
            a = np.exp(self.dt[:, t, :, None] * self.A)
            g = g + dp[:, t, :, None] * f(self.c[:, t])
            dc[:, t] = (dp[:, t, :, None] * states[t + 1]).reshape(B, G, D // G, S).sum(2)
            db[:, t] = (f(self.dt * self.u)[:, t, :, None] * g).reshape(B, G, D // G, S).sum(2)
            gb = (g * f(self.b[:, t])).sum(-1)
            g = g * a
            along = g * states[t]
            dd[:, t] = ((along * f(self.A)).sum(-1) + f(self.u[:, t]) * gb) * self.slope[:, t]
            du[:, t] = f(self.dt[:, t]) * gb + f(self.skip) * dp[:, t]
            dA += (along * f(self.dt[:, t, :, None])).sum(0)
        return du, dd, dA, db, dc, (dp * f(self.u)).sum((0, 1)), dz, dd.sum((0, 1)), g


def conv(x, w, bias=None, silu=True, lengths=None, state_in=None, dy=None, dstate_out=None, absolute=False):
    """y, state_out, and with dy also dx, dw, dbias, dstate_in. absolute: magnitudes of the terms, with those of silu and its
    derivative s(1 + p) and s(1 + p)^2, p the sum of pre's magnitudes (see test_short_conv.py)."""
    f = np.abs if absolute else (lambda v: v)
    x, w = _np(x), _np(w)
    B, N, D = x.shape
    W = w.shape[1]
    n = [N] * B if lengths is None else [min(max(int(v), 0), N) for v in lengths]
    live = (np.arange(N)[None] < np.array(n)[:, None])[..., None]
    first = np.zeros((B, W - 1, D)) if state_in is None else _np(state_in)
    rows = np.concatenate([first, np.where(live, x, 0)], 1)
    bias = np.zeros(D) if bias is None else _np(bias)
    pre = sum(rows[:, j:j + N] * w[:, j] for j in range(W)) + bias
    apre = sum(np.abs(rows[:, j:j + N] * w[:, j]) for j in range(W)) + np.abs(bias)
    s = sigmoid(pre) if silu else np.ones_like(pre)
    y = np.where(live, (apre * ((1 + apre) if silu else 1) if absolute else pre) * s, 0)
    last = np.stack([rows[i, k:k + W - 1] for i, k in enumerate(n)])
    if dy is None:
        return y, last
    slope = s * (1 + pre * (1 - s)) if silu else np.ones_like(pre)
    if absolute and silu:
        slope = s * (1 + apre) ** 2
    dpre = np.where(live, f(_np(dy)) * slope, 0)
    drows = np.zeros_like(rows)
    for j in range(W):
        drows[:, j:j + N] += dpre * f(w[:, j])
    if dstate_out is not None:
        for i, k in enumerate(n):
            drows[i, k:k + W - 1] += f(_np(dstate_out)[i])
    dw = np.stack([(dpre * f(rows[:, j:j + N])).sum((0, 1)) for j in range(W)], 1)
    return y, last, np.where(live, drows[:, W - 1:], 0), dw, dpre.sum((0, 1)), drows[:, :W - 1]


def close(name, got, ref, half, slack):
    """got (a tensor) is ref but for a rounding of `half` relative and `slack`, a number or an array; and for what fp32 has no
    digits for: a decay below 2^-126 is 0, and what it multiplies is below 2^16 in these tests."""
    slack = slack + 2.0 ** -110
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not got.size:
        return
    assert np.isfinite(got).all(), name
    over = np.abs(got - ref) - half * (np.abs(ref) + slack) - slack
    worst = float(over.max())
    assert worst <= 0, "%s: off by %.3g more than its bound of %.3g" % (
        name, worst, float((half * (np.abs(ref) + slack) + slack + 0 * ref).flat[int(over.argmax())]))


def half_step(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


def rand(gen, *shape, scale=1.0, dtype=None):
    import torch
    return (scale * torch.randn(shape, generator=gen)).to(dtype or torch.float32)


def scan_inputs(B, N, D, S, G, dtype, seed, lead=None):
    """u, dt, A, b, c, d_skip, z, dt_bias on the CPU: steps in 0.001 .. 0.5, decay rates around -1 .. -S."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    lead = (B, N) if lead is None else lead
    u, dt, z = (rand(gen, *lead, D, dtype=dtype) for _ in range(3))
    b, c = (rand(gen, *lead, G, S, dtype=dtype) for _ in range(2))
    A = -torch.arange(1, S + 1).float() * torch.exp(rand(gen, D, S, scale=0.3))
    bias = torch.empty(D).uniform_(-6.0, -1.5, generator=gen)
    return dict(u=u, dt=dt, A=A, b=b, c=c, d_skip=rand(gen, D), z=z, dt_bias=bias)


def cuda(d):
    return {k: None if v is None else v.cuda() if hasattr(v, "cuda") else v for k, v in d.items()}
