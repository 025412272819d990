"""The gated delta rule token by token in 64 bits (numpy), forward and gradients, and the inputs of its tests."""
import numpy as np


def forward(q, k, v, g, beta, scale, state=None, lengths=None):
    """q, k [B,N,Hk,dk], v [B,N,H,dv], g, beta [B,N,H] -> o [B,N,H,dv], state [B,H,dk,dv], states before each token."""
    B, N, Hk, dk = q.shape
    H, dv = v.shape[2:]
    rep = H // Hk
    S = np.zeros((B, H, dk, dv)) if state is None else state.astype(np.float64).copy()
    o, before = np.zeros((B, N, H, dv)), []
    for t in range(N):
        before.append(S)
        live = np.ones(B, bool) if lengths is None else t < lengths
        qt, kt = (np.repeat(x[:, t].astype(np.float64), rep, axis=1) for x in (q, k))
        Sa = S * np.exp(g[:, t].astype(np.float64))[..., None, None]
        e = v[:, t].astype(np.float64) - np.einsum("bhk,bhkv->bhv", kt, Sa)
        u = beta[:, t].astype(np.float64)[..., None] * e
        S1 = Sa + kt[..., None] * u[:, :, None, :]
        o[live, t] = scale * np.einsum("bhk,bhkv->bhv", qt, S1)[live]
        S = np.where(live[:, None, None, None], S1, S)
    return o, S, before


def term_sums(q, k, v, g, beta, scale, before):
    """Sums of magnitudes behind each output when it is computed from the state entering its chunk of 64 tokens and the
    chunk's residuals R = V - exp(G) K S0: scale exp(G_i) sum_d |q_id S0_dc| + sum_j |(P T)_ij R_jc|."""
    B, N, Hk, dk = q.shape
    H, dv = v.shape[2:]
    rep = H // Hk
    out = np.zeros((B, N, H, dv))
    for c in range(0, N, 64):
        e = min(c + 64, N)
        S0 = before[c]
        qc, kc = (np.repeat(x[:, c:e].astype(np.float64), rep, axis=2).transpose(0, 2, 1, 3) for x in (q, k))
        vc = v[:, c:e].astype(np.float64).transpose(0, 2, 1, 3)
        G = np.cumsum(g[:, c:e].astype(np.float64), 1).transpose(0, 2, 1)
        be = beta[:, c:e].astype(np.float64).transpose(0, 2, 1)
        low = np.tril(np.ones((e - c, e - c)))
        D = np.exp((G[..., :, None] - G[..., None, :]) * low) * low * be[..., None, :]
        A = np.einsum("bhid,bhjd->bhij", kc, kc) * D * np.tril(np.ones_like(low), -1)
        T = np.linalg.inv(np.eye(e - c) + A)
        PT = np.matmul(scale * np.einsum("bhid,bhjd->bhij", qc, kc) * D, T)
        R = vc - np.exp(G)[..., None] * np.matmul(kc, S0)
        m = scale * np.exp(G)[..., None] * np.matmul(np.abs(qc), np.abs(S0)) + np.matmul(np.abs(PT), np.abs(R))
        out[:, c:e] = m.transpose(0, 2, 1, 3)
    return out


def gradients(q, k, v, g, beta, scale, dout, state=None, dstate_out=None, lengths=None):
    """Gradients of sum(dout o) + sum(dstate_out state): dq, dk, dv, dg, dbeta, dstate_in."""
    B, N, Hk, dk = q.shape
    H, dv = v.shape[2:]
    rep = H // Hk
    _, _, before = forward(q, k, v, g, beta, scale, state, lengths)
    dS = np.zeros((B, H, dk, dv)) if dstate_out is None else dstate_out.astype(np.float64).copy()
    dq, dkk = np.zeros((B, N, H, dk)), np.zeros((B, N, H, dk))
    dvv, dg, db = np.zeros((B, N, H, dv)), np.zeros((B, N, H)), np.zeros((B, N, H))
    for t in reversed(range(N)):
        live = (np.ones(B, bool) if lengths is None else t < lengths)
        m = live[:, None, None]
        qt, kt = (np.repeat(x[:, t].astype(np.float64), rep, axis=1) for x in (q, k))
        al, be = np.exp(g[:, t].astype(np.float64)), beta[:, t].astype(np.float64)
        Sa = before[t] * al[..., None, None]
        e = v[:, t].astype(np.float64) - np.einsum("bhk,bhkv->bhv", kt, Sa)
        u = be[..., None] * e
        S1 = Sa + kt[..., None] * u[:, :, None, :]
        d = dout[:, t].astype(np.float64)
        D = dS + scale * qt[..., None] * d[:, :, None, :]
        du = np.einsum("bhk,bhkv->bhv", kt, D)
        dw = -be[..., None] * du
        with np.errstate(invalid="ignore"):
            dq[:, t] = np.where(m, scale * np.einsum("bhkv,bhv->bhk", S1, d), 0)
            dkk[:, t] = np.where(m, np.einsum("bhkv,bhv->bhk", D, u) + np.einsum("bhkv,bhv->bhk", Sa, dw), 0)
            dvv[:, t] = np.where(m, -dw, 0)
            db[:, t] = np.where(live[:, None], (du * e).sum(-1), 0)
            D = D + kt[..., None] * dw[:, :, None, :]
            dg[:, t] = np.where(live[:, None], (D * Sa).sum((-1, -2)), 0)
            dS = np.where(live[:, None, None, None], D * al[..., None, None], dS)
    fold = lambda x: x.reshape(B, N, Hk, rep, dk).sum(3)  # noqa: E731
    return fold(dq), fold(dkk), dvv, dg, db, dS


def inputs(seed, B, N, H, Hk, dk, dv, dtype, gates="f32", strong=False):
    """torch CPU tensors: keys of unit length that lean one way, decays from weak to strong, writes in (0, 1)."""
    import torch
    t = {"f32": torch.float32, "bf16": torch.bfloat16}
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = (unit(torch.nn.functional.silu(rn(B, N, Hk, dk))).to(t[dtype]) for _ in range(2))
    x = dict(q=q, k=k, v=rn(B, N, H, dv).to(t[dtype]))
    x["g"] = (-torch.exp(rn(B, N, H) * 0.5 + torch.linspace(-6, 1.5 if strong else -1, H))).to(t[gates])
    x["beta"] = torch.sigmoid(rn(B, N, H)).to(t[gates])
    return x


def np64(t):
    return None if t is None else t.double().numpy()
