"""The operators of a pre-norm gated-delta block, as they are measured: the gated delta rule over a sequence (forward
and gradients) and for single tokens, layer norm over a residual stream (forward and gradients), and the gradients of
the multi-scale retention epilogue.

Each case names one operator ("op") and its sizes. prepare() makes what a program holds before the call, run() makes
one pass: where `own` is false in elementary torch operations, where it is true by the library's entry points.
exact() computes the same outputs in 64 bits from the definitions, token by token.

The gated delta rule: per batch b and head h, with state S (d_k x d_v), decay alpha_t = exp(g_t) and write strength
beta_t,
    S'_t = alpha_t S_{t-1},  u_t = beta_t (v_t - S'_t^T k_t),  S_t = S'_t + k_t u_t^T,  o_t = scale S_t^T q_t.
q and k may have fewer heads than v: value head h reads key head h // (H / Hk). `lengths` gives the tokens of each
sequence of a padded batch; outputs of the padding are zero.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    d = dict
    return [
        # the smallest prefill: 64 tokens of an 8-head layer in fp32, where launches count
        d(name="delta-fwd-tiny-f32", op="delta_fwd", B=1, N=64, H=8, Hk=8, dk=16, dv=16, dtype="f32", gates="f32",
          state=True, ragged=False),
        # prefill of a padded batch, grouped key heads, the heads of a d_model = 4096 layer; the state goes to decode
        d(name="delta-fwd-ragged-d256", op="delta_fwd", B=3, N=2741, H=16, Hk=8, dk=256, dv=512, dtype="bf16",
          gates="f32", state=True, ragged=True),
        # one long sequence: few heads, 65536 tokens, so the sequence itself has to be split
        d(name="delta-fwd-long", op="delta_fwd", B=1, N=65536, H=8, Hk=8, dk=128, dv=128, dtype="bf16", gates="f32",
          state=True, ragged=False),
        # gradients in fp32 at an odd length, grouped key heads, gradients of the states
        d(name="delta-bwd-odd-f32", op="delta_bwd", B=2, N=333, H=6, Hk=2, dk=32, dv=48, dtype="f32", gates="f32",
          state=True, ragged=True),
        # the training step of a d_model = 4096 layer over 8192 tokens
        d(name="delta-bwd-d256", op="delta_bwd", B=1, N=8192, H=16, Hk=16, dk=256, dv=512, dtype="bf16",
          gates="bf16", state=False, ragged=False),
        # one token for one sequence: latency
        d(name="delta-step-one", op="delta_step", B=1, H=8, Hk=8, dk=64, dv=64, dtype="bf16", gates="f32"),
        # one token for each sequence of a batch: the state is read and written once
        d(name="delta-step-batch", op="delta_step", B=128, H=16, Hk=8, dk=128, dv=256, dtype="bf16", gates="f32"),
        # pre-norm of one token per sequence with the residual added, d_model = 4096
        d(name="norm-fwd-decode", op="norm_fwd", rows=128, D=4096, dtype="bf16", residual=True, affine=True),
        # pre-norm of a training batch of an odd width in fp32
        d(name="norm-fwd-odd-f32", op="norm_fwd", rows=16384, D=1001, dtype="f32", residual=False, affine=True),
        # its gradients over 8192 tokens of a d_model = 4096 layer, with the residual stream's gradient
        d(name="norm-bwd-d4096", op="norm_bwd", rows=8192, D=4096, dtype="bf16", residual=True, affine=True),
        # gradients of GroupNorm and gate, d_model = 512 layer: 8 x 2048 tokens
        d(name="epilogue-bwd-d64", op="epi_bwd", rows=16384, H=8, dv=64, dtype="bf16", gate=True, affine=True),
        # the same of the widest heads
        d(name="epilogue-bwd-d512", op="epi_bwd", rows=8192, H=16, dv=512, dtype="bf16", gate=True, affine=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_bwd", "delta_step", "norm_fwd", "norm_bwd",
                     "epi_bwd"])
    f32 = rng.random() < 0.3
    dtype = "f32" if f32 else "bf16"
    if op in ("norm_fwd", "norm_bwd"):
        D = rng.choice([_log_int(rng, 32, 8192), 8 * _log_int(rng, 4, 1024)])
        rows = _log_int(rng, 1, max(2, min(32768, (1 << 25) // D)))
        return dict(op=op, rows=rows, D=D, dtype=dtype, residual=rng.random() < 0.5, affine=rng.random() < 0.8)
    if op == "epi_bwd":
        dv, H = rng.choice([16, 32, 64, 128, 256, 512]), rng.randint(1, 24)
        rows = _log_int(rng, 1, max(2, min(32768, (1 << 25) // (dv * H))))
        return dict(op=op, rows=rows, H=H, dv=dv, dtype=dtype, gate=rng.random() < 0.8, affine=rng.random() < 0.8)
    Hk = rng.randint(1, 12)
    H = Hk * rng.choice([1, 1, 2, 4])
    dk = rng.choice([16, 32, 64, 128] if f32 else [32, 64, 128, 256])
    dv = 16 * _log_int(rng, 1, 8 if f32 else 32)
    if op == "delta_step":
        B = _log_int(rng, 1, max(2, min(512, (1 << 26) // (H * dk * dv))))
        return dict(op=op, B=B, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, gates="f32")
    # tokens such that neither the state products nor the tensors pass those of the largest listed case
    most = (1 << 33 if f32 else 1 << 34) // (dk * dv * H)
    most = max(64, min(most, (1 << 27) // (H * (dk + dv))))
    N = min(_log_int(rng, 1, min(most, 65536 if op == "delta_fwd" else 8192)), most)
    B = max(1, min(rng.randint(1, 6), most // N))
    gates = "f32" if f32 else ("bf16" if op == "delta_bwd" else rng.choice(["f32", "bf16"]))
    return dict(op=op, B=B, N=N, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, gates=gates, state=rng.random() < 0.5,
                ragged=B > 1 and rng.random() < 0.5)


def work(case):
    c, e = case, _SIZE[case["dtype"]]
    if c["op"] == "norm_fwd":
        n = c["rows"] * c["D"]
        return {"bytes": n * e * (4 if c["residual"] else 2) + 8 * c["rows"] + 8 * c["D"] * c["affine"], "flops": 8 * n}
    if c["op"] == "norm_bwd":
        n = c["rows"] * c["D"]
        return {"bytes": n * e * (4 if c["residual"] else 3) + 8 * c["rows"] + 12 * c["D"] * c["affine"],
                "flops": 14 * n}
    if c["op"] == "epi_bwd":
        n = c["rows"] * c["H"] * c["dv"]
        return {"bytes": n * e * (5 if c["gate"] else 3) + 16 * c["H"] * c["dv"] * c["affine"], "flops": 24 * n}
    B, H, Hk, dk, dv = c["B"], c["H"], c["Hk"], c["dk"], c["dv"]
    ge = _SIZE[c["gates"]]
    if c["op"] == "delta_step":
        return {"bytes": B * (2 * Hk * dk * e + 2 * H * dv * e + 2 * H * ge + 8 * H * dk * dv),
                "flops": 7 * B * H * dk * dv}
    T = B * c["N"]
    states = 4 * B * H * dk * dv
    if c["op"] == "delta_fwd":
        return {"bytes": T * (2 * Hk * dk * e + 2 * H * dv * e + 2 * H * ge) + states * (2 if c["state"] else 0),
                "flops": 6 * T * H * dk * dv}
    return {"bytes": T * (4 * Hk * dk * e + 3 * H * dv * e + 4 * H * ge) + states * (3 if c["state"] else 0),
            "flops": 18 * T * H * dk * dv}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _silu(x):
    return x / (1 + torch.exp(-x))


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6)


def _delta_inputs(c, g, lead):
    """q, k of unit length from a SiLU (so keys of one head lean the same way), v, log decays -A dt with A per head in
    (0, 16) and dt per token around a per-head value in 0.001 .. 0.1, write strengths in (0, 1)."""
    H, Hk, t = c["H"], c["Hk"], _DT[c["dtype"]]
    gt = _DT[c["gates"]]
    s = {"q": _unit(_silu(_normal(g, *lead, Hk, c["dk"]))).to(t), "k": _unit(_silu(_normal(g, *lead, Hk, c["dk"]))).to(t),
         "v": _normal(g, *lead, H, c["dv"]).to(t), "beta": torch.sigmoid(_normal(g, *lead, H)).to(gt)}
    A = 16 * torch.rand((H,), generator=g, device="cuda")
    dt = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand((H,), generator=g, device="cuda"))
    s["g"] = (-A * dt * torch.exp(0.5 * _normal(g, *lead, H))).to(gt)
    return s


def prepare(case, seed):
    c, g = case, _gen(seed)
    t = _DT[c["dtype"]]
    s = {"case": dict(c)}
    if c["op"] in ("norm_fwd", "norm_bwd"):
        rows, D = c["rows"], c["D"]
        s["x"] = (1.5 * _normal(g, rows, D) + 0.3 * _normal(g, rows, 1)).to(t)
        if c["affine"]:
            s["w"], s["b"] = 1 + 0.1 * _normal(g, D), 0.1 * _normal(g, D)
        if c["op"] == "norm_fwd":
            if c["residual"]:
                s["res"] = _normal(g, rows, D).to(t)
                s["sum"] = torch.empty_like(s["x"])
            s["y"] = torch.empty_like(s["x"])
            s["mean"], s["rstd"] = (torch.empty((rows,), device="cuda") for _ in range(2))
            return s
        s["dy"] = _normal(g, rows, D).to(t)
        if c["residual"]:
            s["dsum"] = _normal(g, rows, D).to(t)
        x = s["x"].double()
        s["mean"] = x.mean(1).float()
        s["rstd"] = (1 / (x.var(1, unbiased=False) + 1e-5).sqrt()).float()
        s["dx"] = torch.empty_like(s["x"])
        if c["affine"]:
            s["dw"], s["db"] = torch.empty_like(s["w"]), torch.empty_like(s["b"])
        if own:
            from linear_recurrent_sequence_amd import retention as R
            s["ws"] = R.layer_norm_bwd_workspace(s["x"])
        return s
    if c["op"] == "epi_bwd":
        shape = (c["rows"], c["H"], c["dv"])
        s["o"], s["dy"] = (0.7 * _normal(g, *shape) + 0.1).to(t), _normal(g, *shape).to(t)
        s["do"] = torch.empty_like(s["o"])
        if c["gate"]:
            s["gate"] = _normal(g, *shape).to(t)
            s["dgate"] = torch.empty_like(s["gate"])
        if c["affine"]:
            s["w"], s["b"] = 1 + 0.1 * _normal(g, c["H"] * c["dv"]), 0.1 * _normal(g, c["H"] * c["dv"])
            s["dw"], s["db"] = torch.empty_like(s["w"]), torch.empty_like(s["b"])
        if own:
            from linear_recurrent_sequence_amd import retention as R
            s["ws"] = R.msr_epilogue_bwd_workspace(s["o"])
        return s
    B, H, dk, dv = c["B"], c["H"], c["dk"], c["dv"]
    if c["op"] == "delta_step":
        s |= _delta_inputs(c, g, (B,))
        s["state"] = 0.3 * _normal(g, B, H, dk, dv)
        s["o"] = torch.empty_like(s["v"])
        return s
    N = c["N"]
    s |= _delta_inputs(c, g, (B, N))
    s["lengths"] = None
    if c["ragged"]:
        n = torch.randint(0, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[0] = N
        s["lengths"] = n
    if c["state"]:
        s["state_in"] = 0.3 * _normal(g, B, H, dk, dv)
    if c["op"] == "delta_fwd":
        s["o"] = torch.empty_like(s["v"])
        if c["state"]:
            s["state_out"] = torch.empty_like(s["state_in"])
    else:
        s["do"] = _normal(g, B, N, H, dv).to(_DT[c["dtype"]])
        for name in ("q", "k", "v", "g", "beta"):
            s["d" + name] = torch.empty_like(s[name])
        if c["state"]:
            s["dstate_out"] = 0.3 * _normal(g, B, H, dk, dv)
            s["dstate_in"] = torch.empty_like(s["state_in"])
    if own:
        from linear_recurrent_sequence_amd import retention as R
        make = R.gated_delta_workspace if c["op"] == "delta_fwd" else R.gated_delta_bwd_workspace
        s["ws"] = make(s["q"], s["v"])
    return s


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from linear_recurrent_sequence_amd import retention as R
    op = s["case"]["op"]
    if op == "norm_fwd":
        R.ret_layer_norm_fwd(s["x"], s["y"], s.get("w"), s.get("b"), residual=s.get("res"), sum_out=s.get("sum"),
                             mean=s["mean"], rstd=s["rstd"])
        return [s["y"], s.get("sum"), s["mean"], s["rstd"]]
    if op == "norm_bwd":
        R.ret_layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["dx"], weight=s.get("w"), dsum=s.get("dsum"),
                             dweight=s.get("dw"), dbias=s.get("db"), workspace=s["ws"])
        return [s["dx"], s.get("dw"), s.get("db")]
    if op == "epi_bwd":
        R.ret_msr_epilogue_bwd(s["dy"], s["o"], s["do"], gate=s.get("gate"), dgate=s.get("dgate"),
                               gn_weight=s.get("w"), gn_bias=s.get("b"), dweight=s.get("dw"), dbias=s.get("db"),
                               workspace=s["ws"])
        return [s["do"], s.get("dgate"), s.get("dw"), s.get("db")]
    if op == "delta_step":
        R.ret_gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], s["state"])
        return [s["o"], s["state"]]
    if op == "delta_fwd":
        R.ret_gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], lengths=s["lengths"],
                              state_in=s.get("state_in"), state_out=s.get("state_out"), workspace=s["ws"])
        return [s["o"], s.get("state_out")]
    R.ret_gated_delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], s["dq"], s["dk"], s["dv"], s["dg"],
                          s["dbeta"], lengths=s["lengths"], state_in=s.get("state_in"),
                          dstate_out=s.get("dstate_out"), dstate_in=s.get("dstate_in"), workspace=s["ws"])
    return [s["dq"], s["dk"], s["dv"], s["dg"], s["dbeta"], s.get("dstate_in")]


def _run_plain(s):
    op = s["case"]["op"]
    if op == "norm_fwd":
        return _plain_norm_fwd(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "epi_bwd":
        return _plain_epi_bwd(s)
    if op == "delta_step":
        return _plain_step(s)
    return _plain_delta_fwd(s) if op == "delta_fwd" else _plain_delta_bwd(s)


def _plain_norm_fwd(s):
    x, t = s["x"], s["x"].dtype
    total = None
    if "res" in s:
        x = total = (x.float() + s["res"].float()).to(t)
    x = x.float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / (d.square().mean(1) + 1e-5).sqrt()
    y = d * rstd[:, None]
    if "w" in s:
        y = y * s["w"] + s["b"]
    return [y.to(t), total, mean, rstd]


def _plain_norm_bwd(s):
    x, dy, t = s["x"].float(), s["dy"].float(), s["x"].dtype
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    a = dy * s["w"] if "w" in s else dy
    dx = (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    if "dsum" in s:
        dx = dx + s["dsum"].float()
    if "w" not in s:
        return [dx.to(t), None, None]
    return [dx.to(t), (dy * xh).sum(0), dy.sum(0)]


def _plain_epi_bwd(s):
    o, dy, t = s["o"].float(), s["dy"].float(), s["o"].dtype
    d = o - o.mean(-1, keepdim=True)
    rstd = 1 / (d.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    xh = d * rstd
    H, dv = o.shape[1:]
    w, b = (s["w"].view(H, dv), s["b"].view(H, dv)) if "w" in s else (None, None)
    dn, dgate = dy, None
    if "gate" in s:
        x = s["gate"].float()
        sg = 1 / (1 + torch.exp(-x))
        dn = dy * (x * sg)
        n = xh * w + b if w is not None else xh
        dgate = (dy * n * (sg * (1 + x * (1 - sg)))).to(t)
    a = dn * w if w is not None else dn
    do = (a - a.mean(-1, keepdim=True) - xh * (a * xh).mean(-1, keepdim=True)) * rstd
    if w is None:
        return [do.to(t), dgate, None, None]
    return [do.to(t), dgate, (dn * xh).sum(0).reshape(-1), dn.sum(0).reshape(-1)]


def _plain_step(s):
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(rep, 1) for n in ("q", "k"))
    S = s["state"] * torch.exp(s["g"].float())[..., None, None]
    u = s["beta"].float()[..., None] * (s["v"].float() - (S * k[..., None]).sum(2))
    S = S + k[..., None] * u[:, :, None, :]
    o = (S * q[..., None]).sum(2) * (q.shape[-1] ** -0.5)
    s["state"].copy_(S)
    return [o.to(s["v"].dtype), s["state"]]


_C = 64  # tokens per chunk of the plain form


def _chunks(x, nc):
    """[B, N, H, ...] -> [B, H, nc, 64, ...] in 32 bits, the tail filled with zeros."""
    x = x.float() if x.dtype == torch.bfloat16 else x
    B, N, H = x.shape[:3]
    full = x.new_zeros((B, nc * _C, H) + x.shape[3:])
    full[:, :N] = x
    return full.view((B, nc, _C, H) + x.shape[3:]).permute((0, 3, 1, 2) + tuple(range(4, x.dim() + 1))).contiguous()


def _tokens(x, N):
    """The inverse of _chunks: [B, H, nc, 64, ...] -> [B, N, H, ...]."""
    B, H, nc = x.shape[:3]
    x = x.permute((0, 2, 3, 1) + tuple(range(4, x.dim()))).reshape((B, nc * _C, H) + x.shape[4:])
    return x[:, :N]


def _plain_chunk_terms(s):
    """What both directions need of each chunk: the inputs by chunks (padding as tokens that change nothing), the
    decays, T = (I + A)^-1 of A_ij = beta_i exp(G_i - G_j) k_i.k_j (j < i), P_ij = scale exp(G_i - G_j) q_i.k_j (j <= i)
    and the state entering each chunk."""
    B, N, H, dv = s["v"].shape
    dk, rep, nc = s["q"].shape[-1], H // s["q"].shape[2], -(-N // _C)
    live = None
    if s["lengths"] is not None:
        live = torch.arange(N, device="cuda")[None, :] < s["lengths"][:, None]
    keep = (lambda x: x if live is None else x * live.view(live.shape + (1,) * (x.dim() - 2)))  # noqa: E731
    q, k = (_chunks(keep(s[n]).repeat_interleave(rep, 2), nc) for n in ("q", "k"))
    v, beta = _chunks(keep(s["v"]), nc), _chunks(keep(s["beta"]), nc)
    G = torch.cumsum(_chunks(keep(s["g"]), nc).double(), 3)
    low = torch.ones((_C, _C), device="cuda").tril()
    D = torch.exp(((G[..., :, None] - G[..., None, :]) * low).float()) * low
    kt = k.transpose(-1, -2).contiguous()
    A = beta[..., None] * torch.matmul(k, kt) * D * (1 - torch.eye(_C, device="cuda"))
    T = torch.zeros_like(A)
    for i in range(_C):
        T[..., i, i] = 1
        if i:
            T[..., i, :i] = -torch.matmul(A[..., i:i + 1, :i], T[..., :i, :i])[..., 0, :]
    P = torch.matmul(q, kt) * D * dk ** -0.5
    gam, tail = torch.exp(G.float()), torch.exp((G[..., -1:] - G).float())
    U = torch.matmul(T, beta[..., None] * v)
    W = torch.matmul(T, (beta * gam)[..., None] * k)
    ktail = (tail[..., None] * k).transpose(-1, -2).contiguous()
    S = s["state_in"] if s.get("state_in") is not None else torch.zeros((B, H, dk, dv), device="cuda")
    S0, Ut = torch.empty((B, H, nc, dk, dv), device="cuda"), torch.empty_like(U)
    for c in range(nc):
        S0[:, :, c] = S
        u = U[:, :, c] - torch.matmul(W[:, :, c], S)
        Ut[:, :, c] = u
        S = gam[:, :, c, -1, None, None] * S + torch.matmul(ktail[:, :, c], u)
    return dict(q=q, k=k, kt=kt, v=v, beta=beta, D=D, A=A, T=T, P=P, gam=gam, tail=tail, S0=S0, Ut=Ut, S=S, keep=keep,
                ktail=ktail)


def _plain_delta_fwd(s):
    N, t = s["v"].shape[1], s["v"].dtype
    x = _plain_chunk_terms(s)
    scale = s["q"].shape[-1] ** -0.5
    o = torch.matmul(x["q"] * (scale * x["gam"])[..., None], x["S0"]) + torch.matmul(x["P"], x["Ut"])
    return [x["keep"](_tokens(o, N)).to(t), x["S"] if s.get("state_in") is not None else None]


def _plain_delta_bwd(s):
    B, N, H, dv = s["v"].shape
    Hk, dk = s["q"].shape[2:]
    t, nc, scale = s["v"].dtype, -(-N // _C), dk ** -0.5
    x = _plain_chunk_terms(s)
    q, k, v, beta, gam, tail = (x[n] for n in ("q", "k", "v", "beta", "gam", "tail"))
    do = _chunks(x["keep"](s["do"]), nc)
    tr = lambda m: m.transpose(-1, -2).contiguous()  # noqa: E731
    dU0, Tt = torch.matmul(tr(x["P"]), do), tr(x["T"])
    dQS = torch.matmul(tr(q * (scale * gam)[..., None]), do)
    kb = tr(k * (beta * gam)[..., None])
    dS = s["dstate_out"] if s.get("dstate_out") is not None else torch.zeros((B, H, dk, dv), device="cuda")
    dS1, dR = torch.empty((B, H, nc, dk, dv), device="cuda"), torch.empty_like(do)
    for c in reversed(range(nc)):
        dS1[:, :, c] = dS
        du = dU0[:, :, c] + tail[:, :, c, :, None] * torch.matmul(k[:, :, c], dS)
        dr = torch.matmul(Tt[:, :, c], du)
        dR[:, :, c] = dr
        dS = gam[:, :, c, -1, None, None] * dS + dQS[:, :, c] - torch.matmul(kb[:, :, c], dr)
    S0t, Ut = tr(x["S0"]), x["Ut"]
    Y = torch.matmul(k, x["S0"])
    read = gam[..., None] * Y + torch.matmul(x["A"] / beta.clamp_min(1e-30)[..., None], Ut)
    dbeta = (dR * (v - read)).sum(-1)
    dqs = scale * gam[..., None] * torch.matmul(do, S0t)
    dP, dA = torch.matmul(do, tr(Ut)), -torch.matmul(dR, tr(Ut))
    X = dP * x["D"] * scale
    Z = dA * x["D"] * beta[..., None] * (1 - torch.eye(_C, device="cuda"))
    dq = dqs + torch.matmul(X, k)
    kread = -(beta * gam)[..., None] * torch.matmul(dR, S0t) + torch.matmul(Z, k)
    kwrite = tail[..., None] * torch.matmul(Ut, tr(dS1)) + torch.matmul(tr(X), q) + torch.matmul(tr(Z), k)
    # decays: each row's exp(G_i) stands with q and the read k, each exp(-G_j) with the written k, exp(G_C) with S
    dG = ((q * dq).sum(-1) + (k * kread).sum(-1)).double() - (k * kwrite).sum(-1).double()
    S1 = torch.cat([x["S0"][:, :, 1:], x["S"][:, :, None]], 2)
    dG[..., -1] += (S1 * dS1).sum((-1, -2))
    dg = torch.flip(torch.cumsum(torch.flip(dG, (3,)), 3), (3,))
    fold = lambda m: _tokens(m, N).reshape(B, N, Hk, H // Hk, dk).sum(3)  # noqa: E731
    gt = s["g"].dtype
    keep = x["keep"]
    return [fold(dq).to(t), keep(fold(kread + kwrite)).to(t), keep(_tokens(beta[..., None] * dR, N)).to(t),
            keep(_tokens(dg, N)).to(gt), keep(_tokens(dbeta, N)).to(gt),
            dS if s.get("dstate_out") is not None else None]


# ---------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        x, total = s["x"].double(), None
        if "res" in s:
            total = (x + s["res"].double()).to(s["x"].dtype)
            x = total.double()
        mean, var = x.mean(1), x.var(1, unbiased=False)
        rstd = (var + 1e-5) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None]
        if "w" in s:
            y = y * s["w"].double() + s["b"].double()
        return [y, None if total is None else total.double(), mean, rstd]
    if op == "norm_bwd":
        # y = w xh + b and xh = (x - mean) rstd: dL/dx by the projection that takes out the mean and xh parts
        r = s["rstd"].double()[:, None]
        xh = (s["x"].double() - s["mean"].double()[:, None]) * r
        dy, D = s["dy"].double(), s["x"].shape[1]
        a = dy * s["w"].double() if "w" in s else dy
        dx = r * (a - (a.sum(1, keepdim=True) + xh * (a * xh).sum(1, keepdim=True)) / D)
        if "dsum" in s:
            dx = dx + s["dsum"].double()
        return [dx] + ([(dy * xh).sum(0), dy.sum(0)] if "w" in s else [None, None])
    if op == "epi_bwd":
        leaves = {n: s[n].double().requires_grad_() for n in ("o", "gate", "w", "b") if n in s}
        o = leaves["o"]
        xh = (o - o.mean(-1, keepdim=True)) * (o.var(-1, unbiased=False, keepdim=True) + 1e-5) ** -0.5
        if "w" in s:
            xh = xh * leaves["w"].view(o.shape[1:]) + leaves["b"].view(o.shape[1:])
        if "gate" in s:
            xh = xh * leaves["gate"] * torch.sigmoid(leaves["gate"])
        grads = dict(zip(leaves, torch.autograd.grad(xh, list(leaves.values()), s["dy"].double())))
        return [grads["o"], grads.get("gate"), grads.get("w"), grads.get("b")]
    if op == "delta_step":
        o, S, _ = _token(s, s["state"].double(), *_token_inputs(s, None))
        return [o, S]
    return _exact_fwd(s) if op == "delta_fwd" else _exact_bwd(s)


def _token_inputs(s, t):
    """q, k, v, exp(g), beta of token t (None: the tensors have no token axis) in 64 bits, key heads repeated."""
    pick = (lambda n: s[n].double()) if t is None else (lambda n: s[n][:, t].double())  # noqa: E731
    rep = s["v"].shape[-2] // s["q"].shape[-2]
    return (pick("q").repeat_interleave(rep, 1), pick("k").repeat_interleave(rep, 1), pick("v"),
            torch.exp(pick("g")), pick("beta"))


def _token(s, S, q, k, v, alpha, beta):
    """(o, state after the token, v - S'^T k)."""
    S = S * alpha[..., None, None]
    e = v - torch.matmul(k[:, :, None, :], S)[:, :, 0]
    S = torch.addcmul(S, k[..., None], (beta[..., None] * e)[:, :, None, :])
    return torch.matmul(q[:, :, None, :], S)[:, :, 0] * (q.shape[-1] ** -0.5), S, e


def _exact_inputs(s):
    """All tokens in 64 bits, padding as tokens that change nothing."""
    x = {n: s[n].double() for n in ("q", "k", "v", "g", "beta") if n in s}
    if s["lengths"] is not None:
        live = torch.arange(s["v"].shape[1], device="cuda")[None, :] < s["lengths"][:, None]
        x = {n: y * live.view(live.shape + (1,) * (y.dim() - 2)) for n, y in x.items()}
        x["live"] = live
    return x


def _first_state(s):
    B, _, H, dv = s["v"].shape
    if s.get("state_in") is not None:
        return s["state_in"].double()
    return torch.zeros((B, H, s["q"].shape[-1], dv), device="cuda", dtype=torch.float64)


def _exact_fwd(s):
    x, S = _exact_inputs(s), _first_state(s)
    out = torch.zeros(s["v"].shape, device="cuda", dtype=torch.float64)
    for t in range(s["v"].shape[1]):
        out[:, t], S, _ = _token(s, S, *_token_inputs(x, t))
    if "live" in x:
        out = out * x["live"][..., None, None]
    return [out, S if s.get("state_in") is not None else None]


def _exact_bwd(s):
    x, S = _exact_inputs(s), _first_state(s)
    B, N, H, dv = s["v"].shape
    Hk, dk = s["q"].shape[2:]
    scale, step = dk ** -0.5, 64
    kept = []
    for t in range(N):
        if t % step == 0:
            kept.append(S)
        _, S, _ = _token(s, S, *_token_inputs(x, t))
    f64 = dict(device="cuda", dtype=torch.float64)
    dq, dk_, dv_ = torch.zeros((B, N, H, dk), **f64), torch.zeros((B, N, H, dk), **f64), torch.zeros((B, N, H, dv), **f64)
    dg, db = torch.zeros((B, N, H), **f64), torch.zeros((B, N, H), **f64)
    do = s["do"].double()
    if "live" in x:
        do = do * x["live"][..., None, None]
    dS = s["dstate_out"].double() if s.get("dstate_out") is not None else torch.zeros((B, H, dk, dv), **f64)
    for b in reversed(range(len(kept))):
        S, before = kept[b], []
        for t in range(b * step, min(N, (b + 1) * step)):
            before.append(S)
            _, S, _ = _token(s, S, *_token_inputs(x, t))
        for t in reversed(range(b * step, min(N, (b + 1) * step))):
            q, k, v, alpha, beta = _token_inputs(x, t)
            Sa = before.pop() * alpha[..., None, None]
            e = v - torch.matmul(k[:, :, None, :], Sa)[:, :, 0]
            u = beta[..., None] * e
            S1 = torch.addcmul(Sa, k[..., None], u[:, :, None, :])
            d = do[:, t]
            dq[:, t] = scale * torch.matmul(S1, d[..., None])[..., 0]
            dS = torch.addcmul(dS, scale * q[..., None], d[:, :, None, :])
            du = torch.matmul(k[:, :, None, :], dS)[:, :, 0]
            db[:, t] = (du * e).sum(-1)
            dw = -beta[..., None] * du
            dv_[:, t] = -dw
            dk_[:, t] = torch.matmul(dS, u[..., None])[..., 0] + torch.matmul(Sa, dw[..., None])[..., 0]
            dS = torch.addcmul(dS, k[..., None], dw[:, :, None, :])
            dg[:, t] = (dS * Sa).sum((-1, -2))
            dS = dS * alpha[..., None, None]
    fold = lambda m: m.view(B, N, Hk, H // Hk, dk).sum(3)  # noqa: E731
    grads = [fold(dq), fold(dk_), dv_, dg, db]
    if "live" in x:
        grads = [m * x["live"].view((B, N) + (1,) * (m.dim() - 2)) for m in grads]
    return grads + [dS if s.get("dstate_out") is not None else None]
