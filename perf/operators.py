"""Measured cases of the gated linear recurrence and of the norms around a block.

Each case names an operator, its sizes and its options.  `run` computes one
pass, either in plain torch operations or through the package's own entry
points, and returns the same outputs in the same order either way.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one generated token for 4 sequences of a 16-head layer: latency counts
        dict(name="step 4 sequences", op="step", B=4, H=16, N=1, d=64, dtype="bf16", gate="dt", value="complement",
             layout="heads", carried=True, ragged=False),
        # one generated token for a full serving batch of a 32-head layer
        dict(name="step 256 sequences", op="step", B=256, H=32, N=1, d=64, dtype="bf16", gate="dt", value="dt",
             layout="heads", carried=True, ragged=False),
        # the small fp32 workload of the operator tests, as a chunk of a prompt that continues a state
        dict(name="recurrence fp32 256", op="recurrence", B=1, H=2, N=256, d=16, dtype="f32", gate="dt", value="dt",
             layout="heads", carried=True, ragged=False),
        # the 2K workload, gate and values read in place from one fused projection [B, N, 2, H, d]
        dict(name="recurrence 2k", op="recurrence", B=4, H=16, N=2048, d=64, dtype="bf16", gate="dt", value="complement",
             layout="tokens", carried=False, ragged=False),
        # the 64K workload, with the log-decay of the Mamba-2S form given
        dict(name="recurrence 64k", op="recurrence", B=1, H=32, N=65536, d=64, dtype="bf16", gate="log", value="none",
             layout="heads", carried=False, ragged=False),
        # a training step on a padded batch of odd length
        dict(name="recurrence train ragged", op="recurrence_train", B=7, H=12, N=2047, d=32, dtype="bf16", gate="dt",
             value="complement", layout="heads", carried=True, ragged=True),
        # a training step of the 16K workload: few channels, long sequences
        dict(name="recurrence train 16k", op="recurrence_train", B=2, H=8, N=16384, d=64, dtype="bf16", gate="dt",
             value="dt", layout="tokens", carried=False, ragged=False),
        # residual add and norm of 8 sequences' tokens in generation
        dict(name="residual norm 8 rows", op="residual_norm", M=8, C=1024, dtype="bf16", stream="bf16", scale=True),
        # the same in a training step over the 2K workload's tokens
        dict(name="residual norm train 8k", op="residual_norm_train", M=8192, C=1024, dtype="bf16", stream="bf16",
             scale=True),
        # a 64K prompt with the residual stream kept in fp32
        dict(name="residual norm 64k", op="residual_norm", M=65536, C=2048, dtype="bf16", stream="f32", scale=False),
        # the gated norm behind the 64K workload's operator: head layout in, token layout out
        dict(name="gated norm 64k", op="gated_norm", B=1, H=32, N=65536, d=64, dtype="bf16", groups=1, after=False),
        # a training step of the gated norm per head over the 4K workload
        dict(name="gated norm train 4k", op="gated_norm_train", B=4, H=16, N=4096, d=32, dtype="bf16", groups=16,
             after=True),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["step", "recurrence", "recurrence_train", "residual_norm", "residual_norm_train", "gated_norm",
                     "gated_norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("residual"):
        C = rng.choice([_log_int(rng, 64, 8192), 8 * _log_int(rng, 8, 1024)])
        M = _log_int(rng, 1, max(1, min(65536, (1 << (25 if op.endswith("train") else 26)) // C)))
        return dict(op=op, M=M, C=C, dtype=dtype, stream=rng.choice([dtype, "f32"]), scale=rng.random() < 0.5)
    B, H = _log_int(rng, 1, 16), _log_int(rng, 1, 32)
    d = rng.choice([16, 32, 64, 64, 8 * _log_int(rng, 1, 16), _log_int(rng, 5, 130)])
    most = 1 << (24 if op.endswith("train") else 25)
    N = _log_int(rng, 1, max(1, min(65536, most // (B * H * d))))
    if op.startswith("gated_norm"):
        groups = rng.choice([1, H])
        return dict(op=op, B=B, H=H, N=N, d=d, dtype=dtype, groups=groups, after=rng.random() < 0.5)
    if op == "step":
        B, N = _log_int(rng, 1, 256), 1
    gate = rng.choice(["dt", "dt", "log"])
    value = rng.choice(["none", "complement"] + (["dt"] if gate == "dt" else []))
    return dict(op=op, B=B, H=H, N=N, d=d, dtype=dtype, gate=gate, value=value, layout=rng.choice(["heads", "tokens"]),
                carried=op == "step" or rng.random() < 0.5, ragged=op != "step" and B > 1 and rng.random() < 0.3)


def _lengths(case):
    """Valid tokens of each sequence of a padded batch: from N down to N / B."""
    return [case["N"] * (case["B"] - b) // case["B"] for b in range(case["B"])]


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op.startswith("residual"):
        M, C, s = case["M"], case["C"], 4 if case["stream"] == "f32" else 2
        n = M * C
        bytes_ = n * (2 * e + 2 * s) + C * 8
        flops = 7 * n
        if op.endswith("train"):
            # dy, the stream's gradient in and out, and x's gradient besides
            bytes_ += n * (2 * e + 2 * s) + C * 8
            flops = 24 * n
        return {"bytes": bytes_, "flops": flops}
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    n = B * H * N * d
    if op.startswith("gated_norm"):
        return {"bytes": n * e * (6 if op.endswith("train") else 3) + 4 * H * d * (2 if op.endswith("train") else 1),
                "flops": n * (30 if op.endswith("train") else 10)}
    if op == "step":
        return {"bytes": n * (3 * e + 8) + 8 * H * d, "flops": 12 * n}
    valid = sum(_lengths(case)) * H * d if case["ragged"] else n
    state = 4 * B * H * d * (2 if case["carried"] else 1)
    if op == "recurrence":
        return {"bytes": e * (2 * valid + n) + state + 8 * H * d, "flops": 12 * valid}
    return {"bytes": e * (3 * valid + 3 * n) + 2 * state + 16 * H * d, "flops": 40 * valid}


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std + mean).to(dtype)


def _silu(x):
    return x * torch.sigmoid(x)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    op = case["op"]
    if op.startswith("residual"):
        M, C = case["M"], case["C"]
        stream = DTYPES[case["stream"]]
        s["x"] = _normal(gen, (M, C), dtype)
        s["residual"] = _normal(gen, (M, C), stream, 2.0)
        s["scale"] = _normal(gen, (C,), std=0.02, mean=0.3) if case["scale"] else None
        s["w"] = _normal(gen, (C,), std=0.1, mean=1.0)
        if op.endswith("train"):
            s["dy"] = _normal(gen, (M, C), dtype)
            s["dstream"] = _normal(gen, (M, C), stream)
        return s
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    if op.startswith("gated_norm"):
        s["x"] = _normal(gen, (B, H, N, d), dtype)
        s["z"] = _normal(gen, (B, N, H * d), dtype)
        s["w"] = _normal(gen, (H * d,), std=0.1, mean=1.0)
        if op.endswith("train"):
            s["dy"] = _normal(gen, (B, N, H * d), dtype)
        return s

    if op == "step":
        x, gate = _normal(gen, (B, H, d)), _normal(gen, (B, H, d))
    else:
        x, gate = _normal(gen, (B, H, N, d)), _normal(gen, (B, H, N, d))
    x = _silu(x).to(dtype)
    if case["gate"] == "log":
        # the per-token log-decay -softplus(z), z ~ N(-2, 1)
        gate = -torch.nn.functional.softplus(gate - 2.0)
    gate = gate.to(dtype)
    if case["layout"] == "tokens" and op != "step":
        both = torch.stack([x.permute(0, 2, 1, 3), gate.permute(0, 2, 1, 3)], dim=2)  # [B, N, 2, H, d]
        x, gate = both[:, :, 0].permute(0, 2, 1, 3), both[:, :, 1].permute(0, 2, 1, 3)
    s["x"], s["gate"] = x, gate
    s["A_log"] = s["dt_bias"] = None
    if case["gate"] == "dt":
        u = torch.rand((2, H * d), generator=gen, device="cuda")
        s["A_log"] = torch.log(1.0 + 15.0 * u[0])
        dt = torch.exp(math.log(1e-3) + u[1] * (math.log(1e-1) - math.log(1e-3)))
        s["dt_bias"] = dt + torch.log(-torch.expm1(-dt))
    if op == "step":
        s["h"] = _normal(gen, (B, H, d))
        return s
    s["h0"] = _normal(gen, (B, H, d)) if case["carried"] else None
    s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
    if op == "recurrence_train":
        s["dy"] = _normal(gen, (B, H, N, d), dtype)
        s["dh"] = _normal(gen, (B, H, d)) if case["carried"] else None
    return s


# -------------------------------------------------------- the plain forms
def _per_channel(p, H, d):
    return p.view(1, H, 1, d)


def _gates(s, x, gate, H, d):
    """(decay a, value factor f, dt, log a, pre-activation) of every token."""
    c = s["case"]
    if c["gate"] == "log":
        dt = p = None
        la = gate.float()
    else:
        p = gate.float() + _per_channel(s["dt_bias"], H, d)
        dt = torch.clamp(p, min=0) + torch.log1p(torch.exp(-p.abs()))
        la = -torch.exp(_per_channel(s["A_log"], H, d)) * dt
    a = torch.exp(la)
    f = dt if c["value"] == "dt" else -torch.expm1(la) if c["value"] == "complement" else torch.ones_like(a)
    return a, f, dt, la, p


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 2 by doubling the span of each partial result."""
    a, h, span = a.clone(), u.clone(), 1
    while span < h.shape[2]:
        h[:, :, span:] = h[:, :, span:] + a[:, :, span:] * h[:, :, :-span]
        a[:, :, span:] = a[:, :, span:] * a[:, :, :-span]
        span *= 2
    return h


def _masked(s, a, u):
    """Tokens behind a sequence's length leave the state as it is."""
    if s["lengths"] is None:
        return a, u, None
    N = a.shape[2]
    live = (torch.arange(N, device=a.device)[None, :] < s["lengths"][:, None]).view(-1, 1, N, 1)
    return torch.where(live, a, 1.0), torch.where(live, u, 0.0), live


def _plain_recurrence(s):
    c = s["case"]
    x, H, d = s["x"], c["H"], c["d"]
    a, f, dt, la, p = _gates(s, x, s["gate"], H, d)
    a, u, live = _masked(s, a, f * x.float())
    if s["h0"] is not None:
        u[:, :, 0] = u[:, :, 0] + a[:, :, 0] * s["h0"]
    h = _scan(a, u)
    h_out = h[:, :, -1].clone()
    y = (h if live is None else torch.where(live, h, 0.0)).to(x.dtype)
    if c["op"] == "recurrence":
        return [y, h_out]
    dy = s["dy"].float()
    if live is not None:
        dy = torch.where(live, dy, 0.0)
    if s["dh"] is not None:
        dy = dy.clone()
        dy[:, :, -1] = dy[:, :, -1] + s["dh"]
    after = torch.cat([a[:, :, 1:], torch.zeros_like(a[:, :, :1])], dim=2)
    lam = _scan(after.flip(2), dy.flip(2)).flip(2)
    h0 = torch.zeros_like(h_out) if s["h0"] is None else s["h0"]
    before = torch.cat([h0[:, :, None], h[:, :, :-1]], dim=2)
    dh0 = a[:, :, 0] * lam[:, :, 0]
    dx = f * lam
    df = lam * x.float()
    dla = a * lam * before
    if c["value"] == "complement":
        dla = dla - a * df
    if c["gate"] == "log":
        dgate, sums = dla, []
    else:
        rate = torch.exp(_per_channel(s["A_log"], H, d))
        ds = -rate * dla
        if c["value"] == "dt":
            ds = ds + df
        dgate = ds * torch.sigmoid(p)
        dA = dla * la
        if live is not None:
            dgate, dA = torch.where(live, dgate, 0.0), torch.where(live, dA, 0.0)
        sums = [dA.sum(dim=(0, 2)).reshape(-1), dgate.sum(dim=(0, 2)).reshape(-1)]
    if live is not None:
        dx, dgate = torch.where(live, dx, 0.0), torch.where(live, dgate, 0.0)
    return [y, h_out, dx.to(x.dtype), dgate.to(x.dtype), dh0] + sums


def _plain_step(s):
    c = s["case"]
    x = s["x"][:, :, None]
    a, f, dt, la, p = _gates(s, x, s["gate"][:, :, None], c["H"], c["d"])
    s["h"].copy_((a * s["h"][:, :, None] + f * x.float())[:, :, 0])  # in place: the next token continues it
    return [s["h"].to(x.dtype), s["h"]]


def _plain_residual_norm(s):
    c = s["case"]
    x, w = s["x"].float(), s["w"]
    branch = x if s["scale"] is None else s["scale"] * x
    # the stream is kept in its own type, and the norm is of what is kept
    r = (s["residual"].float() + branch).to(s["residual"].dtype)
    rf = r.float()
    rstd = torch.rsqrt((rf * rf).mean(dim=1, keepdim=True) + EPS)
    xhat = rf * rstd
    y = (xhat * w).to(s["x"].dtype)
    if c["op"] == "residual_norm":
        return [y, r]
    dy = s["dy"].float()
    gw = dy * w
    dr = rstd * (gw - xhat * (gw * xhat).mean(dim=1, keepdim=True)) + s["dstream"].float()
    dw = (dy * xhat).sum(dim=0)
    out = [y, r, dr.to(s["residual"].dtype), (dr if s["scale"] is None else dr * s["scale"]).to(s["x"].dtype), dw]
    return out if s["scale"] is None else out + [(dr * x).sum(dim=0)]


def _plain_gated_norm(s):
    c = s["case"]
    B, H, N, d, G = c["B"], c["H"], c["N"], c["d"], c["groups"]
    x = s["x"].float().permute(0, 2, 1, 3).reshape(B, N, G, -1)
    z = s["z"].float().view(B, N, G, -1)
    w = s["w"].view(G, -1)
    sig = torch.sigmoid(z)
    silu = z * sig
    u = x if c["after"] else x * silu
    rstd = torch.rsqrt((u * u).mean(dim=3, keepdim=True) + EPS)
    xhat = u * rstd
    n = xhat * w
    y = (n * silu if c["after"] else n).reshape(B, N, H * d).to(s["x"].dtype)
    if c["op"] == "gated_norm":
        return [y]
    dy = s["dy"].float().view(B, N, G, -1)
    dn = dy * silu if c["after"] else dy
    gw = dn * w
    du = rstd * (gw - xhat * (gw * xhat).mean(dim=3, keepdim=True))
    dsilu = dy * n if c["after"] else du * x
    dx = du if c["after"] else du * silu
    dz = dsilu * sig * (1.0 + z * (1.0 - sig))
    dw = (dn * xhat).sum(dim=(0, 1)).reshape(-1)
    dx = dx.reshape(B, N, H, d).permute(0, 2, 1, 3).contiguous()
    return [y, dx.to(s["x"].dtype), dz.reshape(B, N, H * d).to(s["x"].dtype), dw]


# ------------------------------------------------- the package's own calls
def _own(s):
    import mamba_ssd_sequence_b200 as ssd

    c = s["case"]
    op = c["op"]
    if op.startswith("residual"):
        y, r, rstd = ssd.ssd_add_norm(s["x"], s["residual"], s["scale"], s["w"], eps=EPS)
        if op == "residual_norm":
            return [y, r]
        dr, dx, dw, dscale = ssd.ssd_add_norm_bwd(s["dy"], r, rstd, s["w"], x=s["x"], scale=s["scale"],
                                                  dres=s["dstream"])
        return [y, r, dr, dx, dw] + ([] if dscale is None else [dscale])
    if op.startswith("gated_norm"):
        y, rstd = ssd.ssd_gated_norm(s["x"], s["z"], s["w"], groups=c["groups"], eps=EPS, gate_after=c["after"])
        if op == "gated_norm":
            return [y]
        dx, dz, dw = ssd.ssd_gated_norm_bwd(s["dy"], s["x"], rstd, s["z"], s["w"], groups=c["groups"],
                                            gate_after=c["after"])
        return [y, dx, dz, dw]
    kind = dict(value_dt=c["value"] == "dt", value_complement=c["value"] == "complement")
    dt_p, log_decay = (s["gate"], None) if c["gate"] == "dt" else (None, s["gate"])
    if op == "step":
        y = ssd.ssd_glr_step(s["x"], dt_p, s["A_log"], s["dt_bias"], s["h"], log_decay=log_decay, **kind)
        return [y, s["h"]]
    B, H, N, d = s["x"].shape
    h_out = torch.empty((B, H, d), dtype=torch.float32, device="cuda")
    if op == "recurrence":
        y = ssd.ssd_glr_fwd(s["x"], dt_p, s["A_log"], s["dt_bias"], log_decay=log_decay, h0=s["h0"], h_out=h_out,
                            lengths=s["lengths"], **kind)
        return [y, h_out]
    states = ssd.alloc_glr_states(B, H, N, d)
    y = ssd.ssd_glr_fwd(s["x"], dt_p, s["A_log"], s["dt_bias"], log_decay=log_decay, h0=s["h0"], h_out=h_out,
                        states=states, lengths=s["lengths"], **kind)
    dx, dgate, dA_log, ddt_bias, dh0 = ssd.ssd_glr_bwd(
        s["dy"], s["x"], dt_p, s["A_log"], s["dt_bias"], states, log_decay=log_decay, lengths=s["lengths"],
        dh_out=s["dh"], **kind)
    return [y, h_out, dx, dgate, dh0] + ([] if dA_log is None else [dA_log, ddt_bias])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op.startswith("residual"):
        return _plain_residual_norm(state)
    if op.startswith("gated_norm"):
        return _plain_gated_norm(state)
    return _plain_step(state) if op == "step" else _plain_recurrence(state)


# ------------------------------------------------ the definition in 64 bits
def _exact_recurrence(s):
    """Token by token, forward for h and backward for its adjoint; the gate's
    derivative is taken by automatic differentiation of its definition."""
    c = s["case"]
    B, H, N, d = c["B"], c["H"], c["N"], c["d"]
    step = c["op"] == "step"
    time_first = (lambda t: t.double()[None]) if step else (lambda t: t.double().permute(2, 0, 1, 3).contiguous())
    x, gate = time_first(s["x"]), time_first(s["gate"]).requires_grad_()
    leaves = [gate]
    if c["gate"] == "log":
        la = gate
    else:
        A_log, bias = (s[k].double().view(H, d).requires_grad_() for k in ("A_log", "dt_bias"))
        leaves += [A_log, bias]
        dt = torch.logaddexp(gate + bias, torch.zeros((), dtype=torch.float64, device="cuda"))
        la = -torch.exp(A_log) * dt
    a = torch.exp(la)
    f = dt if c["value"] == "dt" else -torch.expm1(la) if c["value"] == "complement" else torch.ones_like(a)
    lens = [N] * B if step or not c["ragged"] else _lengths(c)
    live = torch.tensor([[t < n for n in lens] for t in range(N)], device="cuda").view(N, B, 1, 1)
    h = s["h"] if step else s["h0"]
    h = torch.zeros((B, H, d), dtype=torch.float64, device="cuda") if h is None else h.double()
    before = torch.empty((N, B, H, d), dtype=torch.float64, device="cuda")
    y = torch.zeros_like(before)
    ad, ud = torch.where(live, a.detach(), 1.0), torch.where(live, (f * x).detach(), 0.0)
    for t in range(N):
        before[t] = h
        h = torch.addcmul(ud[t], ad[t], h)
        y[t] = h
    if step:
        return [y[0], h]
    y = torch.where(live, y, 0.0)
    heads_first = lambda t: t.permute(1, 2, 0, 3)  # noqa: E731
    if c["op"] == "recurrence":
        return [heads_first(y), h]
    dy = torch.where(live, time_first(s["dy"]), 0.0)
    lam = torch.zeros_like(h) if s["dh"] is None else s["dh"].double()
    adjoint = torch.empty_like(before)
    for t in range(N - 1, -1, -1):
        lam = lam + dy[t]
        adjoint[t] = lam
        lam = lam * ad[t]
    adjoint = torch.where(live, adjoint, 0.0)
    got = torch.autograd.grad([a, f * x] if c["value"] != "none" else [a],
                              leaves, [adjoint * before, adjoint][:2 if c["value"] != "none" else 1])
    dx = adjoint * f.detach()
    return [heads_first(y), h, heads_first(dx), heads_first(got[0]), lam] + [g.reshape(-1) for g in got[1:]]


def _exact_residual_norm(s):
    c = s["case"]
    x, w = s["x"].double().requires_grad_(), s["w"].double().requires_grad_()
    scale = None if s["scale"] is None else s["scale"].double().requires_grad_()
    r = s["residual"].double() + (x if scale is None else scale * x)
    kept = r.detach().to(s["residual"].dtype).double().requires_grad_()
    y = kept / torch.sqrt(kept.pow(2).mean(1, True) + EPS) * w
    if c["op"] == "residual_norm":
        return [y.detach(), kept.detach()]
    dkept, dw = torch.autograd.grad(y, [kept, w], s["dy"].double())
    dr = dkept + s["dstream"].double()
    got = torch.autograd.grad(r, [x] if scale is None else [x, scale], dr)
    return [y.detach(), kept.detach(), dr, got[0], dw] + list(got[1:])


def _exact_gated_norm(s):
    c = s["case"]
    B, H, N, d, G = c["B"], c["H"], c["N"], c["d"], c["groups"]
    x, z, w = (s[k].double().requires_grad_() for k in ("x", "z", "w"))
    tokens = x.transpose(1, 2).reshape(B, N, H * d)
    gate = z / (1.0 + torch.exp(-z))
    u = tokens if c["after"] else tokens * gate
    parts = u.view(B, N, G, H * d // G)
    y = (parts / torch.sqrt(parts.pow(2).mean(-1, True) + EPS)).view(B, N, H * d) * w
    if c["after"]:
        y = y * gate
    if c["op"] == "gated_norm":
        return [y.detach()]
    dx, dz, dw = torch.autograd.grad(y, [x, z, w], s["dy"].double())
    return [y.detach(), dx, dz, dw]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("residual"):
        return _exact_residual_norm(s)
    if case["op"].startswith("gated_norm"):
        return _exact_gated_norm(s)
    return _exact_recurrence(s)
