"""Plain float64 forms (torch, CPU) of the gated linear recurrence and of the
norms, each with bounds on the error that float32 arithmetic may add.

Bounds count roundings in units of U = 2^-24, the largest relative error of
one float32 rounding.  Of the recurrence, per token:
  log a   softplus (polynomial and hardware base-2 exponential: 5 U), the rate
          exp(A_log) (3 U) and their product (1 U): 9 U relative, so a is off
          by 9 U |log a| relative, and by 3 U from its own evaluation;
  p       gate + dt_bias is rounded once and scaled once inside the exponential,
          so p is off by 2 U |p|, which changes dt by 2 k U relative with
          k = |p| sigmoid(p) / softplus(p) (the logarithmic derivative of the
          softplus times |p|; for p = -14, k = 14), and its slope sigmoid(p)
          by 2 |p| (1 - sigmoid(p)) U relative;
  f       9 U relative for dt; 1 - a = -expm1(log a) is off by at most
          (9 + 3) U relative, since |log a| a / (1 - a) <= 1; f x: 1 U more;
  h       1 U for the multiply-add, 1 U for the running product of decays
          that carries a state over a span of tokens, 1 U where spans join.
The recurrences below carry such bounds along with envelopes (the same sums
of absolute values), so they hold element by element whatever cancels.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def f64(t):
    return None if t is None else t.detach().cpu().double()


def gates(gate, A_log, dt_bias, kind, value):
    """(a, f, log a, dt, d dt / d gate, rate) of [B, H, N, d] gates."""
    B, H, N, d = gate.shape
    if kind == "log":
        la, dt, sg, rate = gate, None, None, None
    else:
        p = gate if dt_bias is None else gate + dt_bias.view(1, H, 1, d)
        dt = torch.logaddexp(p, torch.zeros_like(p))
        dt = torch.where(p == float("-inf"), 0.0, torch.where(p == float("inf"), p, dt))
        sg = torch.sigmoid(p)
        rate = torch.ones(1, H, 1, d, dtype=torch.float64) if A_log is None else torch.exp(A_log.view(1, H, 1, d))
        la = -rate * dt
    a = torch.exp(la)
    f = dt if value == "dt" else -torch.expm1(la) if value == "complement" else torch.ones_like(a)
    return a, f, la, dt, sg, rate


def recurrence(x, gate, A_log=None, dt_bias=None, h0=None, lengths=None, kind="dt", value="none", dy=None,
               dh_out=None):
    """Everything of one forward (and backward, when dy is given) pass in
    float64: a dict of results and, under name + "_tol", of bounds (before the
    rounding of the stored type)."""
    x, gate, A_log, dt_bias, h0, dy, dh_out = (f64(t) for t in (x, gate, A_log, dt_bias, h0, dy, dh_out))
    B, H, N, d = x.shape
    a, f, la, dt, sg, rate = gates(gate, A_log, dt_bias, kind, value)
    lens = torch.full((B,), N) if lengths is None else lengths.cpu().long().clamp(0, N)
    live = (torch.arange(N)[None] < lens[:, None]).view(B, 1, N, 1).expand(B, H, N, d)
    zero = torch.zeros(B, H, d, dtype=torch.float64)
    one = torch.ones((), dtype=torch.float64)
    a = torch.where(live, a, one)
    f, x_ = torch.where(live, f, 0 * one), torch.where(live, x, 0 * one)
    lam_ = torch.where(live, la.clamp(min=-200.0), 0 * one).abs()
    if kind == "log":
        k2, s2 = 0 * one, 0 * one
    else:  # 2 k and 2 |p| (1 - sigmoid(p)) of the roundings of p
        p = gate if dt_bias is None else gate + dt_bias.view(1, H, 1, d)
        fin = torch.isfinite(p) & live
        p = torch.where(fin, p, 0 * one)
        k2 = torch.where(fin, 2 * p.abs() * torch.sigmoid(p) / torch.nn.functional.softplus(p), 0 * one)
        s2 = torch.where(fin, 2 * p.abs() * torch.sigmoid(-p), 0 * one)
    nla, kf = (9 + k2) * lam_, k2 if value != "none" else 0 * k2  # |log a|'s error, f's share of it
    nla, kf = nla.expand(B, H, N, d), kf.expand(B, H, N, d)
    u = f * x_
    h = zero.clone() if h0 is None else h0.clone()
    env, err = h.abs(), zero.clone()
    hb, he, hr, ys, yt = [], [], [], [], []
    for t in range(N):
        hb.append(h), he.append(env), hr.append(err)
        at = a[:, :, t]
        g = at * env
        h = at * h + u[:, :, t]
        err = at * err + U * ((nla[:, :, t] + 5) * g + (13 + kf[:, :, t]) * u[:, :, t].abs())
        env = g + u[:, :, t].abs()
        err = torch.where(live[:, :, t], err + U * env, err)
        ys.append(h), yt.append(err)
    before, env_b, err_b = (torch.stack(v, 2) for v in (hb, he, hr))
    y, ytol = torch.stack(ys, 2), torch.stack(yt, 2)
    out = {"y": torch.where(live, y, 0 * one), "y_tol": ytol, "h_out": h, "h_out_tol": err, "before": before,
           "before_tol": err_b}
    if dy is None:
        return out
    dy = torch.where(live, dy, 0 * one)
    lam = zero.clone() if dh_out is None else dh_out.clone()
    lenv, lerr = lam.abs(), zero.clone()
    L, LE, LR = [None] * N, [None] * N, [None] * N
    for t in range(N - 1, -1, -1):
        lam, lenv = lam + dy[:, :, t], lenv + dy[:, :, t].abs()
        lerr = lerr + 2 * U * lenv
        L[t], LE[t], LR[t] = lam, lenv, lerr
        at = a[:, :, t]
        lerr = at * (lerr + U * torch.where(live[:, :, t], nla[:, :, t] + 5, 0 * one) * lenv)
        lam, lenv = at * lam, at * lenv
    out["dh0"], out["dh0_tol"] = lam, lerr
    L, LE, LR = (torch.stack(v, 2) for v in (L, LE, LR))
    out["dx"], out["dx_tol"] = f * L, f.abs() * (LR + (14 + kf) * U * LE)
    dla, dla_t = a * L * before, a * (LR * env_b + LE * err_b + U * (nla + 8) * LE * env_b)
    if value == "complement":
        dla = dla - a * L * x_
        dla_t = dla_t + a * x_.abs() * (LR + U * (nla + 8) * LE) + U * (a * LE * (env_b + x_.abs()))
    dla, dla_t = torch.where(live, dla, 0 * one), torch.where(live, dla_t, 0 * one)
    if kind == "log":
        out["dgate"], out["dgate_tol"] = dla, dla_t
        return out
    ds, ds_t, mag = -rate * dla, rate * (dla_t + 5 * U * dla.abs()), rate * a * LE * (env_b + x_.abs())
    if value == "dt":
        ds, ds_t, mag = ds + L * x_, ds_t + x_.abs() * (LR + 2 * U * LE), mag + LE * x_.abs()
    sg = torch.where(live, sg, 0 * one)
    # the sigmoid: exponential, sum, quotient, each product: 8 U
    out["dgate"], out["dgate_tol"] = ds * sg, sg * (ds_t + (8 + s2) * U * mag)
    n = N + B + 8  # no chain of additions is longer
    la0 = torch.where(live, la.clamp(min=-200.0), 0 * one)
    for name, term, tol in (("dA_log", dla * la0, lam_ * (dla_t + (12 + k2) * U * a * LE * (env_b + x_.abs()))),
                            ("ddt_bias", out["dgate"], out["dgate_tol"])):
        out[name] = term.sum((0, 2)).reshape(-1)
        out[name + "_tol"] = (tol.sum((0, 2)) + n * U * (term.abs() + tol).sum((0, 2))).reshape(-1)
    return out


def check(got, want, tol, dtype, what):
    """|got - want| within tol plus the rounding to dtype, element by element."""
    got, want, tol = got.detach().cpu().double(), want, tol
    assert got.shape == want.shape, (what, got.shape, want.shape)
    room = tol + HALF[dtype] * (want.abs() + tol) + 1e-37
    bad = ~((got - want).abs() <= room)
    if bad.any():
        i = int(torch.argmax(((got - want).abs() / room).nan_to_num(nan=float("inf")).reshape(-1)))
        at = np.unravel_index(i, tuple(want.shape))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {at}: got "
                             f"{got.reshape(-1)[i]:.9g}, want {want.reshape(-1)[i]:.9g}, room {room.reshape(-1)[i]:.3g}")


# ------------------------------------------------------------------- norms
# A sum of C squares in float32, in any order: C U relative at the most (all
# terms positive), halved by the root; rsqrt and products: 8 U.

def norm_terms(v, eps, dims=-1):
    ms = (v * v).mean(dims, keepdim=True)
    return 1.0 / torch.sqrt(ms + eps)


def add_norm(x, residual, scale, w, eps, dtype, res_dtype):
    """(out, out_tol, r, rstd, rstd_tol); r as stored (rounded in float32 steps
    like the stream: product, sum, storage)."""
    xf = x.detach().cpu().float()
    v = xf if scale is None else scale.cpu().float() * xf
    v = v if residual is None else residual.cpu().float() + v
    r = v.to(res_dtype).double()
    rstd = norm_terms(r, eps)
    C = r.shape[-1]
    rel = (C / 2 + 8) * U
    out = r * rstd * (1.0 if w is None else f64(w))
    return out, out.abs() * rel, r, rstd[..., 0], rstd[..., 0] * rel


def add_norm_bwd(dy, r, rstd, w, x, scale, dres):
    """Gradients with bounds; rows flattened.  r, rstd as given to the kernel."""
    dy, r, rstd, w, x, scale, dres = (f64(t) for t in (dy, r, rstd, w, x, scale, dres))
    C = r.shape[-1]
    dy, r = dy.reshape(-1, C), r.reshape(-1, C)
    rs = rstd.reshape(-1, 1)
    xhat = r * rs
    g = dy if w is None else dy * w
    gx = g * xhat
    dr = rs * (g - xhat * gx.mean(-1, keepdim=True))
    dot_t = (C + 6) * U * gx.abs().mean(-1, keepdim=True)
    tol = rs * (xhat.abs() * dot_t + 6 * U * (g.abs() + xhat.abs() * gx.mean(-1, keepdim=True).abs()))
    if dres is not None:
        dr = dr + dres.reshape(-1, C)
        tol = tol + 2 * U * dr.abs()
    out = {"dr": dr, "dr_tol": tol}
    out["dx"], out["dx_tol"] = (dr, tol) if scale is None else (dr * scale, scale.abs() * (tol + U * dr.abs()))
    n = (dr.shape[0] + 8) * U
    if w is not None:
        out["dw"], out["dw_tol"] = (dy * xhat).sum(0), (n + 3 * U) * (dy * xhat).abs().sum(0)
    if scale is not None:
        x = x.reshape(-1, C)
        out["dscale"] = (dr * x).sum(0)
        out["dscale_tol"] = (tol * x.abs()).sum(0) + (n + U) * (dr * x).abs().sum(0)
    return out


def _tokens(x):
    B, H, N, d = x.shape
    return x.permute(0, 2, 1, 3).reshape(B, N, H * d)


def gated_norm(x, z, w, groups, eps, after):
    """(out, out_tol, rstd, rstd_tol) of [B, H, N, d] x and [B, N, H d] z."""
    x, z, w = _tokens(f64(x)), f64(z), f64(w)
    B, N, C = x.shape
    s = torch.ones_like(x) if z is None else z * torch.sigmoid(z)
    u = (x if after else x * s).view(B, N, groups, -1)
    rstd = norm_terms(u, eps)
    L = C // groups
    # SiLU: exponential (3 U, |z| of it from rounding z's product), sum, quotient, product
    sil = 8 * U
    rel = (L / 2 + 8) * U + 2 * sil
    out = (u * rstd).reshape(B, N, C)
    out = out * s if after else out
    out = out if w is None else out * w
    return out, out.abs() * rel, rstd[..., 0], rstd[..., 0] * rel


def gated_norm_bwd(dy, x, z, w, rstd, groups, after):
    B, H, N, d = x.shape
    dy, x, z, w, rstd = f64(dy), _tokens(f64(x)), f64(z), f64(w), f64(rstd)
    C = H * d
    L = C // groups
    sig = torch.zeros_like(x) if z is None else torch.sigmoid(z)
    s = torch.ones_like(x) if z is None else z * sig
    rs = rstd.view(B, N, groups, 1).expand(B, N, groups, L).reshape(B, N, C)
    u = x if after else x * s
    xhat = u * rs
    dn = dy * s if after else dy
    g = dn if w is None else dn * w
    mean = lambda t: t.view(B, N, groups, L).mean(-1, keepdim=True).expand(B, N, groups, L).reshape(B, N, C)  # noqa: E731
    m = mean(g * xhat)
    sil = 8 * U
    m_t = mean((g * xhat).abs()) * ((L + 6) * U + 2 * sil)
    du = rs * (g - xhat * m)
    du_t = rs * (xhat.abs() * m_t + (6 * U + sil) * (g.abs() + (xhat * m).abs()))
    n = xhat if w is None else xhat * w
    dsil = dy * n if after else du * x
    dsil_t = 4 * U * dsil.abs() if after else x.abs() * (du_t + 2 * U * du.abs())
    dx, dx_t = (du, du_t) if after else (du * s, s.abs() * (du_t + (sil + U) * du.abs()))
    out = {"dx": dx.view(B, N, H, d).permute(0, 2, 1, 3), "dx_tol": dx_t.view(B, N, H, d).permute(0, 2, 1, 3)}
    if z is not None:
        zz = sig * (1 + z * (1 - sig))
        zt = 12 * U * sig * (1 + 2 * z.abs() * (1 - sig)) + 2 * U * sig * z.abs()
        out["dz"], out["dz_tol"] = dsil * zz, dsil_t * zz.abs() + (dsil.abs() + dsil_t) * (zt + U * zz.abs())
    if w is not None:
        t = dn * xhat
        out["dw"] = t.sum((0, 1))
        out["dw_tol"] = ((B * N + 16) * U + 2 * sil) * t.abs().sum((0, 1))
    return out
