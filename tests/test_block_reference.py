"""The float64 forms that the recurrence and the norms are tested against have
the right gradients: against automatic differentiation of a separate writing
of the definition, and against central differences."""
import pytest
import torch

from block_reference import add_norm_bwd, gated_norm_bwd, recurrence

D = torch.float64


def rnd(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed), dtype=D)


def scan(x, gate, A_log, bias, h0, lengths, kind, value):
    B, H, N, d = x.shape
    if kind == "log":
        la = gate
    else:
        dt = torch.log(1 + torch.exp(gate + bias.view(1, H, 1, d)))
        la = -torch.exp(A_log.view(1, H, 1, d)) * dt
    a = torch.exp(la)
    f = dt if value == "dt" else 1 - a if value == "complement" else 1.0
    u = f * x
    h, y = h0, []
    for t in range(N):
        new = a[:, :, t] * h + u[:, :, t]
        live = torch.ones(B, 1, 1, dtype=torch.bool) if lengths is None else (t < lengths).view(B, 1, 1)
        y.append(torch.where(live, new, torch.zeros_like(new)))
        h = torch.where(live, new, h)
    return torch.stack(y, 2), h


@pytest.mark.parametrize("kind,value", [("dt", "none"), ("dt", "dt"), ("dt", "complement"), ("log", "none"),
                                        ("log", "complement")])
@pytest.mark.parametrize("padded", [False, True])
def test_recurrence_gradients(kind, value, padded):
    B, H, N, d = 3, 2, 9, 4
    x, h0, dy, dh = rnd(B, H, N, d, seed=1), rnd(B, H, d, seed=3), rnd(B, H, N, d, seed=4), rnd(B, H, d, seed=5)
    gate = rnd(B, H, N, d, seed=2)
    gate = -gate.abs() if kind == "log" else gate
    A, b = (rnd(H * d, seed=6), rnd(H * d, seed=7)) if kind == "dt" else (None, None)
    lengths = torch.tensor([9, 0, 4]) if padded else None
    leaves = [t.clone().requires_grad_() for t in (x, gate, h0)] + ([A.clone().requires_grad_(), b.clone().requires_grad_()]
                                                                     if kind == "dt" else [None, None])

    def loss(lv):
        y, h = scan(lv[0], lv[1], lv[3], lv[4], lv[2], lengths, kind, value)
        return (y * dy).sum() + (h * dh).sum()

    live = [t for t in leaves if t is not None]
    got = torch.autograd.grad(loss(leaves), live)
    ref = recurrence(x, gate, A, b, h0, lengths, kind, value, dy, dh)
    names = ["dx", "dgate", "dh0", "dA_log", "ddt_bias"][:len(live)]
    for name, g in zip(names, got):
        torch.testing.assert_close(ref[name].reshape(g.shape), g, rtol=1e-10, atol=1e-12)
    y, h = scan(x, gate, A, b, h0, lengths, kind, value)
    torch.testing.assert_close(ref["y"], y)
    torch.testing.assert_close(ref["h_out"], h)
    # central differences along a random direction of each input
    for i, name in enumerate(names):
        j = [k for k, t in enumerate(leaves) if t is live[i]][0]
        v, eps = rnd(*live[i].shape, seed=20 + i), 1e-5
        ends = []
        for s in (eps, -eps):
            moved = [None if t is None else t.detach() for t in leaves]
            moved[j] = moved[j] + s * v
            ends.append(loss(moved))
        want = (ends[0] - ends[1]) / (2 * eps)
        torch.testing.assert_close((ref[name].reshape(v.shape) * v).sum(), want, rtol=1e-6, atol=1e-7)


def test_add_norm_gradients():
    M, C, eps = 4, 6, 1e-3
    x, res, scale, w = (rnd(*s, seed=i).requires_grad_() for i, s in enumerate([(M, C), (M, C), (C,), (C,)]))
    dy, dr2 = rnd(M, C, seed=8), rnd(M, C, seed=9)
    r = res + scale * x
    rstd = (r.pow(2).mean(1) + eps).rsqrt()
    got = torch.autograd.grad((r * rstd[:, None] * w * dy).sum() + (r * dr2).sum(), [res, x, w, scale])
    ref = add_norm_bwd(dy, r, rstd, w, x, scale, dr2)
    for name, g in zip(("dr", "dx", "dw", "dscale"), got):
        torch.testing.assert_close(ref[name], g, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("groups", [1, 3])
def test_gated_norm_gradients(after, groups):
    B, H, N, d, eps = 2, 3, 4, 5, 1e-3
    x, z, w = (rnd(*s, seed=i).requires_grad_() for i, s in enumerate([(B, H, N, d), (B, N, H * d), (H * d,)]))
    dy = rnd(B, N, H * d, seed=5)
    t = x.transpose(1, 2).reshape(B, N, H * d)
    silu = torch.nn.functional.silu(z)
    u = (t if after else t * silu).view(B, N, groups, -1)
    rstd = (u.pow(2).mean(-1) + eps).rsqrt()
    y = (u * rstd[..., None]).view(B, N, H * d) * w
    y = y * silu if after else y
    got = torch.autograd.grad((y * dy).sum(), [x, z, w])
    ref = gated_norm_bwd(dy, x, z, w, rstd, groups, after)
    for name, g in zip(("dx", "dz", "dw"), got):
        torch.testing.assert_close(ref[name], g, rtol=1e-10, atol=1e-12)
