"""The recurrence and the norms together, as a block uses them: a training step
of residual norm -> projections -> recurrence -> gated norm -> projection ->
residual norm, and generation after a prefill; the gated norm behind the SSD
operator."""
import pytest

import mamba_ssd_sequence_b200 as ssd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
EPS = 1e-5
# Relative 2-norm error of the chain in float32.  A product of K = 64 terms is
# off by at most K roundings of 2^-24 of the sum of its absolute terms, which
# is up to sqrt(K) = 8 times the result for terms of either sign: on the mean
# of random roundings sqrt(K) 8 2^-24 = 64 2^-24 = 3.8e-6.  Ten such products
# lie between an input and its gradient (three forward, their two gradients
# each, and one more), and the recurrence and norms between them add at most 30
# roundings each, 3.6e-6 in all four of a direction: below 5e-5 together.
TOL = 5e-5


def params(C, H, d, dtype=F32, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    return {k: v.to(dtype).cuda() for k, v in dict(
        w1=1 + 0.1 * rn(C), W_in=rn(C, 3 * H * d) / C ** 0.5, A_log=torch.log(1 + 15 * torch.rand(H * d, generator=g, dtype=F64)),
        bias=rn(H * d) - 3, wg=1 + 0.1 * rn(H * d), W_out=rn(H * d, C) / (H * d) ** 0.5, scale=0.3 + 0.05 * rn(C),
        w2=1 + 0.1 * rn(C)).items()}


def split(p, B, N, H, d):
    """x, gate ([B, H, N, d] views) and z ([B, N, H*d] view) of one projection."""
    q = p.view(B, N, 3, H, d)
    return q[:, :, 0].permute(0, 2, 1, 3), q[:, :, 1].permute(0, 2, 1, 3), p.view(B, N, 3, H * d)[:, :, 2]


def block(P, x, res, H, d, lengths=None, h0=None, h_out=None, keep=None):
    B, N, C = x.shape
    n1, r1, s1 = ssd.ssd_add_norm(x, res, None, P["w1"], eps=EPS)
    proj = (n1.view(-1, C) @ P["W_in"]).view(B, N, -1)
    xv, gate, z = split(proj, B, N, H, d)
    states = None if keep is None else ssd.alloc_glr_states(B, H, N, d)
    y = ssd.ssd_glr_fwd(xv, gate, P["A_log"], P["bias"], value_complement=True, h0=h0, h_out=h_out, states=states,
                        lengths=lengths)
    o, sg = ssd.ssd_gated_norm(y, z, P["wg"], groups=H, eps=EPS)
    b = (o.view(-1, H * d) @ P["W_out"]).view(B, N, C)
    n2, r2, s2 = ssd.ssd_add_norm(b, r1, P["scale"], P["w2"], eps=EPS)
    if keep is not None:
        keep.update(n1=n1, r1=r1, s1=s1, proj=proj, states=states, y=y, o=o, sg=sg, b=b, r2=r2, s2=s2)
    return n2, r2


def block_bwd(P, k, dn2, dr2, H, d, lengths=None):
    B, N, C = dn2.shape
    xv, gate, z = split(k["proj"], B, N, H, d)
    dr1, db, dw2, dscale = ssd.ssd_add_norm_bwd(dn2, k["r2"], k["s2"], P["w2"], x=k["b"], scale=P["scale"], dres=dr2)
    do = (db.view(-1, C) @ P["W_out"].T).view(B, N, -1)
    dW_out = k["o"].view(-1, H * d).T @ db.view(-1, C)
    dproj = torch.empty_like(k["proj"])
    dxv, dgate, dz = split(dproj, B, N, H, d)  # written in place
    dy, _, dwg = ssd.ssd_gated_norm_bwd(do, k["y"], k["sg"], z, P["wg"], groups=H, dz=dz)
    _, _, dA, dbias, _ = ssd.ssd_glr_bwd(dy, xv, gate, P["A_log"], P["bias"], k["states"], value_complement=True,
                                         lengths=lengths, dx=dxv, dgate=dgate)
    dn1 = (dproj.view(-1, dproj.shape[-1]) @ P["W_in"].T).view(B, N, C)
    dW_in = k["n1"].view(-1, C).T @ dproj.view(-1, dproj.shape[-1])
    dres, dx, dw1, _ = ssd.ssd_add_norm_bwd(dn1, k["r1"], k["s1"], P["w1"], dres=dr1)
    return dict(x=dx, res=dres, w1=dw1, W_in=dW_in, A_log=dA, bias=dbias, wg=dwg, W_out=dW_out, scale=dscale, w2=dw2)


def reference(P, x, res, H, d, lengths=None):
    B, N, C = x.shape
    norm = lambda v: v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + EPS)  # noqa: E731
    r1 = res + x
    proj = (norm(r1) * P["w1"]) @ P["W_in"]
    xv, gate, z = split(proj, B, N, H, d)
    la = -torch.exp(P["A_log"]).view(H, 1, d) * torch.nn.functional.softplus(gate + P["bias"].view(H, 1, d))
    a = torch.exp(la)
    h, ys = torch.zeros(B, H, d, dtype=F64, device=x.device), []
    for t in range(N):
        h = a[:, :, t] * h + (1 - a[:, :, t]) * xv[:, :, t]
        ys.append(h)
    y = torch.stack(ys, 2)
    if lengths is not None:
        y = y * (torch.arange(N, device=x.device)[None] < lengths[:, None]).view(B, 1, N, 1)
    u = y.transpose(1, 2).reshape(B, N, H * d) * torch.nn.functional.silu(z)
    o = norm(u.view(B, N, H, d)).reshape(B, N, H * d) * P["wg"]
    r2 = r1 + P["scale"] * (o @ P["W_out"])
    return norm(r2) * P["w2"], r2


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("padded", [False, True])
def test_training_step(padded):
    B, N, C, H, d = 3, 150, 64, 2, 32
    P = params(C, H, d)
    x, res, dn2, dr2 = (torch.randn(B, N, C, device="cuda", generator=torch.Generator("cuda").manual_seed(i)) for i in range(4))
    lengths = torch.tensor([150, 97, 1], dtype=torch.int32, device="cuda") if padded else None
    keep = {}
    n2, r2 = block(P, x, res, H, d, lengths, keep=keep)
    got = block_bwd(P, keep, dn2, dr2, H, d, lengths)
    Q = {k: v.double().requires_grad_() for k, v in P.items()}
    xd, rd = x.double().requires_grad_(), res.double().requires_grad_()
    m2, q2 = reference(Q, xd, rd, H, d, lengths)
    assert rel(n2, m2.detach()) < TOL and rel(r2, q2.detach()) < TOL
    names = ["x", "res"] + list(P)
    want = torch.autograd.grad((m2 * dn2.double()).sum() + (q2 * dr2.double()).sum(), [xd, rd] + [Q[k] for k in P])
    for name, w in zip(names, want):
        assert rel(got[name], w) < TOL, name
    # and the loss's change along a random direction of every input at once
    g = torch.Generator("cuda").manual_seed(9)
    move = {n: torch.randn(v.shape, generator=g, device="cuda", dtype=F64) for n, v in [("x", xd), ("res", rd)] + list(Q.items())}

    def loss(s):
        R = {k: v.detach() + s * move[k] for k, v in Q.items()}
        a, b = reference(R, xd.detach() + s * move["x"], rd.detach() + s * move["res"], H, d, lengths)
        return float((a * dn2.double()).sum() + (b * dr2.double()).sum())

    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    mine = sum(float((got[n].double() * move[n]).sum()) for n in names)
    size = sum(float((got[n].double() * move[n]).norm()) for n in names)
    assert abs(slope - mine) < 1e-4 * size


def test_generation_continues_a_padded_prefill():
    """Sequences of different lengths are prefilled together, then continued
    token by token from the state that each had at its own end."""
    B, N, C, H, d, more = 3, 60, 64, 2, 32, 5
    P = params(C, H, d, seed=3)
    g = torch.Generator("cuda").manual_seed(5)
    lens = [60, 33, 1]
    x, res = (torch.randn(B, N + more, C, device="cuda", generator=g) for _ in range(2))
    h = torch.empty(B, H, d, device="cuda")
    block(P, x[:, :N].contiguous(), res[:, :N].contiguous(), H, d, torch.tensor(lens, dtype=torch.int32, device="cuda"),
          h_out=h)
    outs = []
    for s in range(more):  # token lens[b] + s of sequence b
        at = lambda t: torch.stack([t[b, lens[b] + s] for b in range(B)])  # noqa: E731
        n1, r1, _ = ssd.ssd_add_norm(at(x), at(res), None, P["w1"], eps=EPS)
        xv, gate, z = split((n1 @ P["W_in"]).view(B, 1, -1), B, 1, H, d)
        y = ssd.ssd_glr_step(xv[:, :, 0], gate[:, :, 0], P["A_log"], P["bias"], h, value_complement=True)
        o, _ = ssd.ssd_gated_norm(y[:, :, None], z, P["wg"], groups=H, eps=EPS)
        n2, _, _ = ssd.ssd_add_norm(o.view(B, -1) @ P["W_out"], r1, P["scale"], P["w2"], eps=EPS)
        outs.append(n2)
    Q = {k: v.double() for k, v in P.items()}
    for b in range(B):
        m2, _ = reference(Q, x[b:b + 1, :lens[b] + more].double(), res[b:b + 1, :lens[b] + more].double(), H, d)
        got = torch.stack([o[b] for o in outs])
        assert rel(got, m2[0, lens[b]:]) < TOL


def test_gated_norm_behind_the_operator():
    """ssd_fwd's output goes through the gated norm in place, in bf16 at the
    operator's own sizes: the same as the norm's float64 form on that output,
    to bf16's half step (2^-8) and the sums' roundings (1024 / 2 + 24) 2^-24."""
    B, H, N, d = 2, 16, 256, 64
    g = torch.Generator("cuda").manual_seed(7)
    q, k, v = (torch.nn.functional.silu(torch.randn(B, H, N, d, device="cuda", generator=g)).to(BF16) for _ in range(3))
    dt_p = torch.randn(B, H, N, device="cuda", generator=g)
    A_log, bias = torch.zeros(H, device="cuda"), torch.full((H,), -3.0, device="cuda")
    z = torch.randn(B, N, H * d, device="cuda", generator=g).to(BF16)
    w = 1 + 0.1 * torch.randn(H * d, device="cuda", generator=g)
    y = ssd.ssd_fwd(q, k, v, dt_p, A_log, bias, None, 1, False, 128)
    out, _ = ssd.ssd_gated_norm(y, z, w, eps=EPS)
    u = y.double().transpose(1, 2).reshape(B, N, H * d) * torch.nn.functional.silu(z.double())
    want = u / torch.sqrt(u.pow(2).mean(-1, keepdim=True) + EPS) * w.double()
    room = (2.0 ** -8 + 540 * 2.0 ** -24) * want.abs() * (1 + 2.0 ** -8)
    assert ((out.double() - want).abs() <= room).all()


def test_refusals():
    x = torch.randn(2, 3, 20, 16, device="cuda")
    A = torch.zeros(48, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        ssd.ssd_glr_fwd(x, x[:, :, :10], A, A)
    with pytest.raises(TypeError, match="gate"):
        ssd.ssd_glr_fwd(x, x.to(BF16), A, A)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssd.ssd_glr_fwd(x.half(), x.half(), A, A)
    with pytest.raises(ValueError, match="A_log must have shape"):
        ssd.ssd_glr_fwd(x, x, A[:16], A)
    with pytest.raises(ValueError, match="last dimension"):
        ssd.ssd_glr_fwd(x.transpose(2, 3).contiguous().transpose(2, 3), x, A, A)
    with pytest.raises(ValueError, match="CUDA device"):
        ssd.ssd_glr_fwd(x, x, A.cpu(), A)
    with pytest.raises(TypeError, match="lengths"):
        ssd.ssd_glr_fwd(x, x, A, A, lengths=torch.tensor([1, 2], device="cuda"))
    with pytest.raises(ssd.SSDError):
        ssd.ssd_glr_fwd(x, x, A, A, out=torch.empty(2, 3, 1, 16, device="cuda").expand(2, 3, 20, 16))
    with pytest.raises(ssd.SSDError):
        ssd.ssd_glr_fwd(x[:, :, :0], x[:, :, :0], A, A)
    with pytest.raises(ValueError, match="states"):
        ssd.ssd_glr_bwd(x, x, x, A, A, None)
    states = ssd.alloc_glr_states(2, 3, 20, 16)
    with pytest.raises(ssd.SSDError):
        ssd.ssd_glr_bwd(x, x, x, A, A, states, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="state h"):
        ssd.ssd_glr_step(x[:, :, 0], x[:, :, 0], A, A, None)
    r = torch.randn(4, 3, 32, device="cuda")
    with pytest.raises(ValueError, match="evenly spaced"):
        ssd.ssd_add_norm(torch.randn(4, 5, 32, device="cuda")[:, :3])
    with pytest.raises(ssd.SSDError):
        ssd.ssd_add_norm(r, eps=0.0)
    with pytest.raises(ssd.SSDError):
        ssd.ssd_add_norm(r, residual=r.to(BF16))
    with pytest.raises(ValueError, match="needs x"):
        ssd.ssd_add_norm_bwd(r, r, r[..., 0].contiguous(), scale=r[0, 0])
    with pytest.raises(ssd.SSDError):
        ssd.ssd_gated_norm(x, groups=5)
    with pytest.raises(ValueError, match="dz"):
        ssd.ssd_gated_norm_bwd(torch.zeros(2, 20, 48, device="cuda"), x, torch.zeros(2, 20, 1, device="cuda"),
                               dz=torch.zeros(2, 20, 48, device="cuda"))
