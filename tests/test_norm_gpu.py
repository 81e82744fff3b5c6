"""The residual norm and the gated norm, and their gradients, against float64."""
import pytest

import mamba_ssd_sequence_b200 as ssd
from block_reference import add_norm, add_norm_bwd, check, gated_norm, gated_norm_bwd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def make_rows(M, C, dtype, stream, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rows(dt, std=1.0):
        t = (torch.randn(M, C + pad, generator=g, device="cuda") * std).to(dt)
        return t[:, pad:] if pad else t

    vec = lambda mean, std: torch.randn(C, generator=g, device="cuda") * std + mean  # noqa: E731
    return dict(x=rows(dtype), res=rows(stream, 2.0), dy=rows(dtype), dres=rows(stream), scale=vec(0.3, 0.05),
                w=vec(1.0, 0.1))


def check_add(t, scale=True, res=True, w=True, dres=True):
    x, dtype = t["x"], t["x"].dtype
    scale, w = t["scale"] if scale else None, t["w"] if w else None
    res, dres = t["res"] if res else None, t["dres"] if dres else None
    stream = dtype if res is None else res.dtype
    out, r, rstd = ssd.ssd_add_norm(x, res, scale, w, eps=EPS)
    o, o_t, rr, rs, rs_t = add_norm(x, res, scale, w, EPS, dtype, stream)
    if res is None and scale is None:
        assert r is x
    assert torch.equal(r.cpu().double(), rr)
    check(out, o, o_t, dtype, "out")
    check(rstd, rs, rs_t, F32, "rstd")
    if dres is not None and dres.dtype != r.dtype:
        dres = dres.to(r.dtype)
    dr, dx, dw, ds = ssd.ssd_add_norm_bwd(t["dy"], r, rstd, w, x=x, scale=scale, dres=dres)
    ref = add_norm_bwd(t["dy"], r, rstd, w, x, scale, dres)
    check(dr, ref["dr"].view(dr.shape), ref["dr_tol"].view(dr.shape), r.dtype, "dr")
    check(dx, ref["dx"].view(dr.shape), ref["dx_tol"].view(dr.shape), dtype, "dx")
    assert (dw is None) == (w is None) and (ds is None) == (scale is None)
    if w is not None:
        check(dw, ref["dw"], ref["dw_tol"], F32, "dw")
    if scale is not None:
        check(ds, ref["dscale"], ref["dscale_tol"], F32, "dscale")


TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("M,C", [
    (1, 1), (1, 7), (3, 8), (5, 64), (2, 100), (7, 256), (1, 1000), (33, 1024), (600, 513), (9, 2048), (3, 4096),
    (2, 5000), (3, 8192), (2, 16384), (2, 20001), (2, 40000), (1300, 96)])
def test_add_norm_sizes(M, C, dtype, stream):
    check_add(make_rows(M, C, dtype, stream, seed=M + C))


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("scale,res,w,dres", [
    (False, True, True, True), (True, False, True, True), (False, False, True, False), (True, True, False, True),
    (True, True, True, False), (False, False, False, False)])
def test_add_norm_options(scale, res, w, dres, dtype, stream):
    check_add(make_rows(50, 512, dtype, stream, seed=2), scale, res, w, dres)


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("pad", [1, 8])
def test_add_norm_strided_rows(pad, dtype, stream):
    check_add(make_rows(40, 320, dtype, stream, seed=3, pad=pad))


def test_add_norm_in_place_and_in_more_dimensions():
    t = make_rows(24, 256, BF16, F32, seed=4)
    want = ssd.ssd_add_norm(t["x"], t["res"], t["scale"], t["w"])
    res = t["res"].clone().view(2, 3, 4, 256)
    out, r, rstd = ssd.ssd_add_norm(t["x"].view(2, 3, 4, 256), res, t["scale"], t["w"], r=res)
    assert r is res and out.shape == (2, 3, 4, 256) and rstd.shape == (2, 3, 4)
    for a, b in zip(want, (out, r, rstd)):
        assert torch.equal(a.reshape(-1), b.reshape(-1))
    want = ssd.ssd_add_norm_bwd(t["dy"], want[1], want[2], t["w"], x=t["x"], scale=t["scale"], dres=t["dres"])
    dres = t["dres"].clone()
    got = ssd.ssd_add_norm_bwd(t["dy"], r.view(24, 256), rstd.view(24), t["w"], x=t["x"], scale=t["scale"], dres=dres,
                               dr=dres)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_rows_of_zeros_and_of_infinities():
    """A zero row normalises to zero (eps), and does not meet its neighbours;
    an infinite or NaN row spoils itself only."""
    x = torch.randn(5, 128, device="cuda")
    x[1], x[3, 5] = 0.0, float("inf")
    out, _, rstd = ssd.ssd_add_norm(x, w=torch.ones(128, device="cuda"))
    assert (out[1] == 0).all() and torch.isclose(rstd[1], torch.tensor(EPS ** -0.5, device="cuda"), rtol=1e-5)
    good = torch.tensor([0, 2, 4], device="cuda")
    assert torch.isfinite(out[good]).all()
    want, _, _ = ssd.ssd_add_norm(x[good].contiguous(), w=torch.ones(128, device="cuda"))
    assert torch.equal(out[good], want)


def make_gated(B, H, N, d, dtype, seed=0, layout="heads"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x = rn(B, H, N, d) if layout == "heads" else rn(B, N, H, d).transpose(1, 2)
    z, dy = rn(B, N, H * d) * 2, rn(B, N, H * d)
    if layout == "odd":
        z, dy = (torch.cat([t[..., :1], t], -1)[..., 1:] for t in (z, dy))
    w = torch.randn(H * d, generator=g, device="cuda") * 0.1 + 1
    return dict(x=x, z=z, dy=dy, w=w)


def check_gated(t, groups, after, z=True, w=True):
    x, dtype = t["x"], t["x"].dtype
    z, w = t["z"] if z else None, t["w"] if w else None
    out, rstd = ssd.ssd_gated_norm(x, z, w, groups=groups, eps=EPS, gate_after=after)
    o, o_t, rs, rs_t = gated_norm(x, z, w, groups, EPS, after)
    check(out, o, o_t, dtype, "out")
    check(rstd, rs, rs_t, F32, "rstd")
    dx, dz, dw = ssd.ssd_gated_norm_bwd(t["dy"], x, rstd, z, w, groups=groups, gate_after=after)
    ref = gated_norm_bwd(t["dy"], x, z, w, rstd, groups, after)
    check(dx, ref["dx"], ref["dx_tol"], dtype, "dx")
    assert (dz is None) == (z is None) and (dw is None) == (w is None)
    if z is not None:
        check(dz, ref["dz"], ref["dz_tol"], dtype, "dz")
    if w is not None:
        check(dw, ref["dw"], ref["dw_tol"], F32, "dw")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("B,H,N,d,groups", [
    (1, 1, 1, 1, 1), (2, 2, 3, 16, 1), (2, 2, 3, 16, 2), (1, 16, 40, 64, 1), (1, 16, 40, 64, 16), (2, 3, 50, 24, 3),
    (1, 5, 33, 17, 1), (1, 5, 33, 17, 5), (1, 4, 20, 64, 2), (1, 4, 20, 64, 8), (1, 3, 7, 40, 2), (1, 32, 5, 128, 1),
    (1, 64, 3, 256, 1), (1, 64, 3, 256, 64), (1, 70, 2, 300, 1), (2, 6, 700, 32, 6)])
def test_gated_norm(B, H, N, d, groups, after, dtype):
    check_gated(make_gated(B, H, N, d, dtype, seed=d), groups, after)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("z,w", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("after", [False, True])
def test_gated_norm_options(after, z, w, dtype):
    check_gated(make_gated(2, 4, 30, 32, dtype, seed=1), 4, after, z, w)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["tokens", "odd"])
@pytest.mark.parametrize("groups", [1, 4])
def test_gated_norm_views(groups, layout, dtype):
    check_gated(make_gated(2, 4, 30, 32, dtype, seed=2, layout=layout), groups, True)


@pytest.mark.parametrize("after", [False, True])
def test_gates_of_large_size(after):
    """SiLU at +-100 and +-infinity-sized values: no NaN, the gate closes."""
    t = make_gated(1, 2, 8, 32, F32, seed=3)
    t["z"][0, 1] = -100.0
    t["z"][0, 2] = 100.0
    t["z"][0, 3] = -3e38
    out, rstd = ssd.ssd_gated_norm(t["x"], t["z"], t["w"], gate_after=after)
    assert torch.isfinite(out).all() and (out[0, 3] == 0).all()
    got = ssd.ssd_gated_norm_bwd(t["dy"], t["x"], rstd, t["z"], t["w"], gate_after=after)
    assert all(torch.isfinite(v).all() for v in got)


def test_norms_replay_in_a_graph_and_on_streams():
    t = make_rows(3000, 512, BF16, BF16, seed=5)
    q = make_gated(2, 8, 500, 64, BF16, seed=6)

    def all_of(stream=None):
        a = ssd.ssd_add_norm(t["x"], t["res"], t["scale"], t["w"], stream=stream)
        b = ssd.ssd_add_norm_bwd(t["dy"], a[1], a[2], t["w"], x=t["x"], scale=t["scale"], dres=t["dres"], stream=stream)
        c = ssd.ssd_gated_norm(q["x"], q["z"], q["w"], groups=8, stream=stream)
        e = ssd.ssd_gated_norm_bwd(q["dy"], q["x"], c[1], q["z"], q["w"], groups=8, stream=stream)
        return a + b + c + e

    want = all_of()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [all_of(side) for _ in range(3)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = all_of()
    graph.replay()
    torch.cuda.synchronize()
    for g in got + [captured]:
        assert all(torch.equal(a, b) for a, b in zip(want, g))


def test_norm_guard_bands():
    for dtype in (F32, BF16):
        for C in (40, 41, 1024):
            t = make_rows(37, C, dtype, dtype, seed=7)
            bufs = [torch.full((39, C + 6), 3.0, dtype=dtype, device="cuda") for _ in range(4)]
            v = [b[1:-1, 3:3 + C] for b in bufs]
            _, _, rstd = ssd.ssd_add_norm(t["x"], t["res"], t["scale"], t["w"], r=v[0], out=v[1])
            ssd.ssd_add_norm_bwd(t["dy"], v[0], rstd, t["w"], x=t["x"], scale=t["scale"], dr=v[2], dx=v[3])
            for b in bufs:
                assert not (b[1:-1, 3:3 + C] == 3.0).all()
                b[1:-1, 3:3 + C] = 3.0
                assert (b == 3.0).all()


def test_row_offsets_beyond_32_bits():
    M, C, step = 300, 64, 9_000_001
    big = torch.empty(M * step, dtype=BF16, device="cuda")
    view = lambda at: big[at:].as_strided((M, C), (step, 1))  # noqa: E731
    t = make_rows(M, C, BF16, BF16, seed=8)
    far = {k: view(100 * i) for i, k in enumerate(("x", "res", "dy", "dres"))}
    for k, v in far.items():
        v.copy_(t[k])
    a = ssd.ssd_add_norm(t["x"], t["res"], t["scale"], t["w"])
    b = ssd.ssd_add_norm(far["x"], far["res"], t["scale"], t["w"], r=view(400), out=view(500))
    p = ssd.ssd_add_norm_bwd(t["dy"], a[1], a[2], t["w"], x=t["x"], scale=t["scale"], dres=t["dres"])
    q = ssd.ssd_add_norm_bwd(far["dy"], b[1], b[2], t["w"], x=far["x"], scale=t["scale"], dres=far["dres"],
                             dr=view(600), dx=view(700))
    assert all(torch.equal(u, v) for u, v in zip(a + p, b + q))
