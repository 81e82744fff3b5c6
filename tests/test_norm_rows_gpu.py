"""The norms over more rows than the GPU holds at once, and over rows that lie
in larger buffers, against float64."""
import pytest

import mamba_ssd_sequence_b200 as ssd
from test_norm_gpu import EPS, TYPES, check_add, check_gated, make_gated, make_rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def test_gated_norm_of_the_longest_sequences():
    """Two sequences of 2^31 - 65537 tokens of one channel, batches apart by more
    than a sequence: a token's index and a step add up to more than 2^31.  Half
    a step of bf16 is 2^-8; the fp32 roundings are fewer than 40, and the
    gradient's act on rstd |dy|, of which 1 - xhat^2 is left."""
    N = 2 ** 31 - 65537
    g = torch.Generator(device="cuda").manual_seed(1)

    def rows(gap):  # [2, N] in a buffer of 3.0, gap elements between and behind
        buf = torch.full((2 * (N + gap),), 3.0, dtype=BF16, device="cuda")
        return buf, buf.as_strided((2, N), (N + gap, 1))

    _, x = rows(1000)
    for b in range(2):
        x[b].uniform_(-2, 2, generator=g)
    bufs = [rows(2000), rows(3000)]
    out, dx = (v for _, v in bufs)
    _, rstd = ssd.ssd_gated_norm(x.view(2, 1, N, 1), eps=1.0, out=out.view(2, N, 1))
    ssd.ssd_gated_norm_bwd(out.view(2, N, 1), x.view(2, 1, N, 1), rstd, dx=dx.view(2, 1, N, 1))
    for (buf, _), gap in zip(bufs, (2000, 3000)):
        assert (buf[N:N + gap] == 3.0).all() and (buf[2 * N + gap:] == 3.0).all()
    for b in range(2):
        for lo in range(0, N, 1 << 27):
            s = slice(lo, min(lo + (1 << 27), N))
            xd, rs = x[b, s].double(), (x[b, s].double().square() + 1).rsqrt()
            assert ((rstd[b, s, 0].double() - rs).abs() <= 16 * U * rs).all()
            want = xd * rs
            assert ((out[b, s].double() - want).abs() <= (2.0 ** -8 + 40 * U) * want.abs()).all()
            dy = out[b, s].double()
            want = dy * rs ** 3
            assert ((dx[b, s].double() - want).abs() <= 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8) + 40 * U * (dy * rs).abs()).all()
            del xd, rs, want, dy
    del x, out, dx, rstd, bufs, buf
    torch.cuda.empty_cache()


# Rows that one slot of a block takes one after the other, forward and backward in bf16 and fp32
@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("M,C", [
    (130001, 8),     # 1 and 1, 3 and 3
    (60000, 40),     # 4 and 4, 10 and 13
    (9001, 513),     # 5 and 10, 8 and 8; rows end inside a vector
    (4403, 1024),    # 2 and 5, 4 and 4
    (2999, 2048),    # 3 and 7, 5 and 5
    (1201, 8192),    # 5 and 8, 8 and 8
    (900, 9000),     # 8 and wide, 10 and wide: walked twice by a block, 3 rows each
    (700, 16400)])   # wide
def test_many_rows_of_the_residual_norm(M, C, dtype, stream):
    check_add(make_rows(M, C, dtype, stream, seed=C))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("B,H,N,d,groups", [
    (3, 2, 3001, 64, 1),     # 1 and 2, 4 and 4; a slot passes the end of a batch
    (3, 4, 2999, 64, 4),     # 3 and 4, 8 and 8
    (5, 3, 4001, 17, 3),     # 2 and 3, 6 and 6; element by element
    (2, 32, 1203, 64, 1),    # 3 and 4, 4 and 4
    (7, 16, 301, 64, 16),    # 2 and 4, 7 and 7; steps of up to three batches
    (601, 2, 7, 64, 1),      # 1 and 1, 2 and 2; steps of hundreds of batches
    (9, 8, 1500, 32, 8),     # 4 and 6, 10 and 11
    (2, 70, 400, 300, 1)])   # wide, 3 rows each
def test_many_rows_of_the_gated_norm(B, H, N, d, groups, after, dtype):
    check_gated(make_gated(B, H, N, d, dtype, seed=d), groups, after)


def in_buffer(t, at, gap):
    """t's values as a view of a larger buffer of 3.0: `at` elements in front of each
    row and gap - at behind it, one row in front of a batch's (or head's) rows and two behind."""
    shape = list(t.shape)
    shape[-2] += 3
    shape[-1] += gap
    buf = torch.full(shape, 3.0, dtype=t.dtype, device="cuda")
    view = buf[..., 1:-2, at:at + t.shape[-1]]
    view.copy_(t)
    return buf, view


def untouched(buf, view):
    view.fill_(3.0)
    return (buf == 3.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("at,gap", [(3, 8), (1, 3), (8, 16)])
@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("d,groups", [(17, 1), (17, 4), (64, 1), (64, 4)])
def test_gated_norm_in_larger_buffers(d, groups, after, at, gap, dtype):
    """Inputs and outputs inside of larger buffers, aligned or not: the same bits as
    contiguous ones (which are compared with float64), and nothing around them is written."""
    B, H, N = 3, 4, 1501
    t = make_gated(B, H, N, d, dtype, seed=d + at)
    check_gated(t, groups, after)
    out, rstd = ssd.ssd_gated_norm(t["x"], t["z"], t["w"], groups=groups, eps=EPS, gate_after=after)
    dx, dz, dw = ssd.ssd_gated_norm_bwd(t["dy"], t["x"], rstd, t["z"], t["w"], groups=groups, gate_after=after)
    inputs = {k: in_buffer(t[k], at, gap) for k in ("x", "z", "dy")}
    x, z, dy = (inputs[k][1] for k in ("x", "z", "dy"))
    results = [in_buffer(torch.zeros_like(v), at, gap) for v in (out, dx, dz)]
    o2, dx2, dz2 = (v for _, v in results)
    _, rstd2 = ssd.ssd_gated_norm(x, z, t["w"], groups=groups, eps=EPS, gate_after=after, out=o2)
    _, _, dw2 = ssd.ssd_gated_norm_bwd(dy, x, rstd2, z, t["w"], groups=groups, gate_after=after, dx=dx2, dz=dz2)
    for a, b in ((out, o2), (rstd, rstd2), (dx, dx2), (dz, dz2), (dw, dw2), (t["x"], x), (t["z"], z), (t["dy"], dy)):
        assert torch.equal(a, b)
    assert all(untouched(buf, v) for buf, v in results + list(inputs.values()))


def test_gated_norm_offsets_beyond_32_bits():
    """Rows so far apart that element offsets pass 2^31."""
    H, N, d, step = 2, 300, 16, 9_000_001
    big = torch.empty(N * step, dtype=BF16, device="cuda")
    heads = lambda at: big[at:].as_strided((1, H, N, d), (0, 40, step, 1))  # noqa: E731
    rows = lambda at: big[at:].as_strided((1, N, H * d), (0, step, 1))  # noqa: E731
    t = make_gated(1, H, N, d, BF16, seed=3)
    far = dict(x=heads(0), z=rows(100), dy=rows(200))
    for k, v in far.items():
        v.copy_(t[k])
    a = ssd.ssd_gated_norm(t["x"], t["z"], t["w"], groups=2)
    b = ssd.ssd_gated_norm(far["x"], far["z"], t["w"], groups=2, out=rows(300))
    p = ssd.ssd_gated_norm_bwd(t["dy"], t["x"], a[1], t["z"], t["w"], groups=2)
    q = ssd.ssd_gated_norm_bwd(far["dy"], far["x"], b[1], far["z"], t["w"], groups=2, dx=heads(400), dz=rows(500))
    assert all(torch.equal(u, v) for u, v in zip(a + p, b + q))
