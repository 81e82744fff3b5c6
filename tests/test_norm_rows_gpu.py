"""The norms over more rows than the GPU holds at once, and over rows that lie
in larger buffers, against float64."""
import pytest

import mamba_ssd_sequence_b200 as ssd

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
