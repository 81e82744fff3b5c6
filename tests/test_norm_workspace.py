"""The workspace that the norms' gradients take can be sized from Python."""
import pytest

import mamba_ssd_sequence_b200 as ssd
from mamba_ssd_sequence_b200 import build as ssd_build

torch = pytest.importorskip("torch")


def test_sizes():
    ssd_build.build()
    lib = ssd.load_library()
    for M, C in ((1, 1), (37, 41), (8192, 1024), (70000, 16385)):
        n = ssd.ssd_add_norm_bwd_workspace_bytes(M, C)
        assert n == lib.ssd_add_norm_bwd_workspace_bytes(M, C) and n > 0 and n % 256 == 0
    for size in ((1, 1, 1, 1, 1), (2, 6, 700, 32, 6), (4, 16, 4096, 32, 1)):
        n = ssd.ssd_gated_norm_bwd_workspace_bytes(*size)
        assert n == lib.ssd_gated_norm_bwd_workspace_bytes(*size) and n > 0 and n % 256 == 0
    assert ssd.ssd_add_norm_bwd_workspace_bytes(0, 4) == 0
    assert ssd.ssd_gated_norm_bwd_workspace_bytes(2, 3, 4, 5, groups=4) == 0


@pytest.mark.gpu
def test_given_workspaces():
    """Of exactly that size they serve, with the same bits; a byte less is refused."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dy, r, w = rn(1000, 200), rn(1000, 200), rn(200)
    _, _, rstd = ssd.ssd_add_norm(r, w=w)
    want = ssd.ssd_add_norm_bwd(dy, r, rstd, w)
    ws = torch.empty(ssd.ssd_add_norm_bwd_workspace_bytes(1000, 200), dtype=torch.uint8, device="cuda")
    got = ssd.ssd_add_norm_bwd(dy, r, rstd, w, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(want[:3], got[:3]))
    with pytest.raises(ssd.SSDError):
        ssd.ssd_add_norm_bwd(dy, r, rstd, w, workspace=ws[:-1])
    x, z, dy, w = rn(2, 4, 300, 24), rn(2, 300, 96), rn(2, 300, 96), rn(96)
    _, rstd = ssd.ssd_gated_norm(x, z, w, groups=4)
    want = ssd.ssd_gated_norm_bwd(dy, x, rstd, z, w, groups=4)
    ws = torch.empty(ssd.ssd_gated_norm_bwd_workspace_bytes(2, 4, 300, 24, groups=4), dtype=torch.uint8, device="cuda")
    got = ssd.ssd_gated_norm_bwd(dy, x, rstd, z, w, groups=4, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(ssd.SSDError):
        ssd.ssd_gated_norm_bwd(dy, x, rstd, z, w, groups=4, workspace=ws[:-1])
