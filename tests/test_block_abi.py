"""The recurrence's and the norms' entry points refuse bad arguments on the
host, before any CUDA call (fake pointers, never dereferenced)."""
import struct

import pytest
import torch

import mamba_ssd_sequence_b200 as ssd
from mamba_ssd_sequence_b200 import build as ssd_build

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, FLAGS = 0, 1, 2, 3, 6, 7, 11


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load_library()


def view(ptr=4096, sb=32 * 2 * 16, sh=32 * 16, sn=16):
    return struct.pack("Pqqq", ptr, sb, sh, sn)


def rows(ptr=4096, stride=64):
    return struct.pack("Pq", ptr, stride)


def params(eps=1e-5, groups=1, flags=0):
    return struct.pack("fii", eps, groups, flags)


def glr_fwd(lib, **over):
    a = dict(x=view(), gate=view(), A=64, b=64, h0=None, lengths=None, B=2, H=2, N=32, d=16, dtype=ssd.SSD_F32,
             flags=0, out=view(), h_out=None, states=None)
    a.update(over)
    return lib.ssd_glr_fwd(*[a[k] for k in ("x", "gate", "A", "b", "h0", "lengths", "B", "H", "N", "d", "dtype",
                                            "flags", "out", "h_out", "states")], None)


COMMON = [
    (dict(x=None), NULL), (dict(gate=None), NULL), (dict(x=view(0)), NULL),
    (dict(B=0), SHAPE), (dict(H=0), SHAPE), (dict(N=0), SHAPE), (dict(d=0), SHAPE), (dict(B=-1), SHAPE),
    (dict(H=1 << 20, d=1 << 20), SHAPE), (dict(B=1 << 20, H=1 << 20), SHAPE), (dict(N=(1 << 31) - 1), SHAPE), (dict(B=1, H=1, N=1, d=(1 << 31) - 8), SHAPE),
    (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE),
    (dict(flags=8), FLAGS), (dict(flags=-1), FLAGS), (dict(flags=3), FLAGS), (dict(flags=5), FLAGS), (dict(flags=7), FLAGS),
    (dict(x=view(4098)), ALIGN), (dict(x=view(4097), dtype=ssd.SSD_BF16), ALIGN), (dict(A=66), ALIGN),
    (dict(b=65), ALIGN), (dict(x=view(sb=-1)), SHAPE), (dict(gate=view(sh=-16)), SHAPE), (dict(gate=view(sn=-16)), SHAPE),
]


@pytest.mark.parametrize("over,code", COMMON + [
    (dict(out=None), NULL), (dict(out=view(0)), NULL), (dict(h0=2), ALIGN), (dict(h_out=2), ALIGN),
    (dict(states=2), ALIGN), (dict(lengths=2), ALIGN),
    (dict(out=view(sn=0)), SHAPE), (dict(out=view(sn=15)), SHAPE), (dict(out=view(sb=0)), SHAPE),
    (dict(out=view(sh=16 * 31)), SHAPE), (dict(out=view(sb=1024, sh=8, sn=16)), SHAPE)])
def test_glr_fwd_codes(lib, over, code):
    assert glr_fwd(lib, **over) == code


def glr_bwd(lib, **over):
    a = dict(dy=view(), x=view(), gate=view(), A=64, b=64, states=64, lengths=None, dh=None, B=2, H=2, N=32, d=16,
             dtype=ssd.SSD_F32, flags=0, dx=view(), dgate=view(), dA=64, db=64, dh0=None, ws=256, n=1 << 40)
    a.update(over)
    return lib.ssd_glr_bwd(*[a[k] for k in ("dy", "x", "gate", "A", "b", "states", "lengths", "dh", "B", "H", "N", "d",
                                            "dtype", "flags", "dx", "dgate", "dA", "db", "dh0", "ws", "n")], None)


@pytest.mark.parametrize("over,code", COMMON + [
    (dict(dy=None), NULL), (dict(states=None), NULL), (dict(dx=None), NULL), (dict(dgate=None), NULL),
    (dict(states=66), ALIGN), (dict(dh=66), ALIGN), (dict(dA=66), ALIGN), (dict(db=66), ALIGN), (dict(dh0=66), ALIGN),
    (dict(flags=2), FLAGS), (dict(flags=2, dA=None), FLAGS), (dict(dx=view(sn=0)), SHAPE), (dict(dgate=view(sh=0)), SHAPE),
    (dict(ws=None), WORKSPACE), (dict(n=0), WORKSPACE), (dict(ws=128), ALIGN)])
def test_glr_bwd_codes(lib, over, code):
    assert glr_bwd(lib, **over) == code


def test_glr_workspace_bytes():
    n = ssd.ssd_glr_bwd_workspace_bytes(2, 2, 32, 16, ssd.SSD_F32)
    assert n > 0 and n % 256 == 0
    for bad in ((0, 2, 32, 16, 0, 0), (2, 2, 0, 16, 0, 0), (2, 2, 32, 16, 3, 0), (2, 2, 32, 16, 0, 8)):
        assert ssd.ssd_glr_bwd_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("over,code", [
    (dict(x=None), NULL), (dict(gate=None), NULL), (dict(out=None), NULL), (dict(h=None), NULL), (dict(B=0), SHAPE),
    (dict(d=0), SHAPE), (dict(dtype=9), DTYPE), (dict(flags=3), FLAGS), (dict(h=66), ALIGN), (dict(out=view(sb=0)), SHAPE)])
def test_glr_step_codes(lib, over, code):
    a = dict(x=view(), gate=view(), A=64, b=64, B=2, H=2, d=16, dtype=0, flags=0, h=64, out=view())
    a.update(over)
    assert lib.ssd_glr_step(*[a[k] for k in ("x", "gate", "A", "b", "B", "H", "d", "dtype", "flags", "h", "out")],
                            None) == code


@pytest.mark.parametrize("over,code", [
    (dict(x=None), NULL), (dict(out=None), NULL), (dict(p=None), NULL), (dict(r=None), NULL),
    (dict(r=None, res=None, scale=None, dtype=1, rdtype=0), NULL), (dict(M=0), SHAPE), (dict(C=0), SHAPE),
    (dict(dtype=4), DTYPE), (dict(dtype=0, rdtype=1), DTYPE), (dict(p=params(0.0)), SHAPE), (dict(p=params(-1.0)), SHAPE),
    (dict(p=params(float("nan"))), SHAPE), (dict(out=rows(stride=63)), SHAPE), (dict(r=rows(stride=0)), SHAPE),
    (dict(x=rows(stride=-64)), SHAPE), (dict(x=rows(4098)), ALIGN), (dict(res=rows(4098)), ALIGN), (dict(scale=66), ALIGN),
    (dict(w=66), ALIGN), (dict(rstd=66), ALIGN)])
def test_add_norm_codes(lib, over, code):
    a = dict(x=rows(), res=rows(), scale=64, w=64, M=4, C=64, dtype=0, rdtype=0, p=params(), r=rows(), out=rows(), rstd=64)
    a.update(over)
    assert lib.ssd_add_norm(*[a[k] for k in ("x", "res", "scale", "w", "M", "C", "dtype", "rdtype", "p", "r", "out",
                                             "rstd")], None) == code


@pytest.mark.parametrize("over,code", [
    (dict(dy=None), NULL), (dict(r=None), NULL), (dict(rstd=None), NULL), (dict(dr=None), NULL), (dict(x=None), NULL),
    (dict(M=0), SHAPE), (dict(C=0), SHAPE), (dict(dtype=4), DTYPE), (dict(rdtype=1), DTYPE), (dict(dr=rows(stride=1)), SHAPE),
    (dict(dx=rows(stride=1)), SHAPE), (dict(dw=66), ALIGN), (dict(ds=66), ALIGN), (dict(dres=rows(4097)), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(n=0), WORKSPACE), (dict(ws=8), ALIGN)])
def test_add_norm_bwd_codes(lib, over, code):
    a = dict(dy=rows(), r=rows(), rstd=64, w=64, x=rows(), scale=64, dres=rows(), M=4, C=64, dtype=0, rdtype=0, dr=rows(),
             dx=rows(), dw=64, ds=64, ws=256, n=1 << 40)
    a.update(over)
    assert lib.ssd_add_norm_bwd(*[a[k] for k in ("dy", "r", "rstd", "w", "x", "scale", "dres", "M", "C", "dtype",
                                                 "rdtype", "dr", "dx", "dw", "ds", "ws", "n")], None) == code
    assert lib.ssd_add_norm_bwd_workspace_bytes(0, 4) == 0 and lib.ssd_add_norm_bwd_workspace_bytes(4, 4) > 0


GATED = [
    (dict(x=None), NULL), (dict(p=None), NULL), (dict(z=view(0)), NULL), (dict(B=0), SHAPE), (dict(N=0), SHAPE),
    (dict(p=params(groups=0)), SHAPE), (dict(p=params(groups=3)), SHAPE), (dict(dtype=2), DTYPE),
    (dict(p=params(flags=2)), FLAGS), (dict(w=66), ALIGN), (dict(rstd=66), ALIGN), (dict(x=view(4098)), ALIGN),
    (dict(x=view(sn=-1)), SHAPE)]


@pytest.mark.parametrize("over,code", GATED + [
    (dict(out=None), NULL), (dict(out=view(sn=0)), SHAPE), (dict(p=params(eps=0.0)), SHAPE)])
def test_gated_norm_codes(lib, over, code):
    a = dict(x=view(), z=view(), w=64, B=2, H=2, N=32, d=16, dtype=0, p=params(), out=view(), rstd=64)
    a.update(over)
    assert lib.ssd_gated_norm(*[a[k] for k in ("x", "z", "w", "B", "H", "N", "d", "dtype", "p", "out", "rstd")],
                              None) == code


@pytest.mark.parametrize("over,code", GATED + [
    (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(dz=None), NULL), (dict(z=None), NULL), (dict(rstd=None), NULL),
    (dict(dz=view(sh=0)), SHAPE), (dict(dw=66), ALIGN), (dict(ws=None), WORKSPACE), (dict(n=0), WORKSPACE),
    (dict(ws=64), ALIGN)])
def test_gated_norm_bwd_codes(lib, over, code):
    a = dict(dy=view(), x=view(), z=view(), w=64, rstd=64, B=2, H=2, N=32, d=16, dtype=0, p=params(), dx=view(), dz=view(),
             dw=64, ws=256, n=1 << 40)
    a.update(over)
    assert lib.ssd_gated_norm_bwd(*[a[k] for k in ("dy", "x", "z", "w", "rstd", "B", "H", "N", "d", "dtype", "p", "dx",
                                                   "dz", "dw", "ws", "n")], None) == code
    assert lib.ssd_gated_norm_bwd_workspace_bytes(1, 2, 3, 4, 5) == 0
    assert lib.ssd_gated_norm_bwd_workspace_bytes(1, 2, 3, 4, 8) > 0


def test_binding_refuses_host_tensors_and_mixed_options(lib):
    x = torch.zeros(1, 2, 4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_glr_fwd(x, x, None, None)
    with pytest.raises(ValueError, match="either dt_p or log_decay"):
        ssd.ssd_glr_fwd(x, x, None, None, log_decay=x)
    with pytest.raises(ValueError, match="either dt_p or log_decay"):
        ssd.ssd_glr_fwd(x, None, None, None)
    with pytest.raises(ValueError, match="value_dt"):
        ssd.ssd_glr_fwd(x, None, None, None, log_decay=x, value_dt=True)
    with pytest.raises(ValueError, match="value_dt"):
        ssd.ssd_glr_fwd(x, x, None, None, value_dt=True, value_complement=True)
    for call in (lambda: ssd.ssd_add_norm(x), lambda: ssd.ssd_gated_norm(x), lambda: ssd.ssd_glr_step(x[:, :, 0], x[:, :, 0],
                 None, None, x[:, :, 0]), lambda: ssd.ssd_add_norm_bwd(x, x, x[..., 0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert ssd.glr_states_shape(2, 3, 33, 8) == (2, 3, 3, 8)
