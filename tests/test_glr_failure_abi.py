"""The recurrence's failure-test entries refuse what is out of range, on the host
(fake pointers, never dereferenced)."""
import struct

import pytest

import mamba_ssd_sequence_b200 as ssd
from mamba_ssd_sequence_b200 import build as ssd_build

SHAPE, UNSUPPORTED = 2, 10


@pytest.mark.parametrize("late", [(-2, 0, 0), (8, 0, 0), (0, -1, 0), (0, 10 ** 9 + 1, 0), (0, 0, -1), (0, 0, 10 ** 9 + 1)])
def test_ranges(late):
    ssd_build.build()
    lib = ssd.load_library()
    v = struct.pack("Pqqq", 4096, 1024, 512, 16)
    assert lib.ssd_debug_glr_fwd(v, v, 64, 64, None, None, 2, 2, 32, 16, 0, 0, v, None, None, None, *late) == SHAPE
    assert lib.ssd_debug_glr_bwd(v, v, v, 64, 64, 64, None, None, 2, 2, 32, 16, 0, 0, v, v, None, None, None, 256, 1 << 40,
                                 None, *late) == SHAPE


@pytest.mark.parametrize("over", [dict(d=32), dict(flags=1)])
def test_late_blocks_of_other_kernels(over):
    """Refused before the launch."""
    ssd_build.build()
    lib = ssd.load_library()
    d, flags = over.get("d", 16), over.get("flags", 0)
    v = struct.pack("Pqqq", 4096, 64 * d, 32 * d, d)
    assert lib.ssd_debug_glr_fwd(v, v, 64, 64, None, None, 2, 2, 32, d, 0, flags, v, None, None, None, 0, 0, 0) == UNSUPPORTED
    assert lib.ssd_debug_glr_bwd(v, v, v, 64, 64, 64, None, None, 2, 2, 32, d, 0, flags, v, v, None, None, None, 256, 1 << 40,
                                 None, 0, 0, 0) == UNSUPPORTED
