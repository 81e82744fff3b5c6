"""The recurrence's waits between the blocks of a cluster are bounded.  Here one
block of each cluster starts later than the others' limit: these give up, write
NaN and send nothing more; the late block still computes its first round from
what was sent to it, then finds nothing and gives up too.  No output that depends
on a missing part is a number, the kernel returns, and the next call is right."""
import struct

import pytest

import mamba_ssd_sequence_b200 as ssd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

# One channel block of 16 channels is walked by a cluster of 8, in tiles of 512
# bf16 or 256 fp32 tokens.
H, d, BLOCKS = 4, 16, 8
TILE = {torch.bfloat16: 512, torch.float32: 256}
LATE_NS, LIMIT_NS = 30_000_000, 2_000_000


def view(t):
    return struct.pack("Pqqq", t.data_ptr(), *t.stride()[:3])


class Case:
    def __init__(self, N, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.N, self.dtype, self.code = N, dtype, ssd.SSD_F32 if dtype == torch.float32 else ssd.SSD_BF16
        self.x, self.gate, self.dy = (rn(1, H, N, d).to(dtype) for _ in range(3))
        self.A, self.b, self.dh = rn(H * d), rn(H * d) - 3, rn(1, H, d)
        self.h0 = rn(1, H, d)

    def forward(self, *late):
        out, h = torch.full_like(self.x, 7.0), torch.full_like(self.h0, 7.0)
        states = ssd.alloc_glr_states(1, H, self.N, d).fill_(7.0)
        rc = ssd.load_library().ssd_debug_glr_fwd(
            view(self.x), view(self.gate), self.A.data_ptr(), self.b.data_ptr(), self.h0.data_ptr(), None, 1, H, self.N, d,
            self.code, 0, view(out), h.data_ptr(), states.data_ptr(), torch.cuda.current_stream().cuda_stream, *late)
        assert rc == 0
        torch.cuda.synchronize()
        return out, h, states

    def backward(self, states, *late):
        dx, dg, dh0 = torch.full_like(self.x, 7.0), torch.full_like(self.x, 7.0), torch.full_like(self.h0, 7.0)
        dA, db = torch.full_like(self.A, 7.0), torch.full_like(self.b, 7.0)
        n = ssd.ssd_glr_bwd_workspace_bytes(1, H, self.N, d, self.code)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        rc = ssd.load_library().ssd_debug_glr_bwd(
            view(self.dy), view(self.x), view(self.gate), self.A.data_ptr(), self.b.data_ptr(), states.data_ptr(), None,
            self.dh.data_ptr(), 1, H, self.N, d, self.code, 0, view(dx), view(dg), dA.data_ptr(), db.data_ptr(),
            dh0.data_ptr(), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream, *late)
        assert rc == 0
        torch.cuda.synchronize()
        return dx, dg, dA, db, dh0


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


def only(got, want, tokens, step=1):
    """got has want's numbers at these tokens (every step-th is stored), NaN elsewhere."""
    live = torch.zeros(got.shape[2], dtype=torch.bool, device="cuda")
    live[tokens.start // step:tokens.stop // step] = True
    assert torch.equal(got[:, :, live], want[:, :, live])
    assert torch.isnan(got[:, :, ~live]).all()


@pytest.mark.parametrize("dtype", list(TILE))
@pytest.mark.parametrize("rounds", [1, 2, 5])
@pytest.mark.parametrize("late", [0, 3, 7])
def test_a_late_block(late, rounds, dtype):
    tile = TILE[dtype]
    c = Case(rounds * BLOCKS * tile, dtype, seed=rounds)
    want = c.forward(-1, 0, 0)
    assert not any(torch.isnan(v).any() for v in want)
    out, h, states = c.forward(late, LATE_NS, LIMIT_NS)
    own = slice(late * tile, (late + 1) * tile)
    only(out, want[0], own)
    only(states, want[2], own, ssd.SSD_GLR_CHUNK)
    if rounds == 1 and late == 0:  # the first block writes the final state, and had every part
        assert torch.equal(h, want[1])
    else:
        assert torch.isnan(h).all()
    grads = c.backward(want[2], -1, 0, 0)
    dx, dg, dA, db, dh0 = c.backward(want[2], late, LATE_NS, LIMIT_NS)
    first = (rounds - 1) * BLOCKS * tile  # rounds are walked from the last one
    own = slice(first + own.start, first + own.stop)
    only(dx, grads[0], own)
    only(dg, grads[1], own)
    assert torch.isnan(dA).all() and torch.isnan(db).all()
    if rounds == 1 and late == 0:
        assert torch.equal(dh0, grads[4])
    else:
        assert torch.isnan(dh0).all()
    # the next calls are as before
    assert same(c.forward(-1, 0, 0), want) and same(c.backward(want[2], -1, 0, 0), grads)


@pytest.mark.parametrize("dtype", list(TILE))
def test_a_block_that_comes_in_time(dtype):
    """A delay within the limit changes nothing."""
    c = Case(3 * BLOCKS * TILE[dtype] - 100, dtype, seed=9)
    want = c.forward(-1, 0, 0)
    assert same(c.forward(2, 1_000_000, 0), want)
    assert same(c.backward(want[2], 5, 1_000_000, 0), c.backward(want[2], -1, 0, 0))
