"""The gated linear recurrence against its token-by-token form in float64:
forward, gradients, decode step, padded batches, views, streams and graphs."""
import pytest

import mamba_ssd_sequence_b200 as ssd
from block_reference import check, recurrence

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

F32, BF16 = torch.float32, torch.bfloat16


def make(B, H, N, d, dtype, kind="dt", seed=0, layout="heads"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731

    def act(t):
        t = t.to(dtype)
        if layout == "tokens":    # a slice of a token-major projection
            buf = torch.zeros(B, N, 3, H, d, dtype=dtype, device="cuda")
            buf[:, :, 1] = t.permute(0, 2, 1, 3)
            return buf[:, :, 1].permute(0, 2, 1, 3)
        if layout == "offset":    # element-aligned only, odd row stride
            buf = torch.zeros(B, H, N, d + 3, dtype=dtype, device="cuda")
            buf[..., 1:1 + d] = t
            return buf[..., 1:1 + d]
        return t.contiguous()

    x = act(torch.nn.functional.silu(rn(B, H, N, d)))
    gate = rn(B, H, N, d)
    gate = act(-torch.nn.functional.softplus(gate - 2.0) if kind == "log" else gate)
    dy = act(rn(B, H, N, d))
    A_log = torch.log(1 + 15 * torch.rand(H * d, generator=g, device="cuda")) if kind == "dt" else None
    bias = rn(H * d) - 3.0 if kind == "dt" else None
    return dict(x=x, gate=gate, dy=dy, A_log=A_log, bias=bias, h0=rn(B, H, d), dh=rn(B, H, d))


def kwargs(gate, kind, value):
    k = dict(value_dt=value == "dt", value_complement=value == "complement")
    return (gate, dict(k)) if kind == "dt" else (None, dict(k, log_decay=gate))


def forward(t, kind, value, carried=True, lengths=None, save=True, **more):
    B, H, N, d = t["x"].shape
    dt_p, kw = kwargs(t["gate"], kind, value)
    h_out = torch.full((B, H, d), 7.0, device="cuda")
    states = ssd.alloc_glr_states(B, H, N, d).fill_(7.0) if save else None
    y = ssd.ssd_glr_fwd(t["x"], dt_p, t["A_log"], t["bias"], h0=t["h0"] if carried else None, h_out=h_out,
                        states=states, lengths=lengths, **kw, **more)
    return y, h_out, states


def backward(t, kind, value, states, carried=True, lengths=None, **more):
    dt_p, kw = kwargs(t["gate"], kind, value)
    return ssd.ssd_glr_bwd(t["dy"], t["x"], dt_p, t["A_log"], t["bias"], states, lengths=lengths,
                           dh_out=t["dh"] if carried else None, **kw, **more)


def run_and_check(t, kind, value, carried=True, lengths=None):
    dtype = t["x"].dtype
    y, h_out, states = forward(t, kind, value, carried, lengths)
    got = dict(zip(("dx", "dgate", "dA_log", "ddt_bias", "dh0"), backward(t, kind, value, states, carried, lengths)))
    ref = recurrence(t["x"], t["gate"], t["A_log"], t["bias"], t["h0"] if carried else None, lengths, kind, value,
                     t["dy"], t["dh"] if carried else None)
    check(y, ref["y"], ref["y_tol"], dtype, "y")
    check(h_out, ref["h_out"], ref["h_out_tol"], F32, "h_out")
    N = t["x"].shape[2]
    at = torch.arange(0, N, ssd.SSD_GLR_CHUNK)
    check(states, ref["before"][:, :, at], ref["before_tol"][:, :, at], F32, "states")
    for name, v in got.items():
        if kind == "log" and name in ("dA_log", "ddt_bias"):
            assert v is None
            continue
        check(v, ref[name], ref[name + "_tol"], dtype if name in ("dx", "dgate") else F32, name)


CASES = [  # (kind, value)
    ("dt", "none"), ("dt", "dt"), ("dt", "complement"), ("log", "none"), ("log", "complement")]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind,value", CASES)
@pytest.mark.parametrize("B,H,N,d", [(2, 3, 300, 32), (1, 2, 77, 64)])
def test_options(B, H, N, d, kind, value, dtype):
    run_and_check(make(B, H, N, d, dtype, kind, seed=N), kind, value)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1031])
def test_lengths_of_time(N, dtype):
    run_and_check(make(1, 2, N, 64, dtype, seed=N), "dt", "complement")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [1, 2, 3, 5, 8, 16, 17, 24, 31, 40, 63, 65, 96, 128, 130, 200])
def test_head_sizes(d, dtype):
    run_and_check(make(2, 2, 70, d, dtype, seed=d), "dt", "dt", carried=d % 2 == 0)


@pytest.mark.parametrize("layout", ["tokens", "offset"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [16, 33, 64])
def test_views(d, dtype, layout):
    run_and_check(make(2, 3, 150, d, dtype, seed=d, layout=layout), "dt", "complement")


@pytest.mark.parametrize("layout", ["tokens", "offset"])
def test_view_results_equal_contiguous_ones(layout):
    """The layout of the views does not change a bit; outputs may be views."""
    t = make(2, 3, 150, 64, BF16, seed=5, layout=layout)
    c = {k: v if v is None else v.contiguous() for k, v in t.items()}
    a, b = forward(t, "dt", "dt"), forward(c, "dt", "dt", out=torch.zeros(2, 150, 3, 64, dtype=BF16, device="cuda").transpose(1, 2))
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    buf = torch.zeros(2, 150, 2, 3, 64, dtype=BF16, device="cuda")
    p = backward(t, "dt", "dt", a[2])
    q = backward(c, "dt", "dt", a[2], dx=buf[:, :, 0].transpose(1, 2), dgate=buf[:, :, 1].transpose(1, 2))
    assert all(torch.equal(u, v) for u, v in zip(p, q))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,N,d", [
    (1, 1, 5000, 8), (1, 1, 4099, 64), (1, 3, 2500, 64), (5, 4, 700, 64), (3, 50, 130, 64), (40, 16, 40, 64), (1, 40, 2050, 16),
    (7, 12, 700, 32), (1, 48, 700, 64), (3, 3, 4001, 64), (2, 20, 900, 64)])
def test_splits_of_the_sequence(B, H, N, d, dtype):
    """From one channel block to more than the SMs hold at once."""
    run_and_check(make(B, H, N, d, dtype, seed=N), "dt", "complement")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind,value", [("dt", "dt"), ("log", "complement")])
def test_padded_batch(kind, value, dtype):
    """Tokens behind a length: not used (they hold NaN here), outputs and
    gradients 0, the state that of the last token that counts.  Lengths are
    clamped to [0, N]."""
    N = 530
    lengths = torch.tensor([N, 0, 1, 16, 17, 257, N + 5, -3], dtype=torch.int32, device="cuda")
    t = make(8, 2, N, 32, dtype, kind, seed=9)
    clean = {k: v if v is None else v.clone() for k, v in t.items()}
    dead = (torch.arange(N, device="cuda")[None] >= lengths[:, None]).view(8, 1, N, 1).expand(8, 2, N, 32)
    for k in ("x", "gate", "dy"):
        t[k][dead] = float("nan")
    run_and_check_padded(t, clean, kind, value, lengths, dead)


def run_and_check_padded(t, clean, kind, value, lengths, dead):
    dtype = t["x"].dtype
    y, h_out, states = forward(t, kind, value, lengths=lengths)
    dx, dgate, dA, db, dh0 = backward(t, kind, value, states, lengths=lengths)
    ref = recurrence(clean["x"], clean["gate"], t["A_log"], t["bias"], t["h0"], lengths, kind, value, clean["dy"],
                     t["dh"])
    for v in (y, dx, dgate):
        assert (v[dead] == 0).all()
    check(y, ref["y"], ref["y_tol"], dtype, "y")
    check(h_out, ref["h_out"], ref["h_out_tol"], F32, "h_out")
    assert torch.equal(h_out[1], t["h0"][1])
    check(dx, ref["dx"], ref["dx_tol"], dtype, "dx")
    check(dgate, ref["dgate"], ref["dgate_tol"], dtype, "dgate")
    check(dh0, ref["dh0"], ref["dh0_tol"], F32, "dh0")
    if kind == "dt":
        check(dA, ref["dA_log"], ref["dA_log_tol"], F32, "dA_log")
        check(db, ref["ddt_bias"], ref["ddt_bias_tol"], F32, "ddt_bias")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinite_gates(dtype):
    """-infinity: a softplus gate leaves the state, a log-decay restarts it;
    +infinity in a softplus gate restarts it.  No NaN in any gradient."""
    t = make(1, 2, 200, 16, dtype, seed=3)
    t["gate"][:, :, 50:60] = float("-inf")
    t["gate"][:, :, 120] = float("inf")
    run_and_check(t, "dt", "complement")
    y, _, _ = forward(t, "dt", "complement")
    assert torch.equal(y[:, :, 59], y[:, :, 49])
    t = make(1, 2, 200, 16, dtype, "log", seed=4)
    t["gate"][:, :, 100] = float("-inf")
    run_and_check(t, "log", "none")
    y, _, _ = forward(t, "log", "none")
    assert torch.equal(y[:, :, 100], t["x"][:, :, 100])


@pytest.mark.parametrize("value", ["none", "dt", "complement"])
def test_slow_decay(value):
    """Decays of 1e-6 a token, whose errors add up over the whole sequence."""
    t = make(1, 2, 3000, 16, F32, seed=6)
    t["bias"] = torch.full_like(t["bias"], -14.0)
    run_and_check(t, "dt", value)


def test_without_parameters():
    """A_log and dt_bias None: rate 1, bias 0 (a = 1 - sigmoid(gate))."""
    t = make(2, 2, 90, 32, F32, seed=8)
    t["A_log"] = t["bias"] = None
    y, h_out, states = forward(t, "dt", "complement")
    dx, dgate, dA, db, dh0 = backward(t, "dt", "complement", states)
    assert dA is None and db is None
    ref = recurrence(t["x"], t["gate"], None, None, t["h0"], None, "dt", "complement", t["dy"], t["dh"])
    check(y, ref["y"], ref["y_tol"], F32, "y")
    check(dgate, ref["dgate"], ref["dgate_tol"], F32, "dgate")
    a = 1 - torch.sigmoid(t["gate"].double())
    h1 = (a[:, :, 0] * t["h0"] + (1 - a[:, :, 0]) * t["x"][:, :, 0].double()).float()
    torch.testing.assert_close(y[:, :, 0], h1, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind,value", CASES)
@pytest.mark.parametrize("B,H,d", [(1, 1, 1), (3, 2, 17), (4, 16, 64), (257, 5, 33)])
def test_step(B, H, d, kind, value, dtype):
    t = make(B, H, 1, d, dtype, kind, seed=B)
    gate, kw = kwargs(t["gate"][:, :, 0], kind, value)
    if "log_decay" in kw:
        kw["log_decay"] = t["gate"][:, :, 0]
    h = t["h0"].clone()
    y = ssd.ssd_glr_step(t["x"][:, :, 0], gate, t["A_log"], t["bias"], h, **kw)
    ref = recurrence(t["x"], t["gate"], t["A_log"], t["bias"], t["h0"], None, kind, value)
    check(y, ref["y"][:, :, 0], ref["y_tol"][:, :, 0], dtype, "y")
    check(h, ref["h_out"], ref["h_out_tol"], F32, "h")


def test_prefill_in_pieces_and_steps_continue_a_sequence():
    """One call, two calls that pass the state on, and a call followed by steps."""
    t = make(2, 2, 400, 32, F32, seed=12)
    ref = recurrence(t["x"], t["gate"], t["A_log"], t["bias"], t["h0"], None, "dt", "complement")
    h = t["h0"].clone()
    part = lambda k, s: t[k][:, :, s]  # noqa: E731
    ys = []
    for s in (slice(0, 150), slice(150, 390)):
        ys.append(ssd.ssd_glr_fwd(part("x", s), part("gate", s), t["A_log"], t["bias"], value_complement=True, h0=h,
                                  h_out=h))
    for n in range(390, 400):
        ys.append(ssd.ssd_glr_step(t["x"][:, :, n], t["gate"][:, :, n], t["A_log"], t["bias"], h,
                                   value_complement=True)[:, :, None])
    check(torch.cat(ys, 2), ref["y"], ref["y_tol"], F32, "y")
    check(h, ref["h_out"], ref["h_out_tol"], F32, "h")


def test_same_bits_every_time_on_two_streams():
    t = make(2, 8, 1500, 64, BF16, seed=13)
    want = forward(t, "dt", "dt")
    want_g = backward(t, "dt", "dt", want[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for k in range(6):
        s = streams[k % 2]
        s.wait_stream(torch.cuda.current_stream())
        B, H, N, d = t["x"].shape
        with torch.cuda.stream(s):
            f = forward(t, "dt", "dt")
        got.append((f, backward(t, "dt", "dt", f[2], stream=s)))
    torch.cuda.synchronize()
    for f, g in got:
        assert all(torch.equal(u, v) for u, v in zip(want + tuple(want_g), f + tuple(g)))


def test_side_stream_memory_is_not_reused():
    """A call on a stream other than the current one, whose tensors are dropped at once."""
    t = make(1, 16, 4096, 64, BF16, seed=14)
    want = forward(t, "dt", "dt", save=False)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        x = t["x"].clone()
        side.wait_stream(torch.cuda.current_stream())
        y = ssd.ssd_glr_fwd(x, t["gate"], t["A_log"], t["bias"], value_dt=True, h0=t["h0"], stream=side)
        del x
        junk = torch.full((1, 16, 4096, 64), float("nan"), dtype=BF16, device="cuda")
        side.synchronize()
        assert torch.equal(y, want)
        del junk


def test_graph_replay():
    """Captured forward, backward and step replay on new contents of their inputs."""
    t = make(2, 4, 700, 64, BF16, seed=15)
    forward(t, "dt", "dt"), torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = forward(t, "dt", "dt")
        g = backward(t, "dt", "dt", f[2])
        y1 = ssd.ssd_glr_step(t["x"][:, :, 0], t["gate"][:, :, 0], t["A_log"], t["bias"], f[1])
    new = make(2, 4, 700, 64, BF16, seed=16)
    for k in t:
        t[k].copy_(new[k])
    graph.replay()
    torch.cuda.synchronize()
    want = forward(new, "dt", "dt")
    want_g = backward(new, "dt", "dt", want[2])
    y2 = ssd.ssd_glr_step(new["x"][:, :, 0], new["gate"][:, :, 0], new["A_log"], new["bias"], want[1])
    assert all(torch.equal(u, v) for u, v in zip(f + tuple(g) + (y1,), want + tuple(want_g) + (y2,)))


def test_guard_bands():
    """Nothing outside the outputs is written: rows between a view's rows, the
    ends of the buffers."""
    B, H, N, d = 2, 2, 333, 24
    for dtype in (F32, BF16):
        t = make(B, H, N, d, dtype, seed=17)
        buf = torch.full((B, H, N + 2, d + 5), 3.0, dtype=dtype, device="cuda")
        out = buf[:, :, 1:-1, 2:2 + d]
        _, _, states = forward(t, "dt", "dt", out=out)
        keep = buf.clone()
        keep[:, :, 1:-1, 2:2 + d] = 3.0
        assert (keep == 3.0).all()
        bx, bg = torch.full_like(buf, 3.0), torch.full_like(buf, 3.0)
        backward(t, "dt", "dt", states, dx=bx[:, :, 1:-1, 2:2 + d], dgate=bg[:, :, 1:-1, 2:2 + d])
        for b in (bx, bg):
            assert not (b[:, :, 1:-1, 2:2 + d] == 3.0).all()
            b[:, :, 1:-1, 2:2 + d] = 3.0
            assert (b == 3.0).all()


def test_offsets_beyond_32_bits():
    """Rows so far apart that element offsets pass 2^31 (and bytes 2^32)."""
    N, d, step = 300, 16, 9_000_001
    big = torch.empty(N * step, dtype=BF16, device="cuda")
    view = lambda at: big[at:].as_strided((1, 1, N, d), (0, 0, step, 1))  # noqa: E731
    t = make(1, 1, N, d, BF16, seed=18)
    x, gate, dy = view(0), view(100), view(200)
    for v, k in ((x, "x"), (gate, "gate"), (dy, "dy")):
        v.copy_(t[k])
    far = dict(t, x=x, gate=gate, dy=dy)
    a, b = forward(t, "dt", "dt"), forward(far, "dt", "dt", out=view(300))
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    p = backward(t, "dt", "dt", a[2])
    q = backward(far, "dt", "dt", a[2], dx=view(400), dgate=view(500))
    assert all(torch.equal(u, v) for u, v in zip(p, q))


def test_long_sequence():
    """64K tokens of few channels: the state of the last token, and the whole
    output against the same recurrence in pieces of odd length."""
    t = make(1, 2, 65536, 16, BF16, "log", seed=19)
    y, h_out, _ = forward(t, "log", "none", save=False)
    ref = recurrence(t["x"], t["gate"], None, None, t["h0"], None, "log", "none")
    check(y, ref["y"], ref["y_tol"], BF16, "y")
    check(h_out, ref["h_out"], ref["h_out_tol"], F32, "h_out")
