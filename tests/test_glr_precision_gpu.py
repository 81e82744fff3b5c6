"""dt = softplus(gate + dt_bias) and its slope in fp32, at every size of dt, against
float64: with x = 1, no state and no bias, out of f = dt is dt itself, and the
gradient of the gate its slope.

The bound in units of U = 2^-24: u = exp(-|p|) 3.4 (the hardware's exponential
1.4e-7, the correction 1) and 0.05 |p| (ln 2 in float32 is off by 2.8e-9
relative; an uncorrected rounding of the exponent would be up to |p|), the
polynomial of log1p(u) with its own roundings 3.6 (its float32 Horner steps over
u in (0, 1] against float64), the last multiply-add 1: 8 together.  1 - a =
1 - exp(-dt) adds the logarithm's scaling and back 3, its polynomial 3.6 (2.1e-7)
and a product: 16.  The slope 1 / (1 + u) or u / (1 + u): u 3.4 and at the most
once more through the sum, which is 1, a reciprocal 2, a product 1 and one with
the adjoint: 12."""
import pytest

import mamba_ssd_sequence_b200 as ssd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

U = 2.0 ** -24


def within(got, want, units, p):
    err = (got.double() - want).abs() / want / U - 0.05 * p.abs()
    assert err.max() <= units, f"{float(err.max()):.1f} of {units} roundings"


@pytest.mark.parametrize("value", ["dt", "complement"])
def test_dt(value):
    B, H, N, d = 1, 8, 1, 512
    gate = torch.linspace(-80, 20, B * H * N * d, device="cuda").view(B, H, N, d)
    p = gate.double()
    dt = torch.log1p(torch.exp(-p.abs())) + p.clamp(min=0)
    f, slope = (dt, torch.sigmoid(p)) if value == "dt" else (-torch.expm1(-dt), torch.exp(-dt) * torch.sigmoid(p))
    x = torch.ones_like(gate)
    kind = dict(value_dt=value == "dt", value_complement=value == "complement")
    states = ssd.alloc_glr_states(B, H, N, d)
    units = 8 if value == "dt" else 16
    within(ssd.ssd_glr_fwd(x, gate, None, None, states=states, **kind), f, units, p)
    h = torch.zeros(B, H, d, device="cuda")
    within(ssd.ssd_glr_step(x[:, :, 0], gate[:, :, 0], None, None, h, **kind), f[:, :, 0], units, p[:, :, 0])
    dx, dgate, *_ = ssd.ssd_glr_bwd(x, x, gate, None, None, states, **kind)
    within(dx, f, units, p)
    if value == "dt":
        within(dgate, slope, 12, p)
