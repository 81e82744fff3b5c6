"""The decay polynomial of the gated linear recurrence: the generator
reproduces the coefficients written in the CUDA source, and their float32
error bound holds."""
import os

from mamba_ssd_sequence_b200 import gen_decay_poly

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_coefficients_match_source_and_bound():
    c = gen_decay_poly.coefficients(5)
    src = open(os.path.join(ROOT, "mamba_ssd_sequence_b200", "csrc", "ssd_glr.cuh")).read()
    for v in c:
        assert f"{abs(float(v)):.9e}f" in src
    assert gen_decay_poly.max_rel_error(c) < 2.1e-7
