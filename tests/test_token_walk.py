"""The walk over a batch's tokens (csrc/ssd_view.h), compiled for the host: it
agrees with whole-number division at the largest sizes that are accepted, where
the sum of an index and a step leaves 32 bits with a sign."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LARGEST = 2 ** 31 - 65536 - 1  # tokens of a sequence


@pytest.fixture(scope="module")
def next_token(tmp_path_factory):
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        pytest.skip("needs a C++ compiler")
    d = tmp_path_factory.mktemp("walk")
    src, lib = d / "walk.cpp", d / "walk.so"
    src.write_text('#include "ssd_view.h"\n'
                   'extern "C" int walk(unsigned *n, unsigned step, unsigned N) { return ssd::next_token(*n, step, N); }\n')
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "mamba_ssd_sequence_b200", "csrc"), str(src), "-o", str(lib)], check=True)
    fn = ctypes.CDLL(str(lib)).walk
    fn.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_uint32, ctypes.c_uint32]

    def step_on(n, step, N):
        v = ctypes.c_uint32(n)
        return bool(fn(ctypes.byref(v), step, N)), v.value

    return step_on


@pytest.mark.parametrize("N,step", [
    (1, 0), (2, 1), (5, 3), (1_200_000_000, 1_080_000_128), (1_900_000_000, 380_000_000), (LARGEST, 75776), (LARGEST, LARGEST - 1)])
def test_walk_over_batches(next_token, N, step):
    rng = random.Random(N)
    for start in (0, N - 1, N // 2, N - step, rng.randrange(N)):
        m, n = start % N, start % N
        for _ in range(20):  # steps of the whole walk, over several batches
            passes, n2 = next_token(n, step, N)
            assert passes == ((m + step) // N > m // N)
            m, n = m + step, n2
            assert n == m % N
