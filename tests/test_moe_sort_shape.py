"""How the sort of router choices is spread over a cluster: the rule that the
library's launch takes, compiled for the host.  A device that cannot place
sixteen CTAs of a cluster gets eight, and every slot has a place."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gemm_quantize_b200", "csrc")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
SOURCE = """
#include "moe.h"
extern "C" void shape(int n, int most, int* out) {
    const auto s = w4a8::moe::sort_shape(n, most);
    out[0] = s.ctas, out[1] = s.per_cta, out[2] = s.keep;
}
"""


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    d = tmp_path_factory.mktemp("shape")
    (d / "shape.cpp").write_text(SOURCE)
    so = str(d / "shape.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-I", os.path.join(CUDA, "include"),
                    str(d / "shape.cpp"), "-o", so], check=True)
    fn = ctypes.CDLL(so).shape

    def call(n, most):
        out = (ctypes.c_int * 3)()
        fn(n, most, out)
        return tuple(out)

    return call


@pytest.mark.parametrize("most", [8, 16])
@pytest.mark.parametrize("n", [0, 1, 31, 1024, 1025, 8192, 8193, 16384, 16385, 131072, 196608, 196609, 393216, 393217,
                               500000, (1 << 31) - 256])
def test_every_slot_has_a_place(shape, n, most):
    ctas, per_cta, keep = shape(n, most)
    assert ctas in (1, 2, 4, 8, 16) and ctas <= most
    assert ctas == 1 or n > ctas // 2 * 1024  # no more than the slots ask for
    assert ctas == most or n <= ctas * 1024
    assert per_cta % 32 == 0 and ctas * per_cta >= n
    # the CTAs' pieces are whole steps of 32 slots, and none is longer than what it keeps
    steps = (n + 31) // 32
    assert max((steps * (r + 1) // ctas - steps * r // ctas) * 32 for r in range(ctas)) <= per_cta
    assert keep == (per_cta <= 24576)


def test_eight_where_sixteen_cannot_be_placed(shape):
    assert shape(131072, 16) == (16, 8192, 1)
    assert shape(131072, 8) == (8, 16384, 1)
    assert shape(393216, 16) == (16, 24576, 1)
    assert shape(393216, 8) == (8, 49152, 0)
