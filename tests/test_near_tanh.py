"""CPU check of the three-term tanh that the key weights take near zero: the library's own
fit (csrc/near_tanh.h), built with the host compiler."""

import os
import shutil
import subprocess

import numpy as np
import pytest

from test_tanh_poly import _consts

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "soft_capped_attention_gb300", "csrc")
STEP = 2.0 ** -24  # half a step of fp32, relative


@pytest.fixture(scope="module")
def fit(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not available")
    d = tmp_path_factory.mktemp("near_tanh")
    (d / "fit.cc").write_text("""
#include <stdio.h>
#include <stdlib.h>
#include "near_tanh.h"
int main(int, char** a) {
  float c[3];
  capattn::near_tanh_fit(atof(a[1]), atof(a[2]), c);
  printf("%.17g %.9g %.9g %.9g\\n", capattn::kNearTanh, c[0], c[1], c[2]);
}
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(d / "fit.cc"), "-o", str(d / "fit")], check=True)

    def run(cap, arg):
        x = subprocess.run([str(d / "fit"), repr(cap), repr(arg)], check=True, capture_output=True, text=True).stdout.split()
        return float(x[0]), np.array(x[1:], dtype=np.float32).astype(np.float64)

    return run


def relative_error(c, top, cap, arg):
    X = np.linspace(0, top / arg, 200_001)[1:]
    z = X * X
    q = np.zeros_like(X)
    for x in c[::-1]:
        q = q * z + x
    return np.abs(X * q / (cap * np.tanh(arg * X)) - 1).max()


@pytest.mark.parametrize("cap, arg", [(1.0, 1.0), (50.0, 0.08838834764831845 / 50), (5.0, 0.125 / 5), (300.0, 1e-4)])
def test_the_three_terms_are_no_worse_than_the_five(fit, cap, arg):
    """Coefficients rounded to fp32 add half a step at most (the first one's weight is 1,
    the others' below w = u^2)."""
    top, c = fit(cap, arg)
    five, _ = _consts()
    in64 = [1.0, *five.astype(np.float64)]
    worst = relative_error(np.array(in64), top, 1.0, 1.0)
    assert worst < 3e-8
    assert relative_error(c, top, cap, arg) <= worst + 1.03 * STEP
    assert relative_error(c, top, cap, arg) < 1.4 * STEP
