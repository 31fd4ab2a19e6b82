"""CPU check of the soft-sign cap's polynomial near zero: the library's own fit
(csrc/near_soft_sign.h), built with the host compiler."""

import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "soft_capped_attention_gb300", "csrc")
STEP = 2.0 ** -24  # half a step of fp32, relative


@pytest.mark.parametrize("cap, scale", [(20.0, 0.08838834764831845), (1.0, 1.0), (3.0, 0.125), (300.0, 1e-3), (20.0, -0.1)])
def test_near_soft_sign(tmp_path, cap, scale):
    """Interpolation at n = 7 Chebyshev nodes of [0, R]: |1 / (1 + w) - p| is at most
    2 (R / 4)^n / (1 + w)^(n + 1) / ..., below 2.2e-8 relative here; the coefficients' roundings
    add half a step of each term, and the terms' sizes sum to 1 / (1 - R) of the first."""
    if shutil.which("g++") is None:
        pytest.skip("g++ is not available")
    (tmp_path / "fit.cc").write_text("""
#include <stdio.h>
#include <stdlib.h>
#include "near_soft_sign.h"
int main(int, char** a) {
  float c[7];
  capattn::near_soft_sign_fit(atof(a[1]), atof(a[2]), c);
  printf("%.17g", capattn::kNearSoftSign);
  for (float x : c) printf(" %.9g", x);
}
""")
    exe = tmp_path / "fit"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(tmp_path / "fit.cc"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe), repr(cap), repr(scale)], check=True, capture_output=True, text=True).stdout.split()
    top, c = float(out[0]), np.array(out[1:], dtype=np.float32).astype(np.float64)
    X = np.linspace(0, top * cap / abs(scale), 200_001)[1:]
    q = np.zeros_like(X)
    for x in c[::-1]:
        q = q * X + x
    s = scale * X
    want = s / (1 + np.abs(s) / cap)
    assert np.abs(X * q / want - 1).max() <= 2.2e-8 + STEP * (1 + top) / (1 - top)
