"""The constants of the linear layer's epilogue against what they stand for (CPU only)."""

import os
import re

import numpy as np
import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "transformer_block_gb300", "csrc", "linear_gemm.cuh")


def test_normal_tail_fit():
    # Phi(-a) exp(a^2 / 2) = erfcx(a / sqrt 2) / 2 = t P(t), t = 1 / (1 + a / 4), for a up to 14:
    # the fit's 5.7e-8, and the coefficients' rounding to float32: 2^-25 sum |c_k| t^k / P(t), which
    # is largest at t = 1 with 2^-25 x 1.217 / 0.5 = 7.3e-8; evaluated in float64
    special = pytest.importorskip("scipy.special")
    body = open(SRC).read().split("phi_terms(float")[1].split("uint64_t t =")[0]
    coef = [float(c) for c in re.search(r"kP\[9\] = \{([^}]*)\}", body)[1].replace("f", "").split(",")]
    assert len(coef) == 9 and "f2(0.25f, 0.25f)" in body
    a = np.linspace(0, 14, 100001)
    t = 1 / (1 + a / 4)
    p = np.polynomial.polynomial.polyval(t, np.float32(coef).astype(np.float64))
    want = special.erfcx(a / np.sqrt(2)) / 2
    assert np.abs(t * p / want - 1).max() <= 5.7e-8 + 7.3e-8
    half = float(re.search(r"kHalfLog2e = ([0-9.]+)f", body)[1])
    assert np.float32(half) == np.float32(np.log2(np.e) / 2)


@pytest.mark.parametrize("name", ["qk_rope.cu", "linear.cu", "linear_gemm.cuh", "adamw.cu"])
def test_dependent_launches_read_coherently(name):
    # These kernels may begin while the launch before them still writes what they read. A load
    # through the read-only path is defined only for what nothing writes while the kernel lives.
    body = open(os.path.join(os.path.dirname(SRC), name)).read()
    assert "launch_dependent(" in body
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in body, (name, word)
