"""The acceptance kernel's integer residuals (csrc/residual.cuh, compiled for the host with the same
roundings) against rational arithmetic."""
import ctypes
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
FROM_P, MINUS_Q, MINUS_AQ = 0, 1, 2


@pytest.fixture(scope="module")
def probe():
    from mla_speculative_verify_attention_gb300 import build
    out_dir = os.path.join(HERE, "_build")
    os.makedirs(out_dir, exist_ok=True)
    lib = os.path.join(out_dir, "libresidual_probe.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC,-ffp-contract=off", "-o",
                    lib, os.path.join(HERE, "csrc", "residual_probe.cu")], check=True)
    L = ctypes.CDLL(lib)
    P = ctypes.c_void_p
    L.residual_units.argtypes, L.residual_units.restype = [ctypes.c_int, ctypes.c_double, P, P, ctypes.c_longlong, P], None
    L.residual_sum8.argtypes, L.residual_sum8.restype = [ctypes.c_double, P, P], ctypes.c_longlong
    L.residual_unit.restype = ctypes.c_double
    return L


def units(L, form, A, p, q):
    p, q = np.ascontiguousarray(p, np.float32), np.ascontiguousarray(q, np.float32)
    out = np.zeros(len(p), np.int64)
    L.residual_units(form, A, p.ctypes.data, q.ctypes.data, len(p), out.ctypes.data)
    return out


def pairs(rng, n, kind):
    """n (p, q) in [0, 1] as fp32."""
    if kind == "uniform":
        return rng.random(n).astype(np.float32), rng.random(n).astype(np.float32)
    if kind == "below":                                # q below p: every residual above zero at A = 1
        p = rng.random(n)
        return p.astype(np.float32), (p * rng.random(n)).astype(np.float32)
    if kind == "large":                                # p near 1, where the leading part is often a tie
        return rng.uniform(0.75, 1.0, n).astype(np.float32), rng.uniform(0.0, 0.2, n).astype(np.float32)
    if kind == "close":                                # p within a few steps of q
        q = rng.random(n).astype(np.float32)
        return (q * (1 + rng.integers(-3, 4, n) * 2.0 ** -23)).astype(np.float32).clip(0, 1), q
    p, q = (np.exp(rng.uniform(np.log(1e-12), 0.0, n)).astype(np.float32) for _ in range(2))
    return p, q


# Every element is within one unit of max(p - A q, 0): half a unit where the trailing part is rounded
# to an integer, and less than another half for the fp32 operations before it.  Those round, with p and
# A q in [0, 1] wherever the residual is positive: the product's remainder (2^-24 at most, to 2^-49), that
# remainder off the difference's (2^-23, to 2^-47), the sum with the leading part's remainder (2^-22, to
# 2^-46), and A to 48 bits (2^-48 of A q).  Together below 2^-45, half of the unit 2^-44.
@pytest.mark.parametrize("kind", ["uniform", "below", "large", "close", "log"])
@pytest.mark.parametrize("form,A", [(FROM_P, 0.0), (MINUS_Q, 1.0), (MINUS_AQ, 1.0), (MINUS_AQ, 1.37), (MINUS_AQ, 1.0000001),
                                    (MINUS_AQ, 1.9999999), (MINUS_AQ, 2.718281828459045), (MINUS_AQ, 17.3)])
def test_every_element_is_within_a_unit(probe, kind, form, A):
    rng = np.random.default_rng(int(1000 * A) + 7 * form + len(kind))
    p, q = pairs(rng, 4000, kind)
    got = units(probe, form, A, p, q)
    unit, a = Fraction(probe.residual_unit()), Fraction(A)
    worst = Fraction(0)
    for x, y, g in zip(p.tolist(), q.tolist(), got.tolist()):
        exact = max(Fraction(x) - (a * Fraction(y) if form != FROM_P else 0), Fraction(0))
        worst = max(worst, abs(g - exact / unit))
    assert worst <= 1, float(worst)


def test_forms_agree(probe):
    """The search for the next token sums in the one general form what the passes summed in theirs."""
    rng = np.random.default_rng(5)
    for kind in ("uniform", "large", "close", "log"):
        p, q = pairs(rng, 2000, kind)
        zero = np.zeros_like(q)
        assert np.array_equal(units(probe, MINUS_Q, 1.0, p, q), units(probe, MINUS_AQ, 1.0, p, q))
        for A in (0.0, 1.0, 1.7):
            assert np.array_equal(units(probe, FROM_P, 0.0, p, zero), units(probe, MINUS_AQ, A, p, zero))


def test_sums_are_the_elements_sums(probe):
    rng = np.random.default_rng(6)
    for A in (1.0, 1.25, 2.9):
        for kind in ("uniform", "below", "large", "log"):
            p, q = pairs(rng, 800, kind)
            one = units(probe, MINUS_AQ, A, p, q)
            for i in range(0, 800, 8):
                x, y = np.ascontiguousarray(p[i:i + 8]), np.ascontiguousarray(q[i:i + 8])
                assert probe.residual_sum8(A, x.ctypes.data, y.ctypes.data) == one[i:i + 8].sum()


def test_ends_of_the_range(probe):
    whole = round(1 / probe.residual_unit())
    one, zero = np.ones(1, np.float32), np.zeros(1, np.float32)
    for form, A in ((FROM_P, 0.0), (MINUS_Q, 1.0), (MINUS_AQ, 1.0), (MINUS_AQ, 3.3)):
        assert units(probe, form, A, one, zero)[0] == whole and units(probe, form, A, zero, zero)[0] == 0
    for A in (1.0, 1.5, 40.0):
        assert units(probe, MINUS_AQ, A, one, one)[0] == 0 and units(probe, MINUS_AQ, A, zero, one)[0] == 0
