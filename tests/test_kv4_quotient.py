"""The quotients behind the 4-bit codes (csrc/kv4_quotient.inl), compiled for the host and compared with
the compiler's division: within a step of it for any reciprocal within two steps, equal next to the ties of
codes, where a step would show."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
UNITS = oracle.sampling.e4m3_to_f64(np.arange(1, 126, dtype=np.uint8)).astype(np.float32)
TIES = (oracle.kv4.E2M1[:-1] + oracle.kv4.E2M1[1:]) / 2
FACTORS = [1.0, 2.0 ** -64, 2.0 ** 64, 2.0 ** 17, 3.0, 0.3, 0.7, 1.0 / 3.0, 1.9999999, 1.1e-9, 7.3e12]

DRIVER = r"""
#include <cmath>
#include <cstddef>
#include "kv4_quotient.inl"
struct One {
  typedef float T;
  static float mul(float a, float b) { return a * b; }
  static float fma(float a, float b, float c) { return std::fma(a, b, c); }
};
extern "C" void quotients(size_t n, const float *x, const float *d, int off, float *q, float *divided) {
  for (size_t i = 0; i < n; ++i) {
    float near = 1.0f / d[i];
    for (int k = 0; k < std::abs(off); ++k) near = std::nextafter(near, off > 0 ? INFINITY : -INFINITY);
    const float y = sv::refined_reciprocal<One>(-d[i], near, 1.0f);
    q[i] = sv::corrected_quotient<One>(x[i], -d[i], y);
    divided[i] = x[i] / d[i];
  }
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    at = tmp_path_factory.mktemp("quotient")
    (at / "q.cpp").write_text(DRIVER)
    csrc = os.path.join(ROOT, "speculative_decoding_verify_09_gb300", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                        csrc, "-o", str(at / "q.so"), str(at / "q.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(at / "q.so"))


def quotients(host, x, d, off):
    x, d = (np.ascontiguousarray(np.broadcast_to(a, np.broadcast_shapes(x.shape, d.shape)), np.float32)
            for a in (x, d))
    q, divided = np.empty_like(x), np.empty_like(x)
    ptr = [a.ctypes.data_as(ctypes.c_void_p) for a in (x, d, q, divided)]
    host.quotients(ctypes.c_size_t(x.size), ptr[0], ptr[1], off, ptr[2], ptr[3])
    return x, d, q, divided


@pytest.mark.parametrize("off", [-2, -1, 0, 1, 2])
@pytest.mark.parametrize("f", FACTORS)
def test_next_to_ties(host, f, off):
    """Codes are those of the division, and of the real quotient where the factor is a power of two.  The
    reciprocal is within a step, 2^-23 of 1 / d, and the remainder within d times a step of q, so that the
    correction is off by 2^-23 of a step (and fp64 by far less): where the real quotient is nearer than 2^-22
    of a step to the middle between a tie and its neighbour, either one is its rounding."""
    unit = (UNITS * np.float32(f)).astype(np.float32)[:, None, None]
    x = (unit.astype(np.float64) * TIES[:, None]).astype(np.float32)
    x = (np.broadcast_to(x, (125, 7, 17)).view(np.int32) + np.arange(-8, 9, dtype=np.int32)).view(np.float32)
    x, d, q, divided = quotients(host, x, unit, off)
    codes = oracle.e2m1_nearest(q.astype(np.float64))
    real, tie = x.astype(np.float64) / d, np.broadcast_to(TIES[:, None], x.shape)
    step = np.abs(np.nextafter(tie.astype(np.float32), np.where(real < tie, 0, 9).astype(np.float32)) - tie)
    middle = np.abs(np.abs(real - tie) / step - 0.5) < 2.0 ** -22
    assert np.array_equal(codes[~middle], oracle.e2m1_nearest(divided.astype(np.float64))[~middle])
    assert f > 1.5 and f < 2 or not middle.any()
    if np.log2(f) % 1 == 0:
        assert np.array_equal(codes, oracle.e2m1_nearest(x.astype(np.float64) / d))


@pytest.mark.parametrize("off", [-2, -1, 0, 1, 2])
def test_any_quotients(host, off):
    rng = np.random.default_rng(off + 2)
    f = np.exp2(rng.uniform(-64, 64, 400)).astype(np.float32)
    unit = (rng.choice(UNITS, 400) * f).astype(np.float32)[:, None]
    x = (unit * rng.uniform(-6.5, 6.5, (400, 500))).astype(np.float32)
    x[:, 0] = 0
    _, _, q, divided = quotients(host, x, unit, off)
    away = np.abs(q.view(np.int32) - divided.view(np.int32))
    assert away.max() <= 1 and (away > 0).mean() < 1e-3
