"""Pins of the rotary oracle and of the host-side frequency table (no GPU)."""
import ctypes
import math

import numpy as np
import pytest

import oracle


def test_pairs_turn_by_hand_values():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0, 6.0]]])
    f = np.array([math.pi / 2, math.pi / 4])
    c = math.sqrt(0.5)
    half = oracle.rope_rows(x, [1], f, "half")[0, 0]
    assert np.allclose(half, [-3, c * (2 - 4), 1, c * (2 + 4), 5, 6])
    inter = oracle.rope_rows(x, [1], f, "interleaved")[0, 0]
    assert np.allclose(inter, [-2, 1, c * (3 - 4), c * (3 + 4), 5, 6])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_dot_products_depend_on_the_distance_alone(layout):
    rng = np.random.default_rng(3)
    f, _ = oracle.rope_frequencies(32)
    q, k = rng.standard_normal((2, 1, 1, 48))

    def dot(m, n):
        return float((oracle.rope_rows(q, [m], f, layout) * oracle.rope_rows(k, [n], f, layout)).sum())

    for m, n, s in ((5, 2, 1000), (0, 7, 123456), (40, 40, 2 ** 30)):
        assert abs(dot(m, n) - dot(m + s, n + s)) < 1e-9
    assert abs(dot(5, 2) - dot(6, 2)) > 1e-3


def test_negative_position_is_the_transpose():
    rng = np.random.default_rng(4)
    f, _ = oracle.rope_frequencies(16)
    x, g = rng.standard_normal((2, 1, 1, 20))
    y = oracle.rope_rows(x, [77], f, "half", 1.3)
    back = oracle.rope_rows(g, [-77], f, "half", 1.3)
    assert abs(float((y * g).sum() - (x * back).sum())) < 1e-12
    # and by differences
    for e in range(20):
        d = x.copy()
        d[..., e] += 1e-6
        slope = ((oracle.rope_rows(d, [77], f, "half", 1.3) - y) * g).sum() / 1e-6
        assert abs(slope - back[0, 0, e]) < 1e-6


def test_angles_of_far_positions():
    # one eighth of a turn per token, exactly: every eighth position is a whole turn
    f = np.array([2 * math.pi / 8])
    a = oracle.rope.angles([0, 1, 8, 8 * 10 ** 8 + 1, -1], f)[:, 0]
    assert np.allclose(a, [0, math.pi / 4, 0, math.pi / 4, -math.pi / 4], atol=1e-7)


def test_frequencies_at_their_ends():
    plain, m = oracle.rope_frequencies(64)
    assert m == 1.0 and plain[0] == 1.0 and abs(plain[-1] - 10000.0 ** (-62 / 64)) < 1e-18
    lin, _ = oracle.rope_frequencies(64, kind="linear", factor=4.0)
    assert np.allclose(lin, plain / 4, rtol=1e-15)
    ntk, _ = oracle.rope_frequencies(64, kind="ntk", factor=4.0)
    assert ntk[0] == 1.0 and abs(ntk[-1] / (plain[-1] / 4) - 1) < 1e-12    # the slowest by factor
    yarn, m = oracle.rope_frequencies(128, kind="yarn", factor=8.0, trained=8192)
    p128, _ = oracle.rope_frequencies(128)
    assert abs(m - (0.1 * math.log(8) + 1)) < 1e-15
    turns = 8192 * p128 / (2 * math.pi)
    assert np.allclose(yarn[turns > 40], p128[turns > 40], rtol=1e-15)
    assert np.allclose(yarn[turns < 0.8], p128[turns < 0.8] / 8, rtol=1e-15)
    band, _ = oracle.rope_frequencies(128, kind="banded", factor=8.0, trained=8192)
    assert np.allclose(band[turns > 4], p128[turns > 4], rtol=1e-15)
    assert np.allclose(band[turns < 1], p128[turns < 1] / 8, rtol=1e-15)
    assert np.all(np.diff(band) < 0) and np.all(np.diff(yarn) < 0)


def test_e4m3_rounding_against_torch():
    import torch
    rng = np.random.default_rng(5)
    y = np.concatenate([rng.standard_normal(4000) * s for s in (1e-3, 0.1, 3.0, 200.0)])
    y = y.astype(np.float32).astype(np.float64)
    y = y[np.abs(y) <= 448]
    grid = oracle.sampling.e4m3_to_f64(np.arange(0x7F, dtype=np.uint8))
    y = np.concatenate([y, (grid[1:] + grid[:-1]) / 2, grid, -grid])     # ties and values
    want = torch.from_numpy(y.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.e4m3_nearest(y), want)
    got = oracle.e4m3_nearest(np.array([500.0, -1e9, np.inf, -np.inf, np.nan]))
    assert got.tolist() == [0x7E, 0xFE, 0x7E, 0xFE, 0x7F]


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


@pytest.mark.parametrize("rot", [2, 4, 20, 64, 128, 256])
@pytest.mark.parametrize("kind", ["plain", "linear", "ntk", "yarn", "banded"])
@pytest.mark.parametrize("base,factor,trained", [(10000.0, 8.0, 8192), (500000.0, 1.0, 4096),
                                                 (1e6, 32.0, 131072), (2.0, 3.5, 1)])
def test_host_table_matches_the_oracle(api, rot, kind, base, factor, trained):
    """Entries are f / (2 pi) as a 64-bit fraction.  The double arithmetic of
    the two sides (pow, log, about ten operations of relative error 2^-53, pow's
    exponent up to ln(base) + rot / (rot - 2) ln(factor) < 30 amplifying it) agrees within
    1e-14 relative, and the entry is rounded to an integer."""
    f, m = oracle.rope_frequencies(rot, base, kind, factor, trained)
    turns, mscale = api.rope_turns(rot, base=base, scaling=kind, factor=factor,
                                   trained_len=trained, device="cpu")
    got = turns.numpy().view(np.uint64).astype(np.float64)
    want = np.ldexp(f / (2 * math.pi), 64)
    assert np.all(np.abs(got - want) <= 1e-14 * want + 1.0)
    assert abs(mscale - m) <= 2.0 ** -24 * m


@pytest.mark.parametrize("kw", [
    dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=258), dict(rot_dim=8, base=1.0),
    dict(rot_dim=8, base=float("nan")), dict(rot_dim=8, scaling="linear", factor=0.5),
    dict(rot_dim=8, scaling="ntk", factor=float("inf")),
    dict(rot_dim=8, scaling="yarn", factor=2.0, trained_len=0),
    dict(rot_dim=8, scaling="yarn", factor=2.0, trained_len=9, beta_fast=1.0, beta_slow=2.0),
    dict(rot_dim=8, scaling="banded", factor=2.0, trained_len=9, low_freq=4.0, high_freq=4.0),
    dict(rot_dim=4, scaling="ntk", base=1e200, factor=1e200),
])
def test_host_table_refusals(api, kw):
    from speculative_decoding_verify_09_gb300 import _binding
    with pytest.raises(_binding.SpecVerifyError) as e:
        api.rope_turns(kw.pop("rot_dim"), device="cpu", **kw)
    assert e.value.status == _binding.SV_ERR_INVALID and "rope turns" in str(e.value)
    with pytest.raises(ValueError):
        api.rope_turns(8, scaling="other", device="cpu")


def test_host_table_null_arguments(api):
    from speculative_decoding_verify_09_gb300 import _binding as b
    sc = b.RopeScaling(0, 1, 10000.0, 1.0)
    out = (ctypes.c_uint64 * 4)()
    assert b.lib.sv_rope_turns(None, 8, out, None) == b.SV_ERR_INVALID
    assert b.lib.sv_rope_turns(ctypes.byref(sc), 8, None, None) == b.SV_ERR_INVALID
    assert b.lib.sv_rope_turns(ctypes.byref(sc), 8, out, None) == b.SV_OK
    sc.kind = 5
    assert b.lib.sv_rope_turns(ctypes.byref(sc), 8, out, None) == b.SV_ERR_INVALID
