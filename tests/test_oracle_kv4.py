"""Pins of the oracle's 4-bit cache: code values, rounding, layout, attention."""
from fractions import Fraction

import numpy as np
import pytest

import oracle


def test_e2m1_values_by_the_format():
    """1 sign, 2 exponent (bias 1) and 1 mantissa bit; exponent 0 is subnormal."""
    for code in range(16):
        e, m = code >> 1 & 3, code & 1
        value = Fraction(m, 2) if e == 0 else Fraction(2 + m, 2) * 2 ** (e - 1)
        assert oracle.e2m1_to_f64([code])[0] == (-1 if code & 8 else 1) * float(value)


def test_e2m1_rounding_by_search():
    grid = [Fraction(x) for x in (0, Fraction(1, 2), 1, Fraction(3, 2), 2, 3, 4, 6)]
    for n in range(-64 * 9, 64 * 9 + 1):
        y = Fraction(n, 64)
        a = min(abs(y), Fraction(6))
        best = min(abs(a - x) for x in grid)
        want = [c for c, x in enumerate(grid) if abs(a - x) == best]
        got = int(oracle.e2m1_nearest(float(y)))
        assert got & 7 in want and (len(want) == 1 or got % 2 == 0), y
        assert (got >> 3) == (y < 0)
    assert int(oracle.e2m1_nearest(np.inf)) == 7 and int(oracle.e2m1_nearest(-np.inf)) == 15
    assert int(oracle.e2m1_nearest(-0.0)) == 8


def test_quantize_blocks():
    x = np.zeros(48)
    x[3], x[17], x[40] = 6.0, -3.0, np.nan
    codes, scales = oracle.kv4_quantize(x, 1.0)
    # max 6: scale 1 (E4M3 0x38); max 3: scale .5 (0x30), -3 is -6 of it; a NaN: scale NaN
    assert list(scales) == [0x38, 0x30, 0x7F]
    assert codes[3] == 7 and codes[17] == 15 and not codes[:3].any()
    v = oracle.kv4_values(codes, scales, 1.0)
    assert np.array_equal(v[:32], x[:32]) and np.isnan(v[32:]).all()
    # below half the smallest scale: all zero
    codes, scales = oracle.kv4_quantize(np.full(16, 6 * 2.0 ** -11), 1.0)
    assert not codes.any() and not scales.any()
    # beyond the largest: saturated
    codes, scales = oracle.kv4_quantize(np.full(16, 1e9), 1.0)
    assert (codes == 7).all() and scales[0] == 0x7E
    # the factor stands in front of the scale
    a, b = oracle.kv4_quantize(x[:32], 1.0), oracle.kv4_quantize(4 * x[:32], 4.0)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_quantize_error_is_half_a_step():
    x = np.random.default_rng(1).standard_normal((500, 64))
    codes, scales = oracle.kv4_quantize(x, 0.25)
    v = oracle.kv4_values(codes, scales, 0.25)
    top = np.repeat(np.abs(x.reshape(500, 4, 16)).max(-1), 16, axis=-1).reshape(500, 64)
    # the widest step is 2 of 6 units, half of it 1 / 6 of the unit's share; the scale itself is
    # off by at most 2^-4, which moves a saturated value by 2^-4 of the largest
    assert np.all(np.abs(v - x) <= top * (1 / 6 * (1 + 2.0 ** -4) + 1e-12))


@pytest.mark.parametrize("D,page", [(64, 16), (128, 48), (128, 64)])
def test_store_and_load(D, page):
    rng = np.random.default_rng(D + page)
    Hkv, n = 3, 100
    pages = rng.integers(0, 256, (12, Hkv, page // 16, 18 * D)).astype(np.uint8)
    table = rng.permutation(12)[None, :-(-n // page)]
    want = {}
    for pos in rng.permutation(n):
        for h in range(Hkv):
            for which in (0, 1):
                want[pos, h, which] = (rng.integers(0, 16, D).astype(np.uint8),
                                       rng.integers(0, 256, D // 16).astype(np.uint8))
                oracle.kv4_store(pages, table, page, 0, int(pos), h, which, *want[pos, h, which])
    for h in range(Hkv):
        for which in (0, 1):
            codes, scales = oracle.kv4_load(pages, table, page, 0, n, h, which)
            for pos in range(n):
                assert np.array_equal(codes[pos], want[pos, h, which][0])
                assert np.array_equal(scales[pos], want[pos, h, which][1])


def test_layout_by_hand():
    """Token 17 of a page of 32, head 1, element 5 of K and V: byte offsets counted out."""
    D = 64
    pages = np.zeros((1, 2, 2, 18 * D), np.uint8)
    codes, scales = np.zeros(D, np.uint8), np.zeros(D // 16, np.uint8)
    codes[5], scales[2] = 9, 77
    oracle.kv4_store(pages, np.array([[0]]), 32, 0, 17, 1, 0, codes, scales)
    oracle.kv4_store(pages, np.array([[0]]), 32, 0, 17, 1, 1, codes, scales)
    flat = pages.reshape(-1)
    base = (1 * 2 + 1) * 18 * D                # head 1, slab 1
    at = {base + 1 * 32 + 2: 9 << 4, base + 16 * 32 + 1 * 4 + 2: 77,
          base + 16 * 36 + 1 * 32 + 2: 9 << 4, base + 16 * 36 + 16 * 32 + 1 * 4 + 2: 77}
    assert {int(i): int(flat[i]) for i in flat.nonzero()[0]} == at


def test_attention_against_unpaged_attention():
    """The same values in a contiguous fp32 cache through the unpaged oracle."""
    rng = np.random.default_rng(3)
    B, Hq, Hkv, D, page = 3, 4, 2, 64, 16
    kv_len, rows = np.array([0, 37, 20]), [2, 3, 1]
    cu = np.concatenate([[0], np.cumsum(rows)])
    need = [-(-(int(n) + r) // page) for n, r in zip(kv_len, rows)]
    table = np.full((B, max(need)), -1)
    ids = iter(rng.permutation(sum(need)))
    for i, n in enumerate(need):
        table[i, :n] = [next(ids) for _ in range(n)]
    # random bytes, scales kept to ordinary ones
    pages = rng.integers(0, 256, (sum(need), Hkv, 1, 18 * D)).astype(np.uint8)
    for at in (8 * D, 17 * D):
        pages[..., at:at + D] = rng.integers(0x28, 0x48, (*pages.shape[:3], D))
    q = rng.standard_normal((cu[-1], Hq, D)).astype(np.float32)
    out, mag, _, _ = oracle.kv4_attention(q, pages, table, page, cu, kv_len, k_scale=0.5, v_scale=2.0)
    K, V, kn, vn, start = [], [], [], [], []
    for i in range(B):
        n, r = int(kv_len[i]), rows[i]
        k = np.stack([oracle.kv4_values(*oracle.kv4_load(pages, table, page, i, n + r, h, 0), 0.5)
                      for h in range(Hkv)], 1).astype(np.float32)
        v = np.stack([oracle.kv4_values(*oracle.kv4_load(pages, table, page, i, n + r, h, 1), 2.0)
                      for h in range(Hkv)], 1).astype(np.float32)
        start.append(sum(len(x) for x in K))
        K.append(k[:n]), V.append(v[:n]), kn.append(k[n:]), vn.append(v[n:])
    want = oracle.verify_attention(q, np.concatenate(kn), np.concatenate(vn), np.concatenate(K),
                                   np.concatenate(V), cu, start, kv_len, Hkv,
                                   scale=np.float32(1 / np.sqrt(D)))
    assert np.allclose(out, want, rtol=1e-6, atol=1e-9)
    assert np.all(mag >= np.abs(out) - 1e-12)


def test_head_norm():
    x = np.array([3.0, -4.0])
    assert np.allclose(oracle.head_norm(x, [1, 1], 0.0), x / np.sqrt(12.5))
    assert np.allclose(oracle.head_norm(x, [0.5, 1], 2.0, 1.0), x / np.sqrt(14.5) * [1.5, 2])
    y = oracle.head_norm(np.random.default_rng(0).standard_normal((7, 128)), np.ones(128), 0.0)
    assert np.allclose((y * y).mean(-1), 1)
