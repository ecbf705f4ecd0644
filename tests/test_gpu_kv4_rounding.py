"""Scales and codes of spec_kv4_append next to their ties, for fp32 rows that enter the pages as they
are.  A scale is the E4M3 of the quotient m / (6 f) rounded to fp32, a code the E2M1 of the fp32 quotient
x / (s f): both are compared with the quotients of CUDA's own division, rounded by the oracle.  (Where f is
a power of two that is the nearest scale and code to the real quotients.)"""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev

pytestmark = pytest.mark.gpu

E4 = oracle.sampling.e4m3_to_f64(np.arange(127, dtype=np.uint8))
TIES = (oracle.kv4.E2M1[:-1] + oracle.kv4.E2M1[1:]) / 2
FACTORS = [1.0, 2.0 ** -7, 2.0 ** 64, 2.0 ** -64, 5.0, 0.75, 0.7, 1.0 / 3.0, 1.1e-5, 7.3e9]


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


def steps(x, by):
    """fp32 values some steps from x."""
    return (x.astype(np.float32).view(np.int32) + by).view(np.float32)


def stored(api, x, f):
    """(codes, scales) of fp32 rows x [R, 64] as K and as V of one head."""
    R, D, page = x.shape[0], 64, 64
    n = -(-R // page)
    cache = api.Kv4Cache(n, 1, D, page_size=page, k_scale=f, v_scale=f)
    rows = dev(x)[:, None].contiguous()
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    api.spec_kv4_append(api.kv4_append_args(cache, table, dev(np.array([0, R], np.int32)),
                                            dev(np.zeros(1, np.int32)), rows, rows.clone(), max_q_rows=R))
    torch.cuda.synchronize()
    pages, where = cache.pages.cpu().numpy(), table.cpu().numpy()
    k, v = (oracle.kv4_load(pages, where, page, 0, R, 0, which) for which in (0, 1))
    assert np.array_equal(k[0], v[0]) and np.array_equal(k[1], v[1])
    return k


def divided(a, b):
    """CUDA's fp32 quotient."""
    return (dev(a.astype(np.float32)) / dev(np.broadcast_to(b, a.shape).astype(np.float32))).cpu().numpy()


@pytest.mark.parametrize("f", FACTORS)
def test_scales_next_to_their_ties(api, f):
    f = np.float32(f)
    m = ((E4[:-1] + E4[1:]) / 2)[:, None] * 6 * np.float64(f)
    m = steps(np.broadcast_to(m, (126, 9)), np.arange(-4, 5, dtype=np.int32)).reshape(-1)
    x = np.zeros((m.size, 64), np.float32)
    x[:, 0:64:16] = m[:, None] * np.array([1, -1, 1, -1], np.float32)
    x[:, 5::16] = x[:, 0::16] / 3
    _, scales = stored(api, x, float(f))
    q = (m.astype(np.float64) / (6 * np.float64(f))).astype(np.float32)     # (6 f is exact in fp64)
    want = oracle.e4m3_nearest(q.astype(np.float64))
    assert np.array_equal(scales, np.repeat(want[:, None], 4, 1)), np.argwhere(scales != want[:, None])[:4]
    if np.float32(6) * f == 6 * np.float64(f):
        assert np.array_equal(divided(m, np.float32(6) * f), q)
    if np.log2(f) % 1 == 0:
        assert np.array_equal(want, oracle.e4m3_nearest(m.astype(np.float64) / (6 * np.float64(f))))


@pytest.mark.parametrize("f", FACTORS)
def test_codes_next_to_their_ties(api, f):
    """The largest of a block is 6 units, the others are ties of a code's units and a few steps beside them."""
    f = np.float32(f)
    unit = (E4[1:126].astype(np.float32) * f).astype(np.float32)
    x = np.zeros((125, 64), np.float32)
    near = steps(np.float64(unit)[:, None, None] * TIES[:, None], np.arange(-4, 5, dtype=np.int32)).reshape(125, 63)
    x[:, np.arange(64) % 16 != 0] = near[:, :60] * np.where(np.arange(60) % 2, -1, 1).astype(np.float32)
    x[:, 0::16] = 6 * np.float64(unit)[:, None]
    codes, scales = stored(api, x, float(f))
    assert np.array_equal(scales, np.repeat(np.arange(1, 126, dtype=np.uint8)[:, None], 4, 1))
    want = oracle.e2m1_nearest(divided(x, unit[:, None]).astype(np.float64))
    assert np.array_equal(codes, want), np.argwhere(codes != want)[:4]
    if np.log2(f) % 1 == 0:
        assert np.array_equal(want, oracle.e2m1_nearest(x.astype(np.float64) / unit[:, None]))


def test_scales_at_the_ends(api):
    """Quotients that overflow or saturate, the smallest ones, and NaN."""
    for f, m, want in ((2.0 ** -64, 3e38, 0x7E), (1.0, 3e38, 0x7E), (1.0, float("inf"), 0x7E), (1.0, 6 * 448.0, 0x7E),
                       (1.0, 6 * 464.0, 0x7E), (1.0, 6 * 500.0, 0x7E), (1.0, 6 * 2.0 ** -9, 1), (1.0, 6 * 2.0 ** -10, 0),
                       (2.0 ** 64, 1e-38, 0), (1.0, float("nan"), 0x7F), (1.0, 1e-45, 0)):
        x = np.zeros((1, 64), np.float32)
        x[0, 0::16] = m
        _, scales = stored(api, x, f)
        assert (scales & 0x7F == want).all(), (f, m, scales)
