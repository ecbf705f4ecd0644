"""Attention over the paged 4-bit cache at the ends of its operands' ranges.

Weights enter the product with V as f16.  Held here: 2^-11 relative for weights down to 2^-21 of a row's
largest, and below that an error of at most 2^-32 of the largest each."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host_bits
from test_gpu_kv4 import Attn, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


def check_heaviest(c, scale):
    """Rows whose scores tell their largest one from all others have its V; how many do."""
    Hq, Hkv = c.q.shape[1], c.pages.shape[1]
    got, q = oracle.to_f64(host_bits(c.out)), oracle.to_f64(host_bits(c.q.contiguous()))
    seen, g = 0, Hq // Hkv
    for i in range(2):
        for r in range(c.cu[i], c.cu[i + 1]):
            n = int(c.kv_len[i]) + r - int(c.cu[i]) + 1
            for h in range(Hq):
                if np.abs(q[r, h]).max() > 65504:      # (infinite in f16: 2^14 times 4 and more)
                    assert not np.isfinite(got[r, h]).any()
                    continue
                K, V = (oracle.kv4_values(*oracle.kv4_load(c.pages, c.table, 16, i, n, h // g, w), f)
                        for w, f in ((0, 0.5), (1, 0.25)))
                s = K @ q[r, h]
                order = np.argsort(s)
                gap, unsure = s[order[-1]] - s[order[-2]], (np.abs(K) @ np.abs(q[r, h])).max() * 272 * 2.0 ** -24
                if gap > 2 * unsure and (gap - unsure) * scale > 90:
                    assert np.array_equal(got[r, h], V[order[-1]]), (r, h)
                    seen += 1
                assert np.isfinite(got[r, h]).all()
    return seen


@pytest.mark.parametrize("Hq,Hkv,rows", [(2, 2, 1), (12, 1, 1), (20, 1, 1), (4, 1, 5)])
@pytest.mark.parametrize("power", [12, 18, 21, 23, 25, 27, 30, 45, 90])
def test_scores_far_beyond_exps_range(api, Hq, Hkv, rows, power):
    """At scores of 2^power and more one token has all the weight of a row: its V comes back, bit for bit,
    as long as scores are finite in fp32.  Rows are left out where the two largest scores are closer than
    fp32 tells apart (136 roundings of 2^-24 of the sum of |q k|, twice), or where the second one's weight is
    not 0: pieces of a row are weighed in fp32, so that e^-40 still shows where the first one's V is 0, but
    2^-126 = e^-87.4 and less is flushed."""
    c = Attn(api, [700, 33], [rows, rows], Hq, Hkv, 128, 16, seed=power)
    scale = 2.0 ** power / 30
    c.run(scale=scale)
    seen = check_heaviest(c, scale)
    assert seen >= rows * Hq or power < 18


@pytest.mark.parametrize("Hq,Hkv,rows", [(2, 2, 1), (12, 1, 1), (20, 1, 1), (4, 1, 5)])
@pytest.mark.parametrize("power", [6, 10, 12, 14])
def test_far_scores_of_large_queries_and_keys(api, Hq, Hkv, rows, power):
    """The same with an ordinary scale: scores of up to 2^power 2^8 30 / 11.3."""
    c = Attn(api, [700, 33], [rows, rows], Hq, Hkv, 128, 16, seed=power)
    scales = c.pages[..., 8 * 128:9 * 128]
    scales[scales != 0xFF] += 64                                    # (0.01 .. 1.7 before: 2^8 times)
    assert int(scales[scales != 0xFF].max()) < 0x7F
    c.cache.pages.copy_(dev(c.pages))
    c.q *= 2.0 ** power
    c.run()
    assert check_heaviest(c, 1 / np.sqrt(128)) >= rows * Hq


@pytest.mark.parametrize("g", [1, 12, 20])                 # one, two and three columns of 8 rows
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("power", [-24.6, -25.1, -27.3])
def test_one_heavy_token_and_many_light_ones(api, g, D, power):
    """2^18 tokens whose weight is 2^power and whose V is 1, behind one of weight 1 and V 0: N 2^power /
    (1 + N 2^power).  Wanted within half a step of bf16 and 2^-10: the light tokens' roundings come to 2^18
    2^-32 = 2^-14, and fp32 sums of 2^18 equal terms to at most 2^18 2^-24 of the result, 2^-6 of less than
    2^-6.  So many sequences that a warp has most of one (all of the same two pages), so that one running
    maximum holds for it."""
    n, page, B, Hkv = 1 << 18, 4096, 700, 4
    pages = torch.zeros(2, Hkv, page // 16, 18 * D, dtype=torch.uint8, device="cuda")
    pages[..., 0:8 * D:D // 2] = 2                                  # K: E2M1 1 in element 0, its scales 0
    pages[..., 9 * D:17 * D] = 0x22                                 # V: 1
    pages[..., 17 * D:] = 0x38
    pages[1, :, 0, 8 * D] = 0x38                                    # the first token of page 1: K 1, V 0
    pages[1, :, 0, 9 * D:9 * D + D // 2] = 0
    cache = api.Kv4Cache(2, Hkv, D, page_size=page, pages=pages)
    table = torch.zeros(B, n // page, dtype=torch.int32, device="cuda")
    table[:, 0] = 1
    q = torch.zeros(B, Hkv * g, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    out = torch.zeros_like(q)
    cu, kv_len = dev(np.arange(B + 1, dtype=np.int32)), dev(np.full(B, n - 1, np.int32))
    scale = float(np.float32(-power * np.log(2.0)))
    a = api.kv4_attn_args(cache, table, cu, kv_len, q, out, max_q_rows=1, scale=scale)
    api.spec_kv4_attn(a, api.kv4_workspace(a))
    torch.cuda.synchronize()
    light = (n - 1) * np.exp(-scale)
    want = light / (1.0 + light)
    got = oracle.to_f64(host_bits(out))
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * want + 2.0 ** -10), (got.min(), got.max(), want)


@pytest.mark.parametrize("Hq,Hkv,rows", [(2, 2, 1), (12, 1, 1), (20, 1, 1), (4, 1, 5)])
@pytest.mark.parametrize("power", [-14, -20, -25, -30, -60, -126])
def test_queries_of_small_magnitude(api, Hq, Hkv, rows, power):
    """q times 2^power with a scale of 2^-power (in two factors where fp32 has no such one): the same
    exact scores, and the same tolerance, as of q itself."""
    c = Attn(api, [300, 33], [rows, rows], Hq, Hkv, 128, 16, seed=rows)
    small = dict(scale=2.0 ** min(-power, 100) / 12)
    c.q *= 2.0 ** power
    if power < -100:
        c.cache.k_scale = 0.5 * 2.0 ** (-power - 100)
    c.run(**small)
    close(c.out, c.q.contiguous(), c.pages, c.table, 16, c.cu, c.kv_len, small["scale"],
          (c.cache.k_scale, 0.25))
    assert int(c.status.item()) == 0


def test_rows_and_heads_of_different_magnitude(api):
    """Each row and head by itself: neighbours of other magnitudes, zeros among them, change no bit."""
    c = Attn(api, [300], [3], 8, 2, 128, 16)
    c.q *= 2.0 ** -30
    c.run(scale=2.0 ** 30 / 12)
    want = c.out.clone()
    c.check(scale=2.0 ** 30 / 12)
    keep = [(0, 1), (1, 4), (2, 7)]
    other = torch.ones(3, 8, dtype=torch.bool)
    for r, h in keep:
        other[r, h] = False
    c.q[other.cuda()] *= 2.0 ** 20
    c.q[1, 0], c.q[2, 5] = 0, float("inf")
    c.run(scale=2.0 ** 30 / 12)
    for r, h in keep:
        assert torch.equal(c.out[r, h], want[r, h])
    assert bool(c.out[1, 0].isfinite().all()) and not bool(c.out[2, 5].isfinite().any())


def test_elements_of_different_magnitude(api):
    """Elements of a row down to 2^-31 of its largest keep their bits: the largest meets zeros of K alone."""
    D, page, n = 64, 16, 48
    c = Attn(api, [n - 1], [1], 1, 1, D, page)
    for t in range(n):
        codes, scales = (x[-1].copy() for x in oracle.kv4_load(c.pages, c.table, page, 0, t + 1, 0, 0))
        codes[:8] = 0
        oracle.kv4_store(c.pages, c.table, page, 0, t, 0, 0, codes, scales)
    c.cache.pages.copy_(dev(c.pages))
    c.q *= 2.0 ** -16
    c.q[..., :8] = 1.49 * 2.0 ** 13
    c.run(scale=2.0 ** 13)
    c.check(scale=2.0 ** 13)
