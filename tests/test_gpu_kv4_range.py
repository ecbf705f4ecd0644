"""Attention over the paged 4-bit cache at the ends of its operands' ranges."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host_bits
from test_gpu_kv4 import Attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


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
    got, q = oracle.to_f64(host_bits(c.out)), oracle.to_f64(host_bits(c.q.contiguous()))
    seen, g = 0, Hq // Hkv
    for i in range(2):
        for r in range(c.cu[i], c.cu[i + 1]):
            n = int(c.kv_len[i]) + r - int(c.cu[i]) + 1
            for h in range(Hq):
                K, V = (oracle.kv4_values(*oracle.kv4_load(c.pages, c.table, 16, i, n, h // g, w), f)
                        for w, f in ((0, 0.5), (1, 0.25)))
                s = K @ q[r, h]
                order = np.argsort(s)
                gap, unsure = s[order[-1]] - s[order[-2]], (np.abs(K) @ np.abs(q[r, h])).max() * 272 * 2.0 ** -24
                if gap > 2 * unsure and (gap - unsure) * scale > 90:
                    assert np.array_equal(got[r, h], V[order[-1]]), (r, h)
                    seen += 1
                assert np.isfinite(got[r, h]).all()
    assert seen >= rows * Hq or power < 18
