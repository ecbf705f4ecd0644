"""spec_norm_rope_rows without norms against spec_rope_rows: the same angles and the same products.

What is copied (v, elements that do not turn) is equal.  Turned elements are a cos - b sin (b cos + a
sin) in fp32, products and sum perhaps fused in one and not in the other: three roundings of 2^-24 of |a| + |b|
(times mscale) at most apart, in each; then each is rounded to bf16, by half a step."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host_bits
from test_gpu_norm_rope import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout,D,rot", [("half", 128, 128), ("interleaved", 128, 64), ("half", 64, 20),
                                          ("half", 96, 48), ("interleaved", 72, 70), ("half", 256, 16)])
def test_without_norms_as_the_rotary_operator(api, layout, D, rot, dtype):
    c = Case(api, [3, 90, 1], 4, 2, D, rot, dtype, layout, norms="", mscale=1.25)
    api.spec_norm_rope_rows(c.args())
    torch.cuda.synchronize()
    got = {p: oracle.to_f64(host_bits(o)) for p, o in c.out.items()}
    api.spec_rope_rows(api.rope_args(
        *(c.dx[:, c.heads[p]] for p in "qkv"), *(c.out[p] for p in "qkv"), c.turns, cu_q=dev(c.cu),
        kv_len=dev(c.kv_len), max_q_rows=c.max_rows, layout=layout, mscale=1.25))
    torch.cuda.synchronize()
    half = rot // 2
    pairs = [(i, i + half) if layout == "half" else (2 * i, 2 * i + 1) for i in range(half)]
    one, two = (np.array(x) for x in zip(*pairs))
    step = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]
    for p in "qkv":
        want, x = oracle.to_f64(host_bits(c.out[p])), oracle.to_f64(c.x[:, c.heads[p]])
        if p == "v":
            assert np.array_equal(got[p], want)
            continue
        assert np.array_equal(got[p][..., rot:], want[..., rot:])
        size = 1.25 * (np.abs(x[..., one]) + np.abs(x[..., two]))
        for e in (one, two):
            near = 2 * 3 * 2.0 ** -24 * size + step * (np.abs(got[p][..., e]) + np.abs(want[..., e]))
            assert np.all(np.abs(got[p][..., e] - want[..., e]) <= near), (p, layout)
