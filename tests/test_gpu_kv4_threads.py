"""Two host threads, each with a stream, buffers and a workspace of its own, whose calls
of one kernel need different amounts of shared memory: every call is taken, and
the outputs are those of calls one after the other, bit for bit."""
import threading

import numpy as np
import pytest
import torch

from test_gpu_kv4 import Attn
from test_gpu_norm_rope import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


def side_by_side(calls, times):
    """Makes each of the calls (a function of a stream) many times in a thread of its own."""
    problems, ready = [], threading.Barrier(len(calls))

    def loop(call):
        stream = torch.cuda.Stream()
        try:
            ready.wait()
            for _ in range(times):
                call(stream)
        except Exception as e:          # noqa: BLE001 (shown by the assertion below)
            problems.append(e)
        stream.synchronize()

    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not problems, problems[:2]


@pytest.mark.parametrize("Hq", [1, 12, 20])
def test_attention_of_one_and_of_many_sequences(api, Hq):
    rng = np.random.default_rng(1)
    cases = [Attn(api, [40], [1], Hq, 1, 128, 16, garbage=None),
             Attn(api, rng.integers(0, 30, 768), [1] * 768, Hq, 1, 128, 16, garbage=None)]
    args = [c.args() for c in cases]
    ws = [api.kv4_workspace(a) for a in args]
    for a, w in zip(args, ws):
        api.spec_kv4_attn(a, w)
    torch.cuda.synchronize()
    want = [c.out.clone() for c in cases]
    for c in cases:
        c.check()
        c.out.fill_(123.0)
    torch.cuda.synchronize()
    side_by_side([lambda s, a=a, w=w: api.spec_kv4_attn(a, w, stream=s) for a, w in zip(args, ws)], 3000)
    torch.cuda.synchronize()
    for c, x in zip(cases, want):
        assert torch.equal(c.out, x)


@pytest.mark.parametrize("rot", [1.0, 0.1])
def test_norms_of_small_and_of_large_heads(api, rot):
    cases = [Case(api, [3], 2, 1, 64, 2 * int(32 * rot), "f32"), Case(api, [2600], 2, 1, 256, 2 * int(128 * rot), "f32")]
    args = [c.args() for c in cases]
    for a in args:
        api.spec_norm_rope_rows(a)
    for c in cases:
        c.check()
        for o in c.out.values():
            o.fill_(123.0)
    torch.cuda.synchronize()
    side_by_side([lambda s, a=a: api.spec_norm_rope_rows(a, stream=s) for a in args], 3000)
    for c in cases:
        c.check()
