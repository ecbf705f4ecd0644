"""The paged 4-bit cache in the order a serving loop uses it: prompts enter the
pages, then steps of append (norms and rotation on the way), attention, logits
adjustment and rejection sampling, the lengths advanced by what was accepted;
and a step captured into a graph.  Each operator is compared with the float64
oracle on the inputs it really had."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import compare_sampling, dev, host_bits
from test_gpu_kv4 import close
from test_gpu_norm_rope import NORM
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


class Loop:
    """Buffers of a serving loop: everything is allocated once, lengths and tables advance in place."""

    def __init__(self, api, B=3, K=3, Hq=4, Hkv=2, D=128, V=1000, page=16, steps=4, prompts=(20, 0, 47)):
        self.api, self.B, self.K, self.V, self.page, self.D = api, B, K, V, page, D
        self.rng = np.random.default_rng(11)
        self.R = B * (K + 1)
        self.cu = np.arange(B + 1, dtype=np.int32) * (K + 1)
        most = [n + steps * (K + 1) + 1 for n in prompts]
        need = [-(-n // page) for n in most]
        ids = self.rng.permutation(sum(need) + 2)
        self.table = np.full((B, max(need)), -1, np.int32)
        for i, n in enumerate(need):
            self.table[i, :n], ids = ids[:n], ids[n:]
        self.cache = api.Kv4Cache(sum(need) + 2, Hkv, D, page_size=page, k_scale=0.5, v_scale=0.25)
        self.cache.pages.fill_(0xFF)                       # NaN wherever nothing was stored
        self.kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.turns, self.m = api.rope_turns(D, scaling="yarn", factor=4.0, trained_len=64)
        self.w = [dev((1 + 0.2 * self.rng.standard_normal(D)).astype(np.float32)) for _ in range(2)]
        self.how = dict(turns=self.turns, mscale=self.m, q_weight=self.w[0], k_weight=self.w[1],
                        dev_status=self.status)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.qkv = torch.zeros(self.R, Hq + 2 * Hkv, D, **bf)
        self.q, self.out = torch.zeros(self.R, Hq, D, **bf), torch.zeros(self.R, Hq, D, **bf)
        self.tgt, self.drf = torch.zeros(self.R, V, **bf), torch.zeros(B * K, V, **bf)
        self.drafts = torch.zeros(B * K, dtype=torch.int32, device="cuda")
        self.accepted = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.tokens = torch.zeros(self.R, dtype=torch.int32, device="cuda")
        self.dcu, self.dtable = dev(self.cu), dev(self.table)
        k, v = self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:]
        self.append = api.kv4_append_args(self.cache, self.dtable, self.dcu, self.kv_len, k, v,
                                          max_q_rows=K + 1, q=self.qkv[:, :Hq], q_out=self.q, **self.how)
        self.attn = api.kv4_attn_args(self.cache, self.dtable, self.dcu, self.kv_len, self.q, self.out,
                                      max_q_rows=K + 1, dev_status=self.status)
        self.attn_ws = api.kv4_workspace(self.attn)
        self.adjust = api.adjust_args(self.tgt, self.tgt, self.dcu, max_q_rows=K + 1, presence=0.0,
                                      repetition=1.0, dev_status=self.status)
        self.sample = api.sample_args(self.tgt, self.drf, self.drafts, self.dcu, self.kv_len, self.accepted,
                                      self.tokens, max_q_rows=K + 1, temperature=0.9, top_p=1.0, seed=5,
                                      dev_status=self.status)
        self.sample_ws = api.Workspace(api.workspace_bytes(sample=self.sample))
        # prompts of different lengths, one of none; their q is not needed
        cu = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
        x = dev(self.draw((int(cu[-1]), 2 * Hkv, D)))
        api.spec_kv4_append(api.kv4_append_args(
            self.cache, self.dtable, dev(cu), self.kv_len, x[:, :Hkv], x[:, Hkv:],
            max_q_rows=max(prompts), **self.how))
        self.kv_len += dev(np.array(prompts, np.int32))

    def draw(self, shape, std=1.0):
        return f32_to_bf16_bits((self.rng.standard_normal(shape) * std).astype(np.float32))

    def new_inputs(self):
        self.qkv.copy_(dev(self.draw(tuple(self.qkv.shape))))
        t = (self.rng.standard_normal((self.R, self.V)) * 2).astype(np.float32)
        self.tgt.copy_(dev(f32_to_bf16_bits(t)))
        rows = [r for r in range(self.R) if (r + 1) % (self.K + 1)]
        self.drf.copy_(dev(f32_to_bf16_bits(t[rows] + self.rng.standard_normal((len(rows), self.V)).astype(np.float32) / 2)))
        self.drafts.copy_(self.drf.float().argmax(1))

    def step(self):
        self.api.spec_kv4_append(self.append)
        self.api.spec_kv4_attn(self.attn, self.attn_ws)
        self.api.spec_adjust_logits(self.adjust)
        self.api.spec_reject_sample(self.sample, self.sample_ws)
        self.kv_len.add_(self.accepted).add_(1)

    def check(self, before):
        """Of the step that began at lengths `before`."""
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        freqs, m = oracle.rope_frequencies(self.D, kind="yarn", factor=4.0, trained=64)
        x = oracle.to_f64(host_bits(self.qkv.contiguous()))
        Hq = self.q.shape[1]
        y = oracle.head_norm(x[:, :Hq], self.w[0].cpu().numpy(), 1e-6)
        want = oracle.rope_rows(y, oracle.row_positions(self.cu, before), freqs, "half", m)
        got = oracle.to_f64(host_bits(self.q))
        both = np.abs(y) + np.abs(np.roll(y, self.D // 2, axis=-1))
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 1.01 * (1e-6 + NORM) * m * both)
        close(self.out, self.q, self.cache.pages.cpu().numpy(), self.table, self.page, self.cu, before)
        drafts = self.drafts.cpu().numpy()
        ref = oracle.reject_sample(host_bits(self.tgt), host_bits(self.drf), drafts, self.cu, before,
                                   0.9, 1.0, 5)
        acc = self.accepted.cpu().numpy()
        compare_sampling(ref, acc, self.tokens.cpu().numpy(), self.cu, drafts, self.V)
        assert np.array_equal(self.kv_len.cpu().numpy(), before + acc + 1)


def test_serving_loop(api):
    s = Loop(api)
    for _ in range(4):
        s.new_inputs()
        before = s.kv_len.cpu().numpy()
        s.step()
        s.check(before)


def test_serving_loop_as_a_graph(api):
    """Captured once, replayed over the same buffers as lengths grow."""
    s = Loop(api, steps=6)
    s.new_inputs()
    before = s.kv_len.cpu().numpy()
    s.step()                                              # (loads everything)
    s.check(before)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step()
    for _ in range(5):
        s.new_inputs()
        before = s.kv_len.cpu().numpy()
        g.replay()
        s.check(before)


def test_prefix_handed_to_the_unpaged_pool(api):
    """Rows read back in bf16 hold the cache's values exactly, so the unpaged attention over them
    gives the same outputs within both kernels' rounding (2e-2, as that kernel's own tests have it)."""
    s = Loop(api, prompts=(60, 33, 5))
    s.new_inputs()
    before = s.kv_len.cpu().numpy()
    api.spec_kv4_append(s.append)
    api.spec_kv4_attn(s.attn, s.attn_ws)
    Hkv, D, n = s.cache.num_kv_heads, s.D, before + s.K + 1
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    pool = [torch.zeros(int(cu[-1]), Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    api.spec_kv4_read(api.kv4_read_args(s.cache, s.dtable, dev(cu), torch.zeros_like(s.kv_len), *pool,
                                        max_q_rows=int(n.max())))
    block = torch.cat([torch.arange(int(cu[i]) + int(before[i]), int(cu[i + 1])) for i in range(s.B)]).cuda()
    out = torch.zeros_like(s.out)
    a = api.attn_args(s.q, pool[0][block], pool[1][block], *pool, s.dcu, dev(cu[:-1].astype(np.int64)),
                      s.kv_len, out, max_q_rows=s.K + 1, kv_rows_bound=int(before.max()) * s.B)
    api.spec_verify_attn(a, api.Workspace(api.workspace_bytes(a)))
    torch.cuda.synchronize()
    assert float((out.float() - s.out.float()).abs().max()) < 2e-2
