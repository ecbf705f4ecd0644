"""GPU parity of spec_count_tokens with the oracle (whole numbers: equal)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


class Table:
    def __init__(self, api, slots, vocab, rng=None):
        self.api = api
        self.t = api.TokenCounts(slots, vocab)
        self.ref = np.zeros((slots, vocab), dtype=np.int32)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        if rng is not None:             # something in it already
            fill = rng.random((slots, vocab)) < 0.2
            self.ref[fill] = rng.integers(1, 50, fill.sum())
            self.ref[rng.random((slots, vocab)) < 0.1] |= np.int32(-2 ** 31)
            self.t.counts.copy_(dev(self.ref))
            self.t.seen.copy_(dev(oracle.seen_bits(self.ref)))

    def add(self, tokens, start, status=0, **kw):
        tokens, start = np.asarray(tokens, np.int32), np.asarray(start, np.int32)
        arrays = {k: (dev(np.asarray(v, np.int32)) if k in ("slots", "num_accepted") and
                      v is not None else v) for k, v in kw.items()}
        self.api.spec_count_tokens(self.api.count_args(
            self.t.counts, self.t.seen, dev(tokens), dev(start), dev_status=self.status, **arrays))
        torch.cuda.synchronize()
        self.ref, seen, st = oracle.count_tokens(self.ref, tokens, start, **kw)
        assert np.array_equal(self.t.counts.cpu().numpy(), self.ref)
        assert np.array_equal(self.t.seen.cpu().numpy(), seen)
        assert st == status and int(self.status.item()) == status
        self.status.zero_()


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 100, 1000, 4099])
@pytest.mark.parametrize("B", [1, 3, 40])
def test_prompts_then_steps(api, V, B):
    rng = np.random.default_rng(V * 100 + B)
    t = Table(api, B + 2, V, rng)
    slots = rng.permutation(B + 2)[:B]
    lens = rng.integers(0, 60, B)
    start = np.concatenate([[0], np.cumsum(lens)])
    t.add(rng.integers(0, V, start[-1]), start, slots=slots, prompt=True, reset=True)
    for _ in range(3):
        R = rng.integers(1, 10, B)
        cu = np.concatenate([[0], np.cumsum(R)])
        n = rng.integers(-1, R)
        out = rng.integers(0, V, cu[-1])
        for i in range(B):                      # as a step leaves them: -1 after the last token
            out[cu[i] + n[i] + 1:cu[i + 1]] = -1
        t.add(out, cu, slots=slots, num_accepted=n)
    t.add(rng.integers(0, V, start[-1]), start, slots=slots)
    t.add([], [0] * (B + 1), slots=slots, reset=True)


def test_one_token_many_times(api):
    """Hot tokens: every thread on one or two words."""
    t = Table(api, 2, 300)
    n = 70_000
    tok = np.full(n, 7)
    tok[::3] = 8
    t.add(tok, [0, n // 2, n], slots=[1, 1])
    t.add(tok, [0, n // 2, n], slots=[1, 0], prompt=True)
    assert t.ref[1, 7] == np.int32(-2 ** 31 + (tok == 7).sum())


@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("V", [8191, 8193, 32769, 70000])
def test_reset_over_slices(api, V, prompt):
    """Vocabularies of several slices, prompts longer than a CTA takes at once,
    and three sequences on one slot."""
    rng = np.random.default_rng(V)
    t = Table(api, 4, V, rng)
    lens = [9000, 0, 31, 17000, 1]
    start = np.concatenate([[0], np.cumsum(lens)])
    tok = (rng.random(start[-1]) ** 3 * V).astype(np.int64)
    t.add(tok, start, slots=[1, 3, 1, 0, 1], prompt=prompt, reset=True)
    n = np.array([2 ** 31 - 1, -1, 3, -2 ** 31, 0])
    t.add(tok, start, slots=[0, 2, 1, 3, 1], prompt=prompt, reset=True, num_accepted=n)


def test_shared_and_absent_slots(api):
    t = Table(api, 3, 50, np.random.default_rng(3))
    t.add([1, 2, 3, 4, 5, 6], [0, 2, 4, 6], slots=[2, -1, 2], reset=True)
    assert t.ref[2].sum() == 4
    t.add([1, 2, 3], [0, 1, 2, 3])              # no slots: sequence i has row i


def test_many_sequences(api):
    """More sequences than start values are kept in shared memory for."""
    B = 5000
    rng = np.random.default_rng(9)
    t = Table(api, B, 40, rng)
    start = np.concatenate([[0], np.cumsum(rng.integers(0, 4, B))])
    tok = rng.integers(0, 40, start[-1])
    t.add(tok, start, slots=rng.integers(-1, B, B))
    t.add(tok, start, slots=rng.permutation(B), reset=True, prompt=True)
    t.add(tok, start, slots=rng.integers(0, 7, B), reset=True)


def test_bad_tokens_and_slots(api):
    t = Table(api, 3, 50, np.random.default_rng(4))
    t.add([1, 50, -1, 4, 2 ** 31 - 1, 6], [0, 2, 4, 6], slots=[0, 1, 2],
          status=oracle.sampling.DEV_BAD_TOKEN)
    t.add([1, 2, 3, 4, 5, 6], [0, 2, 4, 6], slots=[0, 3, -2], status=oracle.DEV_BAD_PARAM)
    t.add([1, 2, 3, 4, 5, 6], [0, 2, 4, 6], slots=[0, 2 ** 31 - 1, 1], reset=True,
          status=oracle.DEV_BAD_PARAM)


@pytest.mark.parametrize("start", [[0, 4, 2, 6], [-1, 2, 4, 6], [0, 2, 4, 7], [6, 4, 2, 0],
                                   [0, 2 ** 31 - 1, 5, 6]])
def test_bad_start_values_write_nothing_wrong(api, start):
    """The bit is set, and nothing outside the named slots or the vocabulary changes."""
    t = Table(api, 4, 50)
    tok = np.array([1, 2, 3, 4, 5, 6], np.int32)
    t.api.spec_count_tokens(api.count_args(t.t.counts, t.t.seen, dev(tok),
                                           dev(np.array(start, np.int32)), dev_status=t.status))
    torch.cuda.synchronize()
    c = t.t.counts.cpu().numpy()
    assert int(t.status.item()) == oracle.DEV_BAD_LENGTH
    assert c.min() >= 0 and c.sum() <= 6 and not c[3].any() and not c[:, 7:].any()
    assert np.array_equal(t.t.seen.cpu().numpy(), oracle.seen_bits(c))


def test_tokens_behind_the_last_sequence_do_not_count(api):
    t = Table(api, 2, 50)
    t.add([1, 2, 3, 9, 9, 9], [0, 1, 3])
    assert t.ref[:, 9].sum() == 0


def test_offsets_past_32_bits(api):
    V, S = 128256, 17000                        # 2.2 G words
    t = api.TokenCounts(S, V)
    tok = dev(np.array([V - 1, V - 1, 0], np.int32))
    a = api.count_args(t.counts, t.seen, tok, dev(np.array([0, 3], np.int32)),
                       slots=dev(np.array([S - 1], np.int32)))
    api.spec_count_tokens(a)
    torch.cuda.synchronize()
    row = t.counts[-1].cpu().numpy()
    assert row[V - 1] == 2 and row[0] == 1 and np.count_nonzero(row) == 2
    assert int(t.counts.count_nonzero()) == 2 and int(t.seen.count_nonzero()) == 2
    api.spec_count_tokens(api.count_args(t.counts, t.seen, tok, dev(np.array([0, 0], np.int32)),
                                         slots=dev(np.array([S - 1], np.int32)), reset=True))
    torch.cuda.synchronize()
    assert int(t.counts.count_nonzero()) == 0 and int(t.seen.count_nonzero()) == 0


def test_captured_and_replayed(api):
    t = Table(api, 2, 100)
    tok, start = dev(np.array([1, 2, 2, 99], np.int32)), dev(np.array([0, 3, 4], np.int32))
    acc = dev(np.array([1, 0], np.int32))
    a = api.count_args(t.t.counts, t.t.seen, tok, start, num_accepted=acc)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.spec_count_tokens(a)
    graph.replay()
    tok.copy_(dev(np.array([5, 2, 2, 98], np.int32)))
    acc.copy_(dev(np.array([2, -1], np.int32)))
    graph.replay()
    torch.cuda.synchronize()
    c = t.t.counts.cpu().numpy()
    assert c[0, [1, 2, 5]].tolist() == [1, 3, 1] and c[1, 99] == 1 and c.sum() == 6


def test_torch_call_refusals(api):
    t = api.TokenCounts(2, 100)
    tok, start = dev(np.array([1, 2], np.int32)), dev(np.array([0, 2], np.int32))
    bad = [
        lambda: api.count_args(t.counts.long(), t.seen, tok, start),
        lambda: api.count_args(t.counts, t.seen[:, :3], tok, start),
        lambda: api.count_args(t.counts, t.seen, tok.long(), start),
        lambda: api.count_args(t.counts, t.seen, tok, start.long()),
        lambda: api.count_args(t.counts, t.seen, tok, start, slots=start),
        lambda: api.count_args(t.counts, t.seen, tok, start, num_accepted=start),
        lambda: api.count_args(t.counts.t(), t.seen, tok, start),
        lambda: api.count_args(t.counts, t.seen, tok.cpu(), start),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
