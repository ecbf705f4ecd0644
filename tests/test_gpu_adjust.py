"""GPU parity of spec_adjust_logits with the float64 oracle.

Tolerance per value: the repetition penalty's reciprocal and the product with
it, the fused frequency * times + presence, the subtraction and the bias sum
round at 2^-24 of their results each, all bounded by
S = |x| max(r, 1 / r) + |f| times + |p| + |bias|: at most 5 * 2^-24 S; the store
rounds by half a step, 2^-8 of the value for bf16.  Values that nothing touches
keep their bits."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host_bits
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu

BAD_TOKEN = oracle.sampling.DEV_BAD_TOKEN


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


def _logits(rng, shape, dtype):
    x = rng.standard_normal(shape, dtype=np.float32) * np.float32(3)
    return f32_to_bf16_bits(x) if dtype == "bf16" else x


def _bits(allowed, width=None):
    """Truth [M, V] as [M, W] int32 words."""
    M, V = allowed.shape
    W = width or (V + 31) // 32
    pad = np.zeros((M, W * 32), dtype=bool)
    pad[:, :V] = allowed
    pad[:, V:] = np.arange(W * 32 - V) % 2 == 0       # bits past V say nothing
    return np.packbits(pad, axis=1, bitorder="little").view("<u4").astype(np.uint32).view(np.int32)


class Case:
    """Random inputs of one call; `ref` holds the oracle's keyword arguments."""

    def __init__(self, api, rows, V, dtype="bf16", seed=0, draft=True, table=True, hist=40, ctx=0,
                 bias=0, masked=0.0, penal=True, allow=0.5, mask_width=None):
        rng = self.rng = np.random.default_rng(seed)
        self.api, self.V, self.dtype = api, V, dtype
        B = self.B = len(rows)
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        R = self.R = int(self.cu[-1])
        self.max_rows = max(rows)
        self.target = _logits(rng, (R, V), dtype)
        self.draft = _logits(rng, (R - B, V), dtype) if draft and R > B else None
        self.tokens = rng.integers(0, V, R - B).astype(np.int32) if R > B else None
        if self.tokens is not None and len(self.tokens) > 2:
            self.tokens[1] = self.tokens[0]           # the same token twice in a block
        self.kw, self.ref = {}, {}
        if table:
            counts = np.zeros((B + 2, V), dtype=np.int32)
            for s in range(B + 2):
                np.add.at(counts[s], rng.integers(0, V, hist), 1)
                counts[s, rng.integers(0, V, hist)] |= np.int32(-2 ** 31)
            slots = rng.permutation(B + 2)[:B].astype(np.int32)
            self.kw.update(counts=counts, seen=oracle.seen_bits(counts), slots=slots)
            self.ref.update(counts=counts, slots=slots)
        if penal:
            for k in ("repetition", "presence", "frequency"):
                v = (rng.random(B) + (0.6 if k == "repetition" else -0.3)).astype(np.float32)
                self.kw[k + "s" if k != "frequency" else "frequencies"] = v
                self.ref[k] = v
        if ctx:
            c = rng.integers(-1, V, (ctx, B)).astype(np.int32)
            self.kw["ctx_tokens"] = self.ref["ctx"] = c
        if bias:
            per = [[(int(t), float(np.float32(v))) for t, v in
                    zip(rng.integers(0, V, n), rng.standard_normal(n))]
                   for n in rng.integers(0, bias + 1, B)]
            self.set_bias(per)
        if masked:
            M = max(1, int(masked * R))
            self.allowed = rng.random((M, V)) < allow
            at = np.full(R, -1, dtype=np.int32)
            at[rng.permutation(R)[:M]] = rng.permutation(M)
            self.kw.update(mask=_bits(self.allowed, mask_width), mask_rows=at)
            self.ref.update(mask=self.kw["mask"], mask_rows=at)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def set_bias(self, per):
        self.ref["bias"] = per
        flat = [e for seq in per for e in seq]
        self.kw.update(bias_start=np.concatenate([[0], np.cumsum([len(s) for s in per])]).astype(np.int32),
                       bias_tokens=np.array([t for t, _ in flat], np.int32),
                       bias_values=np.array([v for _, v in flat], np.float32))

    def args(self, in_place=False, **more):
        kw = {k: dev(v) if isinstance(v, np.ndarray) else v for k, v in (self.kw | more).items()}
        cu = kw.pop("cu", None)
        self.dt, self.dd = dev(self.target), None if self.draft is None else dev(self.draft)
        self.ot = self.dt if in_place else torch.full_like(self.dt, 77.0)
        self.od = None if self.draft is None else self.dd if in_place else \
            torch.full_like(self.dd, 77.0)
        return self.api.adjust_args(
            self.dt, self.ot, dev(self.cu) if cu is None else cu, max_q_rows=self.max_rows,
            draft=self.dd, draft_out=self.od, dev_status=self.status,
            draft_tokens=None if self.tokens is None else dev(self.tokens), **kw)

    def run(self, in_place=False, status=0, **more):
        self.api.spec_adjust_logits(self.args(in_place, **more))
        torch.cuda.synchronize()
        self.check(status)

    def check(self, status=0):
        want_t, want_d, st = oracle.adjust_logits(self.target, self.cu, self.draft, self.tokens,
                                                  **self.ref)
        assert int(self.status.item()) == st == status
        seq = np.repeat(np.arange(self.B), np.diff(self.cu))
        last = self.cu[1:] - 1
        for got_t, x, want, rows in ((self.ot, self.target, want_t, seq),
                                     (self.od, self.draft, want_d,
                                      np.delete(seq, last))):
            if x is None:
                continue
            got, x64 = oracle.to_f64(host_bits(got_t)), oracle.to_f64(x)
            assert np.array_equal(np.isnan(got), np.isnan(want))
            fin = np.isfinite(want)
            assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])

            def of(k):
                v = np.asarray(self.ref.get(k, 1.0 if k == "repetition" else 0.0), np.float64)
                v = np.where(np.isfinite(v), v, 0.0)
                return (v[rows] if v.ndim else np.full(len(rows), v))[:, None]

            r = np.abs(of("repetition")) + 1e-30
            times = 40 + self.ref.get("counts", np.zeros(1, np.int32)).view(np.uint32) \
                .astype(np.int64).__and__(0x7FFFFFFF).max()
            top = 0.0 if "bias" not in self.ref else \
                max([abs(v) for s in self.ref["bias"] for _, v in s if np.isfinite(v)] + [0.0])
            S = np.where(np.isfinite(x64), np.abs(x64), 0.0) * np.maximum(r, 1 / r) + \
                np.abs(of("frequency")) * times + np.abs(of("presence")) + top
            want, got = np.where(fin, want, 0.0), np.where(fin, got, 0.0)
            tol = 5 * 2.0 ** -24 * S + (2.0 ** -8 if self.dtype == "bf16" else 0.0) * np.abs(want)
            err = np.abs(got - want)
            assert np.all(err <= tol), float((err - tol).max())
            same = fin & (want == x64) & (x64 != 0)     # untouched: to the bit
            assert np.array_equal(host_bits(got_t)[same], x[same])


VOCABS = [1, 7, 8, 31, 33, 100, 255, 2047, 2048, 2049, 2056, 4100, 6151]


@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("in_place", [False, True])
def test_everything_at_once(api, V, dtype, in_place):
    c = Case(api, [1, 4, 2, 9, 1], V, dtype, seed=V, ctx=3, bias=20, masked=0.5,
             hist=min(3 * V, 60))
    c.run(in_place)


@pytest.mark.parametrize("kw", [
    dict(table=False, penal=False), dict(penal=False), dict(table=False), dict(table=False, ctx=5),
    dict(bias=1, penal=False), dict(bias=900, penal=False), dict(masked=1.0, penal=False),
    dict(masked=1.0, allow=0.01, mask_width=200), dict(masked=0.3, allow=0.99),
    dict(hist=20000), dict(draft=False), dict(draft=False, ctx=40, bias=3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_parts_alone(api, kw, in_place):
    for dtype in ("bf16", "f32"):
        Case(api, [3, 1, 16, 2], 5003, dtype, seed=9, **kw).run(in_place)


@pytest.mark.parametrize("B", [1, 2, 70])
@pytest.mark.parametrize("in_place", [False, True])
def test_single_rows(api, B, in_place):
    """A draft position: one row per sequence, the drafts so far as ctx."""
    c = Case(api, [1] * B, 32000, seed=B, ctx=4, bias=5, masked=0.5, hist=500)
    c.run(in_place)


def test_large_vocabulary(api):
    c = Case(api, [9, 3], 128256, seed=1, bias=300, masked=0.4, hist=4000)
    c.run()
    c.run(in_place=True)


@pytest.mark.parametrize("V,dtype", [(65536, "bf16"), (65541, "bf16"), (70003, "f32")])
@pytest.mark.parametrize("kw", [dict(ctx=2, bias=40, masked=0.4, hist=3000), dict(masked=1.0, allow=0.02),
                                dict(penal=False, bias=3), dict(hist=60000, draft=False)])
def test_in_place_of_many_long_rows(api, V, dtype, kw):
    """Sequences and vocabulary enough that single tokens are changed in memory:
    thin and dense lists, single rows and whole blocks, parts of a block's rows."""
    c = Case(api, [1, 3, 2] * 10, V, dtype, seed=V, **kw)
    c.run(in_place=True)


@pytest.mark.parametrize("rows", [[16, 2], [9] * 13])
@pytest.mark.parametrize("V", [4097, 33001])
def test_rows_split_over_ctas(api, rows, V):
    """Few sequences with many rows: the rows of a block are worked on in parts."""
    for in_place in (False, True):
        Case(api, rows, V, seed=3, ctx=1, bias=9, masked=0.3, hist=300).run(in_place)


def test_scalar_penalties(api):
    c = Case(api, [2, 3], 3001, "f32", seed=4, penal=False)
    c.ref.update(repetition=1.25, presence=0.5, frequency=-0.125)
    c.run(repetition=1.25, presence=0.5, frequency=-0.125)
    # one penalty alone
    for k, v in (("repetition", 0.5), ("presence", 2.0), ("frequency", 0.25)):
        c.ref.update(repetition=1.0, presence=0.0, frequency=0.0)
        c.ref[k] = v
        c.run(in_place=True, **{k: v})


def test_mask_rows_by_default_and_shared(api):
    c = Case(api, [2, 3], 777, seed=5, masked=1.0)
    c.kw.pop("mask_rows")
    c.ref["mask_rows"] = None
    c.run()
    c.kw["mask_rows"] = c.ref["mask_rows"] = np.array([0, 0, -1, 4, 0], np.int32)
    c.run(in_place=True)


def test_shared_and_absent_slots(api):
    c = Case(api, [2, 3, 1], 777, seed=6)
    c.kw["slots"] = c.ref["slots"] = np.array([1, -1, 1], np.int32)
    c.run()
    c.kw.pop("slots")
    c.ref["slots"] = None
    c.run()


def test_rows_that_keep_nothing(api):
    """A mask that bars every token: the row is all -inf, whatever stood there,
    and the sampler fails the sequence."""
    c = Case(api, [2, 2], 500, seed=7, masked=1.0)
    x = c.target.copy()
    x[0, :3] = f32_to_bf16_bits(np.array([np.nan, np.inf, -np.inf], np.float32))
    c.target = x
    c.kw["mask"][:] = 0
    for in_place in (False, True):
        c.run(in_place)
        assert bool((c.ot == -float("inf")).all())
    out = torch.zeros(4, dtype=torch.int32, device="cuda")
    acc = torch.zeros(2, dtype=torch.int32, device="cuda")
    kv = torch.zeros(2, dtype=torch.int32, device="cuda")
    s = api.sample_args(c.ot, c.od, dev(c.tokens), dev(c.cu), kv, acc, out, max_q_rows=2,
                        temperature=1.0, top_p=1.0, seed=0, dev_status=c.status)
    api.spec_reject_sample(s, api.Workspace.for_args(None, s))
    torch.cuda.synchronize()
    assert acc.tolist() == [-1, -1] and int(c.status.item()) == oracle.DEV_NONFINITE


def test_special_values(api):
    """NaN and infinities stay where nothing bars them; signed zeros and NaN
    payloads of untouched tokens keep their bits."""
    V = 2500
    for dtype in ("bf16", "f32"):
        c = Case(api, [2, 1], V, dtype, seed=8, masked=0.7, allow=0.6, bias=4)
        put = np.array([np.nan, np.inf, -np.inf, -0.0, 1e-40, 1e37], np.float32)
        at = c.rng.integers(0, V, (3, 60))
        x = c.target.copy()
        for r in range(3):
            x[r, at[r]] = np.resize(f32_to_bf16_bits(put) if dtype == "bf16" else put, 60)
        c.target = x
        for in_place in (False, True):
            c.run(in_place)
        plain = Case(api, [1, 2], V, dtype, seed=8, table=False, penal=False)
        plain.target = x
        plain.run()
        assert np.array_equal(host_bits(plain.ot).view(np.uint8), x.view(np.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_the_lowest_value(api, dtype):
    """Masks by the type's lowest finite value: a known token's product beyond the type is -inf
    (which the sampler reads as masked), everything else keeps the value."""
    V = 1500
    c = Case(api, [2, 2], V, dtype, seed=18, draft=False, hist=300)
    low = f32_to_bf16_bits(np.float32([-3.3895314e38]))[0] if dtype == "bf16" else \
        np.finfo(np.float32).min
    c.target = np.full_like(c.target, low)
    c.kw["repetitions"] = c.ref["repetition"] = np.array([1.5, 0.5], np.float32)
    for in_place in (False, True):
        api.spec_adjust_logits(c.args(in_place))
        torch.cuda.synchronize()
        want, _, st = oracle.adjust_logits(c.target, c.cu, None, c.tokens, **c.ref)
        got = oracle.to_f64(host_bits(c.ot))
        most = 3.39e38 if dtype == "bf16" else float(np.finfo(np.float32).max)
        over = want < -most * 1.01
        assert over.any() and np.all(got[over] == -np.inf)
        assert np.all(np.abs(got[~over] - want[~over]) <= 2.0 ** -8 * np.abs(want[~over]))
        assert int(c.status.item()) == st == 0


def test_many_sequences(api):
    Case(api, [1] * 3000 + [2] * 2100, 130, seed=20, hist=20, ctx=1, bias=3, masked=0.2).run()


def test_biases_twice_out_of_range_and_infinite(api):
    c = Case(api, [2, 1, 1, 1], 2100, "f32", seed=10, draft=False)
    c.set_bias([[(5, 1.0), (5, -2.0), (2099, 3.0)], [(2100, 1.0), (-1, 1.0), (7, 0.0), (8, 4.0)],
                [], [(0, -np.inf), (1, np.inf), (2049, -100.0)]])
    for in_place in (False, True):
        c.status.zero_()
        c.run(in_place, status=BAD_TOKEN)


@pytest.mark.parametrize("what,value", [
    ("repetitions", 0.0), ("repetitions", -1.0), ("repetitions", 1e-20), ("repetitions", 1e20), ("repetitions", np.nan), ("repetitions", np.inf),
    ("presences", np.nan), ("frequencies", -np.inf), ("slots", 9), ("slots", -2),
    ("mask_rows", 99), ("mask_rows", -2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_failing_sequences_are_nan(api, what, value, in_place):
    c = Case(api, [2, 3, 1], 2345, seed=11, masked=0.5, bias=3)
    at = 2 if what == "mask_rows" else 1        # row 2 is sequence 1's first
    key = {"repetitions": "repetition", "presences": "presence",
           "frequencies": "frequency"}.get(what, what)
    v = c.kw[what].copy()
    v[at] = value
    c.kw[what] = c.ref[key] = v
    c.run(in_place, status=oracle.DEV_BAD_PARAM)
    assert bool(torch.isnan(c.ot[2:5].float()).all()) and not bool(torch.isnan(c.ot[:2].float()).any())


@pytest.mark.parametrize("start", [[0, 9, 9, 9], [-1, 0, 2, 3], [0, 3, 2, 3]])
def test_bad_bias_ranges_are_nan(api, start):
    c = Case(api, [1, 1, 1], 300, seed=12)
    c.set_bias([[(1, 1.0)], [(2, 1.0)], [(3, 1.0)]])
    c.status.zero_()
    api.spec_adjust_logits(c.args(bias_start=np.array(start, np.int32)))
    torch.cuda.synchronize()
    assert int(c.status.item()) == oracle.DEV_BAD_PARAM
    s = np.array(start)
    bad = (s[:-1] < 0) | (s[1:] < s[:-1]) | (s[1:] > 3)
    assert torch.isnan(c.ot.float()).all(1).cpu().numpy().tolist() == bad.tolist()


@pytest.mark.parametrize("cu,skipped", [([0, 2, 1, 6], [2, 3, 4, 5]), ([-1, 2, 4, 6], [0, 1]),
                                        ([0, 2, 4, 7], [4, 5]), ([0, 2, 2, 6], [2, 3, 4, 5])])
def test_inconsistent_sequences_are_skipped(api, cu, skipped):
    c = Case(api, [2, 2, 2], 300, seed=13, table=False, penal=False, draft=False)
    c.max_rows = 3
    api.spec_adjust_logits(c.args(cu=dev(np.array(cu, np.int32))))
    torch.cuda.synchronize()
    assert int(c.status.item()) == oracle.DEV_BAD_LENGTH
    got = host_bits(c.ot)
    for r in range(6):
        if r in skipped:
            assert bool((c.ot[r] == 77).all()), r
        else:
            assert np.array_equal(got[r], c.target[r])


def test_draft_tokens_outside_the_vocabulary(api):
    c = Case(api, [4, 3], 1000, seed=14)
    c.tokens[:3] = [-1, 1000, 2 ** 31 - 1]
    c.run()


def test_captured_and_replayed_on_another_stream(api):
    c = Case(api, [3, 2], 2500, seed=15, ctx=2, masked=0.5, bias=3)
    a = c.args()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        api.spec_adjust_logits(a)
    for seed in (1, 2):
        c.target = _logits(np.random.default_rng(seed), c.target.shape, "bf16")
        c.dt.copy_(dev(c.target))
        graph.replay()
        torch.cuda.synchronize()
        c.check()
    c.ot.zero_()
    side.wait_stream(torch.cuda.current_stream())
    api.spec_adjust_logits(a, stream=side)
    side.synchronize()
    c.check()


def test_offsets_past_32_bits(api):
    """2.2 G logits in place: the last sequence's rows are right, the others stay."""
    B, K, V = 1075, 16, 128256
    x = torch.zeros(B * K, V, dtype=torch.bfloat16, device="cuda")
    x[-K:] = 1.0
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * K
    drafts = torch.full((B * (K - 1),), V - 1, dtype=torch.int32, device="cuda")
    pres = torch.zeros(B, device="cuda")
    pres[-1] = 0.5
    freq = torch.zeros(B, device="cuda")
    freq[-1] = 0.25
    api.spec_adjust_logits(api.adjust_args(x, x, cu, max_q_rows=K, draft_tokens=drafts,
                                           presences=pres, frequencies=freq))
    torch.cuda.synchronize()
    want = [1.0] + [1.0 - 0.5 - 0.25 * j for j in range(1, K)]
    assert x[-K:, V - 1].tolist() == want
    assert bool((x[-K:, :V - 1] == 1).all()) and float(x[:-K].abs().max()) == 0.0


def test_torch_call_refusals(api):
    c = Case(api, [2, 1], 100, seed=16, ctx=1, masked=1.0, bias=2)
    t, cu = dev(c.target), dev(c.cu)
    o = torch.empty_like(t)
    d = {k: dev(v) for k, v in c.kw.items()}

    def call(**kw):
        kw = dict(max_q_rows=2) | kw
        return api.adjust_args(kw.pop("target", t), kw.pop("out", o), kw.pop("cu", cu), **kw)

    call(**d)
    bad = [dict(target=t.half()), dict(out=o.float()), dict(out=o[:2]), dict(cu=cu.long()),
           dict(target=t[:, :50]), dict(draft=t[:1]), dict(draft=t, draft_out=o),
           dict(draft_tokens=cu[:2]), dict(counts=d["counts"]), dict(seen=d["seen"]),
           dict(counts=d["counts"], seen=d["seen"][:, :1]),
           dict(counts=d["counts"], seen=d["seen"], slots=cu),
           dict(repetition=0.0), dict(repetition=float("nan")), dict(repetitions=d["repetitions"].double()),
           dict(presences=d["presences"][:1]), dict(bias_start=d["bias_start"]),
           dict(bias_start=d["bias_start"], bias_tokens=d["bias_tokens"],
                bias_values=torch.zeros(d["bias_tokens"].numel() + 1, device="cuda")),
           dict(mask=d["mask"].long()), dict(mask=d["mask"], mask_rows=cu[:2]),
           dict(ctx_tokens=torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
           dict(ctx_tokens=torch.zeros(2, 2, dtype=torch.int32, device="cuda").t()),
           dict(dev_status=torch.zeros(1, device="cuda"))]
    for i, kw in enumerate(bad):
        with pytest.raises(ValueError):
            call(**kw)
            pytest.fail(f"call {i} was not refused")
    from speculative_decoding_verify_09_gb300._binding import SpecVerifyError
    with pytest.raises(SpecVerifyError, match="mask_stride"):
        api.spec_adjust_logits(call(mask=d["mask"][:, :2].contiguous(), mask_rows=d["mask_rows"]))
    with pytest.raises(SpecVerifyError, match="num_masks"):
        api.spec_adjust_logits(call(mask=d["mask"][:2].contiguous()))


# Shapes that every way of cutting the work takes: short chunks, long ones,
# single tokens changed in memory (in place, with sequences enough).
CUTS = [(6, 5003, False), (20, 32000, False), (20, 33001, False), (30, 65536, True), (30, 70003, True)]


@pytest.mark.parametrize("B,V,in_place", CUTS)
@pytest.mark.parametrize("few", [1, 40])
def test_blocks_of_repeated_drafts(api, B, V, in_place, few):
    """Blocks of 16 rows whose drafts are one token, or a few, next to the table's
    and the biased ones: each row counts the drafts before it alone."""
    c = Case(api, ([16, 1, 9] * B)[:B], V, seed=few, hist=200, ctx=2, bias=8, masked=0.2)
    near = c.rng.integers(0, V - 40)
    c.tokens[:] = near + c.rng.integers(0, few, len(c.tokens))
    c.kw["ctx_tokens"][0] = near
    c.set_bias([[(near, 0.5), (near + few, -1.0)]] * B)
    c.run(in_place)


@pytest.mark.parametrize("B,V,in_place", CUTS)
def test_failing_and_skipped_sequences_among_others(api, B, V, in_place):
    """A value, a slot and a mask row out of range give rows of NaN, and only there."""
    c = Case(api, ([2, 1, 3] * B)[:B], V, seed=V, hist=300, masked=0.3, bias=4)
    c.kw["repetitions"][1] = c.ref["repetition"][1] = np.nan
    slots = c.kw["slots"].copy()
    slots[2] = B + 2
    c.kw["slots"] = c.ref["slots"] = slots
    c.kw["mask_rows"][c.cu[4]] = c.ref["mask_rows"][c.cu[4]] = len(c.kw["mask"])
    c.run(in_place, status=oracle.DEV_BAD_PARAM)


@pytest.mark.parametrize("B,V,in_place", CUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_and_nan_in_rows(api, B, V, in_place, dtype):
    """Listed, plain and barred places that hold infinities, NaN or the lowest value."""
    c = Case(api, ([2, 1] * B)[:B], V, dtype, seed=3, hist=2000, masked=0.5, penal=False)
    ones = np.ones(B, np.float32)
    c.kw.update(repetitions=ones * 2, presences=ones * 0.5)
    c.ref.update(repetition=ones * 2, presence=ones * 0.5)
    low = np.float32(-3.3895314e38)             # the lowest bf16; a quarter, so that twice it is finite
    vals = np.array([np.inf, -np.inf, np.nan, low / 4, 0.0, -0.0], np.float32)
    x = vals[c.rng.integers(0, len(vals), c.target.shape)]
    at = c.rng.random(c.target.shape) < 0.2
    c.target = np.where(at, f32_to_bf16_bits(x) if dtype == "bf16" else x, c.target)
    c.run(in_place)


@pytest.mark.parametrize("B,V,in_place", CUTS)
def test_the_same_call_twice_gives_the_same_bits(api, B, V, in_place):
    c = Case(api, ([5, 2] * B)[:B], V, seed=8, hist=1500, ctx=3, bias=100, masked=0.3)
    got = []
    for _ in range(2):
        api.spec_adjust_logits(c.args(in_place))
        got.append((host_bits(c.ot).copy(), host_bits(c.od).copy()))
    assert all(np.array_equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("cu,skipped", [([2 ** 31 - 1, -2 ** 31 + 1, 4, 6], [0, 1, 2, 3]),
                                        ([2 ** 31 - 1, -2 ** 31, 4, 6], [0, 1, 2, 3]),
                                        ([0, 2 ** 31 - 1, -2 ** 31 + 2, 6], [0, 1, 2, 3, 4, 5])])
def test_row_bounds_whose_difference_wraps(api, cu, skipped):
    """Bounds so far apart that their 32-bit difference is a plausible number of rows."""
    c = Case(api, [2, 2, 2], 300, seed=23, table=False, penal=False, draft=False)
    c.max_rows = 3
    api.spec_adjust_logits(c.args(cu=dev(np.array(cu, np.int32))))
    torch.cuda.synchronize()
    assert int(c.status.item()) == oracle.DEV_BAD_LENGTH
    got = host_bits(c.ot)
    for r in range(6):
        if r in skipped:
            assert bool((c.ot[r] == 77).all()), r
        else:
            assert np.array_equal(got[r], c.target[r])


@pytest.mark.parametrize("B,V,in_place", CUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_repetition_quotient_is_rounded_once(api, B, V, in_place, dtype):
    """Prompt tokens under a repetition penalty alone: the fp32 product, and for logits
    between 2^-60 and 2^60 the fp32 quotient, to the bit (rounded again to bf16 there); a
    logit that equals the penalty becomes 1.  Farther positive logits are multiplied by
    the rounded reciprocal: two roundings of 2^-24 (or half of the least subnormal)."""
    c = Case(api, ([2, 1] * B)[:B], V, dtype, seed=31, draft=False, penal=False, hist=1)
    rng = c.rng
    r = np.exp(rng.uniform(-1, 1, B)).astype(np.float32)
    r[:4] = [1.1, 2.0 ** -64, 2.0 ** 64, 1.3]
    if dtype == "bf16":
        r[4:] = bf16_bits_to_f32(f32_to_bf16_bits(r[4:]))
    counts = np.where(rng.random((B + 2, V)) < 0.05, np.int32(-2 ** 31), 0).astype(np.int32)
    c.kw.update(counts=counts, seen=oracle.seen_bits(counts), repetitions=r)
    seq = np.repeat(np.arange(B), np.diff(c.cu))
    x = rng.standard_normal((c.R, V), dtype=np.float32) * np.float32(3)
    far = rng.random(x.shape) < 0.2
    x[far] *= np.exp2(rng.uniform(-140, 124, far.sum())).astype(np.float32)
    own = rng.random(x.shape) < 0.1
    x = np.where(own, r[seq][:, None], x)
    if dtype == "bf16":
        c.target = f32_to_bf16_bits(x)
        x = bf16_bits_to_f32(c.target)
    else:
        c.target = x
    api.spec_adjust_logits(c.args(in_place))
    torch.cuda.synchronize()
    with np.errstate(over="ignore", under="ignore"):
        want = np.where(x > 0, x / r[seq][:, None], x * r[seq][:, None])
    known = counts[c.kw["slots"][seq]] != 0
    for i in np.flatnonzero(np.diff(c.cu) == 2):        # the second row of a block knows its draft
        known[c.cu[i] + 1, c.tokens[c.cu[i] - i]] = True
    want = np.where(known, want, x)
    got = host_bits(c.ot)
    if dtype == "bf16":
        got = bf16_bits_to_f32(got)
        big = np.abs(want) >= np.float32(3.3961775e38)      # rounds past the largest bf16
        want = np.where(big, np.copysign(np.float32(np.inf), want),
                        bf16_bits_to_f32(f32_to_bf16_bits(np.where(big, 0, want))))
    far = known & (x > 0) & ((x < 2.0 ** -60) | (x > 2.0 ** 60))
    assert far.any() and np.array_equal(got[~far], want[~far])
    got, exact = got[far].astype(np.float64), (x.astype(np.float64) / r[seq][:, None])[far]
    top, half, least = (2.0 ** 128 * (1 - 2.0 ** -9), 2.0 ** -8, 2.0 ** -134) if dtype == "bf16" else \
        (2.0 ** 128 * (1 - 2.0 ** -25), 0.0, 0.0)
    two = 2.0 ** -23 * (1 + 2.0 ** -24)
    assert np.all(exact[np.isinf(got)] >= top * (1 - two))
    assert np.all(got[exact >= top * (1 + two)] == np.inf)
    fin = np.isfinite(got)
    assert np.all(np.abs(got - exact)[fin] <= ((two + half) * exact + 2.0 ** -149 + least)[fin])
    got = bf16_bits_to_f32(host_bits(c.ot)) if dtype == "bf16" else host_bits(c.ot)
    assert bool((got[known & own & (x == r[seq][:, None])] == 1).all())
    assert int(c.status.item()) == 0


def test_masks_and_tables_without_rows(api):
    """A mask of no rows has no row that could be named, and a table of no rows no slot."""
    c = Case(api, [2, 1], 100, seed=16)
    none = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    c.run(mask=none, mask_rows=np.full(3, -1, np.int32))                # nothing masked
    api.spec_adjust_logits(c.args(mask=none, mask_rows=np.array([-1, -1, 0], np.int32)))
    torch.cuda.synchronize()
    assert int(c.status.item()) == oracle.DEV_BAD_PARAM
    assert torch.isnan(c.ot.float()).all(1).tolist() == [False, False, True]
    from speculative_decoding_verify_09_gb300._binding import SpecVerifyError
    with pytest.raises(SpecVerifyError, match="num_masks"):
        api.spec_adjust_logits(c.args(mask=none))
    with pytest.raises(ValueError, match="row"):
        c.args(counts=torch.zeros(0, 100, dtype=torch.int32, device="cuda"), seen=none)


@pytest.mark.parametrize("B,V,in_place", CUTS)
def test_as_many_ctx_tokens_as_allowed_and_long_bias_lists(api, B, V, in_place):
    c = Case(api, ([2, 1] * B)[:B], V, seed=41, hist=300, ctx=1024, bias=6000, masked=0.2)
    near = c.rng.integers(0, V - 200)
    c.kw["ctx_tokens"][:20] = near + c.rng.integers(0, 100, (20, B))       # some of them often
    c.run(in_place)
    c = Case(api, ([3, 1] * B)[:B], V, "f32", seed=42, draft=False, table=False, bias=20000)
    c.run(in_place)
