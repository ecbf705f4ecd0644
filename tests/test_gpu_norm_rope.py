"""GPU parity of spec_norm_rope_rows with the float64 oracle.

Tolerances.  The sum of squares of D <= 256 elements: two chains of 8 fused products in a
lane, one sum of the two, 4 sums across lanes at most, all of positive terms: within 13
roundings of 2^-24; times 1 / D (itself rounded) plus eps in one fused product: 15.  The
root halves them, 7.5, and its reciprocal is within 2 ulp, 4 roundings; weight + offset and
two products, 3: below 17 roundings, i.e. 1.02e-6 of the normed element.  The rotation adds
1e-6 m (|a| + |b|) (derived in test_gpu_rope.py).  The store rounds by half a step of the
type."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host_bits
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

NORM = 1.02e-6


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


def draw(rng, shape, dtype):
    x = rng.standard_normal(shape, dtype=np.float32)
    return f32_to_bf16_bits(x) if dtype == "bf16" else x


def turned(x, weight, eps, offset, positions, freqs, layout, mscale):
    """(exact value, tolerance before the store) of q or k rows."""
    y = x if weight is None else oracle.head_norm(x, weight, eps, offset)
    err = np.zeros_like(y) if weight is None else NORM * np.abs(y)
    if freqs is None:
        return y, err
    want = oracle.rope_rows(y, positions, freqs, layout, mscale)
    h = len(freqs)
    one = (slice(0, h), slice(h, 2 * h)) if layout == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    part = (1e-6 + (NORM if weight is not None else 0)) * mscale * \
        (np.abs(y[..., one[0]]) + np.abs(y[..., one[1]]))
    for s in one:
        err[..., s] = part
    return want, err


class Case:
    """Ragged rows cut out of one fused projection tensor, and their outputs."""

    def __init__(self, api, rows, Hq, Hkv, D, rot, dtype="bf16", layout="half", kv8=False, seed=0,
                 far=5000, extra_rows=0, mscale=1.0, eps=1e-6, offset=0.0, norms="qk", parts="qkv"):
        rng = np.random.default_rng(seed)
        self.api, self.layout, self.kv8, self.dtype = api, layout, kv8, dtype
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        R = int(self.cu[-1]) + extra_rows
        self.R, self.live, self.D, self.mscale = R, int(self.cu[-1]), D, mscale
        self.eps, self.offset, self.parts = eps, offset, parts
        self.scale = {"k": np.float32(0.0625), "v": np.float32(0.03)}
        self.kv_len = rng.integers(0, far, len(rows)).astype(np.int32)
        self.x = draw(rng, (R, Hq + 2 * Hkv, D), dtype)
        self.heads = {"q": slice(0, Hq), "k": slice(Hq, Hq + Hkv), "v": slice(Hq + Hkv, Hq + 2 * Hkv)}
        self.weight = {p: (rng.standard_normal(D).astype(np.float32) if p in norms else None) for p in "qk"}
        self.freqs = oracle.rope_frequencies(rot)[0] if rot else None
        self.turns = api.rope_turns(rot)[0] if rot else None
        self.dx = dev(self.x)
        if dtype == "bf16":
            self.dx = self.dx.view(torch.bfloat16)
        self.out = {}
        for p in parts:
            h = self.heads[p].stop - self.heads[p].start
            if kv8 and p != "q":
                self.out[p] = torch.full((R, h, D), 0xAB, dtype=torch.uint8, device="cuda")
            else:
                self.out[p] = torch.full((R, h, D), 123.0, dtype=self.dx.dtype, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.max_rows = max(max(rows), 1)

    def args(self, **kw):
        t = {p: (self.dx[:, self.heads[p]] if p in self.parts else None) for p in "qkv"}
        if "positions" not in kw:
            kw = dict(cu_q=dev(self.cu), kv_len=dev(self.kv_len), max_q_rows=self.max_rows) | kw
        w = {p: None if x is None else dev(x) for p, x in self.weight.items()}
        return self.api.norm_rope_args(
            t["q"], t["k"], t["v"], *(self.out.get(p) for p in "qkv"), self.turns, q_weight=w["q"],
            k_weight=w["k"], eps=self.eps, weight_offset=self.offset, layout=self.layout,
            mscale=self.mscale, k_scale=float(self.scale["k"]), v_scale=float(self.scale["v"]),
            dev_status=self.status, **kw)

    def check(self, positions=None, rows=None):
        torch.cuda.synchronize()
        rows = np.arange(self.live) if rows is None else np.asarray(rows)
        pos = oracle.row_positions(self.cu, self.kv_len) if positions is None else positions
        pos = [int(pos[r]) for r in rows]
        eps = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[self.dtype]
        for p in self.parts:
            x = oracle.to_f64(self.x[rows][:, self.heads[p]])
            got = host_bits(self.out[p][torch.from_numpy(rows).cuda()])
            if p == "v":
                want, err = x, np.zeros_like(x)
                if not self.kv8:
                    assert np.array_equal(got, self.x[rows][:, self.heads[p]])
                    continue
            else:
                want, err = turned(x, self.weight[p], self.eps, self.offset, pos, self.freqs, self.layout,
                                   self.mscale)
            if self.kv8 and p != "q":
                s = float(self.scale[p])
                y = np.clip(want / s, -448, 448)
                slack = err / s + 2.0 ** -24 * np.abs(y)
                best = np.abs(oracle.sampling.e4m3_to_f64(oracle.e4m3_nearest(y)) - y)
                assert np.all(np.abs(oracle.sampling.e4m3_to_f64(got) - y) <= best + 2 * slack), p
            else:
                got = oracle.to_f64(got)
                bad = np.abs(got - want) > err * (1 + eps) + eps * np.abs(want)
                assert not bad.any(), (p, np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])
        if self.live < self.R:                 # rows behind the last sequence
            for p, o in self.out.items():
                fill = 0xAB if o.dtype == torch.uint8 else 123.0
                assert bool((o[self.live:] == fill).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,kv8", [("bf16", False), ("bf16", True), ("f32", False), ("f32", True)])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 64), (128, 64), (128, 20), (96, 96), (80, 38), (8, 8),
                                   (8, 2), (72, 48), (256, 256), (256, 16), (136, 128), (16, 16), (24, 24)])
def test_shapes(api, D, rot, dtype, kv8, layout):
    c = Case(api, [1, 3, 0, 2], 6, 2, D, rot, dtype, layout, kv8, seed=D + rot, mscale=1.25, extra_rows=2)
    api.spec_norm_rope_rows(c.args())
    c.check()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("norms", ["", "q", "k", "qk"])
@pytest.mark.parametrize("rot", [0, 64])
def test_which_are_normed(api, norms, rot):
    c = Case(api, [2, 5], 3, 2, 64, rot, "f32", norms=norms, offset=1.0, eps=1e-3)
    api.spec_norm_rope_rows(c.args())
    c.check()


@pytest.mark.parametrize("Hq,Hkv,parts", [(1, 1, "qkv"), (5, 0, "q"), (0, 3, "kv"), (48, 8, "qkv"), (7, 7, "qk")])
@pytest.mark.parametrize("rows", [[1], [1] * 40, [700], [33, 1, 500, 0, 2], [9] * 64])
def test_heads_and_rows(api, Hq, Hkv, parts, rows):
    c = Case(api, rows, Hq, Hkv, 128, 128, parts=parts, seed=len(rows))
    api.spec_norm_rope_rows(c.args())
    c.check()


def test_positions_and_no_rotation_agree_with_rows_alone(api):
    """Explicit positions (negative ones among them); without a table only norms."""
    c = Case(api, [6], 2, 2, 64, 64, "f32")
    pos = np.array([0, -5, 1 << 30, -(1 << 31) + 1, 77, (1 << 31) - 1])
    api.spec_norm_rope_rows(c.args(positions=torch.from_numpy(pos).cuda()))
    c.check(positions=pos)


def test_without_norms_it_is_the_rotary_operator(api):
    """Bit for bit: both round the same exact angles and the same products."""
    for layout, D, rot in (("half", 128, 128), ("interleaved", 128, 64), ("half", 64, 20)):
        c = Case(api, [3, 9, 1], 4, 2, D, rot, "bf16", layout, norms="")
        api.spec_norm_rope_rows(c.args())
        got = {p: o.clone() for p, o in c.out.items()}
        api.spec_rope_rows(api.rope_args(
            *(c.dx[:, c.heads[p]] for p in "qkv"), *(c.out[p] for p in "qkv"), c.turns, cu_q=dev(c.cu),
            kv_len=dev(c.kv_len), max_q_rows=c.max_rows, layout=layout))
        for p in "qkv":
            # (fused products may be contracted otherwise: one rounding of fp32 before the store)
            same = (got[p] == c.out[p]).float().mean().item()
            assert same > 0.999, (layout, p, same)


@pytest.mark.parametrize("Hq,Hkv,parts", [(5, 3, "qv"), (0, 20, "v"), (37, 11, "qkv"), (2, 1, "qv"), (3, 30, "kv")])
@pytest.mark.parametrize("rows", [[3], [900], [400, 0, 211]])
@pytest.mark.parametrize("D,dtype,kv8", [(128, "bf16", False), (64, "f32", True), (136, "bf16", True)])
def test_some_kinds_of_heads(api, Hq, Hkv, parts, rows, D, dtype, kv8):
    """Tensors left out, and heads of several kinds with one CTA, the last ones fewer than it has places."""
    c = Case(api, rows, Hq if "q" in parts else 0, Hkv, D, D, dtype, "interleaved" if D == 128 else "half", kv8,
             seed=Hq, parts=parts)
    api.spec_norm_rope_rows(c.args())
    c.check()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_many_heads_in_place(api, layout):
    c = Case(api, [700], 32, 8, 128, 128, "bf16", layout)
    t = {p: c.dx[:, c.heads[p]].contiguous() for p in "qkv"}
    c.out = t
    w = {p: dev(x) for p, x in c.weight.items()}
    api.spec_norm_rope_rows(api.norm_rope_args(
        t["q"], t["k"], t["v"], t["q"], t["k"], t["v"], c.turns, q_weight=w["q"], k_weight=w["k"],
        cu_q=dev(c.cu), kv_len=dev(c.kv_len), max_q_rows=c.max_rows, layout=layout))
    c.check()


def test_in_place(api):
    for layout, rot in (("half", 64), ("half", 20), ("interleaved", 64)):
        c = Case(api, [4, 2], 2, 2, 64, rot, "f32", layout)
        t = {p: c.dx[:, c.heads[p]].contiguous() for p in "qkv"}
        c.out = t
        w = {p: dev(x) for p, x in c.weight.items()}
        api.spec_norm_rope_rows(api.norm_rope_args(
            t["q"], t["k"], t["v"], t["q"], t["k"], t["v"], c.turns, q_weight=w["q"], k_weight=w["k"],
            cu_q=dev(c.cu), kv_len=dev(c.kv_len), max_q_rows=c.max_rows, layout=layout, k_scale=1.0))
        c.check()


def test_zeros_large_and_small_rows(api):
    """A row of zeros stays zero with an eps; magnitudes whose squares stay in range keep their norm."""
    c = Case(api, [4], 1, 1, 128, 0, "f32", parts="qk", eps=1e-30)
    c.x[0], c.x[1], c.x[2] = 0.0, c.x[1] * 1e17, c.x[2] * 1e-13
    c.dx.copy_(torch.from_numpy(c.x))
    api.spec_norm_rope_rows(c.args())
    c.check()
    assert bool((c.out["q"][0] == 0).all())


def test_nan_and_infinity_stay_with_their_head(api):
    c = Case(api, [3], 4, 2, 128, 128, "f32")
    clean = {p: o for p, o in c.out.items()}
    api.spec_norm_rope_rows(c.args())
    want = {p: o.clone() for p, o in clean.items()}
    c.dx[1, 2, 7], c.dx[2, 4, 9] = float("nan"), float("inf")      # q head 2 of row 1, k head 0 of row 2
    api.spec_norm_rope_rows(c.args())
    assert bool(c.out["q"][1, 2].isnan().all()) and bool(c.out["k"][2, 0, 9].isnan())
    c.out["q"][1, 2], want["q"][1, 2] = 0, 0
    c.out["k"][2, 0], want["k"][2, 0] = 0, 0
    for p in "qkv":
        assert torch.equal(c.out[p], want[p])


@pytest.mark.parametrize("rows,max_rows", [([2, 3, 2], 0), ([20, 300, 1], 300)])
def test_bad_sequences(api, rows, max_rows):
    c = Case(api, rows, 2, 2, 64, 64)
    c.max_rows = max_rows or c.max_rows
    c.kv_len[1] = -1
    api.spec_norm_rope_rows(c.args())
    torch.cuda.synchronize()
    assert int(c.status.item()) == 16
    assert bool((c.out["q"][c.cu[1]:c.cu[2]] == 123.0).all())
    keep = [r for r in range(c.live) if not c.cu[1] <= r < c.cu[2]]
    c.check(rows=keep)


@pytest.mark.parametrize("B", [33, 70, 1100])
def test_many_ragged_sequences(api, B):
    """Rows that search their sequence, over one, two and three rounds of a warp; some have none."""
    rng = np.random.default_rng(B)
    rows = list(rng.integers(0, 3, B))
    rows[B // 2], rows[-1] = 60, 0
    c = Case(api, rows, 2, 1, 64, 64, "bf16", seed=B, extra_rows=3)
    assert c.max_rows > 16 and B * c.max_rows > 1.25 * c.R
    api.spec_norm_rope_rows(c.args())
    c.check()
    assert int(c.status.item()) == 0


def test_streams_and_graphs(api):
    c = Case(api, [5, 1, 4], 8, 2, 128, 128)
    args = c.args()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    api.spec_norm_rope_rows(args, stream=s)
    s.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.spec_norm_rope_rows(args)
    x = draw(np.random.default_rng(9), c.x.shape, "bf16")
    for o in c.out.values():
        o.fill_(0)
    c.x = x
    c.dx.copy_(dev(x).view(torch.bfloat16))
    g.replay()
    c.check()


@pytest.mark.parametrize("D,rot,dtype", [(128, 20, "bf16"), (256, 250, "f32")])
def test_a_first_call_may_be_a_captured_one(api, D, rot, dtype):
    """Partners far apart, which take more shared memory than a kernel has by default; two calls in one
    graph, the second on the first one's rows."""
    c = Case(api, [70, 3, 40], 8, 2, D, rot, dtype, norms="")
    t = {p: c.dx[:, c.heads[p]].contiguous() for p in "qk"}
    back = {p: torch.zeros_like(x) for p, x in t.items()}
    where = torch.tensor(oracle.row_positions(c.cu, c.kv_len), dtype=torch.int64, device="cuda")
    there = api.norm_rope_args(t["q"], t["k"], None, c.out["q"], c.out["k"], None, c.turns, positions=where)
    again = api.norm_rope_args(c.out["q"], c.out["k"], None, back["q"], back["k"], None, c.turns,
                               positions=-where)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.spec_norm_rope_rows(there)
        api.spec_norm_rope_rows(again)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for p in "qk":                     # turned and turned back: two roundings of each of a pair
        x = t[p].double()
        size = torch.sqrt(2 * (x ** 2).amax()).item()
        assert (back[p].double() - x).abs().max().item() <= 4 * size * {"bf16": 2.0 ** -8, "f32": 2.0 ** -22}[dtype]
        assert not torch.equal(c.out[p][:, :, :rot], t[p][:, :, :rot])
