"""GPU parity of spec_rope_rows with the float64 oracle.

Tolerances.  Per output: the angle's fixed-point fraction is rounded to fp32
(relative 2^-24 of at most pi: 1.9e-7 radians), sincospif is within 2 ulp
(2.4e-7 absolute) and the product with mscale, the two products and the sum
round at 2^-24 each: below 1e-6 m (|a| + |b|) in all.  The store rounds by half
a step of the type, eps / 2 of the value (fp32: included).  E4M3: the code is the
nearest one to a value within 1e-6 m (|a| + |b|) / scale (+ 2^-24 relative for
the division) of the exact quotient, so its distance to the exact quotient is
at most the nearest code's plus twice that."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host_bits
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


def _draw(rng, shape, dtype):
    x = rng.standard_normal(shape, dtype=np.float32)
    return f32_to_bf16_bits(x) if dtype == "bf16" else x


def _f64(x):
    return oracle.to_f64(x)


class Case:
    """Ragged rows cut out of one fused projection tensor, and their outputs."""

    def __init__(self, api, rows, Hq, Hkv, D, rot, dtype="bf16", layout="half", kv8=False, seed=0,
                 far=5000, extra_rows=0, mscale=1.0, k_scale=0.0625, v_scale=0.03, parts="qkv",
                 pad=0):
        rng = np.random.default_rng(seed)
        self.api, self.layout, self.kv8, self.dtype = api, layout, kv8, dtype
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        R = int(self.cu[-1]) + extra_rows
        self.R, self.live, self.D, self.mscale = R, int(self.cu[-1]), D, mscale
        self.k_scale, self.v_scale = np.float32(k_scale), np.float32(v_scale)
        self.kv_len = rng.integers(0, far, len(rows)).astype(np.int32)
        self.x = _draw(rng, (R, Hq + 2 * Hkv + pad, D), dtype)
        self.heads = {"q": slice(0, Hq), "k": slice(Hq, Hq + Hkv), "v": slice(Hq + Hkv, Hq + 2 * Hkv)}
        self.parts = parts
        self.freqs, _ = oracle.rope_frequencies(rot)
        self.turns, _ = api.rope_turns(rot)
        self.dx = dev(self.x)
        tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.out = {}
        for p in parts:
            h = self.heads[p].stop - self.heads[p].start
            if kv8 and p != "q":
                self.out[p] = torch.full((R, h, D), 0xAB, dtype=torch.uint8, device="cuda")
            else:
                self.out[p] = torch.full((R, h, D), 123.0, dtype=tdt, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.max_rows = max(max(rows), 1)

    def args(self, **kw):
        t = {p: (self.dx[:, self.heads[p]] if p in self.parts else None) for p in "qkv"}
        if "positions" not in kw:
            kw = dict(cu_q=dev(self.cu), kv_len=dev(self.kv_len), max_q_rows=self.max_rows) | kw
        return self.api.rope_args(
            t["q"], t["k"], t["v"], *(self.out.get(p) for p in "qkv"), self.turns,
            layout=self.layout, mscale=self.mscale, k_scale=float(self.k_scale),
            v_scale=float(self.v_scale), dev_status=self.status, **kw)

    def check(self, positions=None, rows=None):
        torch.cuda.synchronize()
        rows = np.arange(self.live) if rows is None else np.asarray(rows)
        pos = oracle.row_positions(self.cu, self.kv_len) if positions is None else positions
        pos = [int(pos[r]) for r in rows]
        eps = {"bf16": 2.0 ** -8, "f32": 0.0}[self.dtype]
        h = len(self.freqs)
        for p in self.parts:
            x = _f64(self.x[rows][:, self.heads[p]])
            got_t = self.out[p][torch.from_numpy(rows).cuda()]
            if p == "v":
                want, mag = x, np.zeros_like(x)
            else:
                want = oracle.rope_rows(x, pos, self.freqs, self.layout, self.mscale)
                a = np.abs(x)
                mag = np.zeros_like(x)
                if self.layout == "half":
                    both = a[..., :h] + a[..., h:2 * h]
                    mag[..., :h], mag[..., h:2 * h] = both, both
                else:
                    both = a[..., 0:2 * h:2] + a[..., 1:2 * h:2]
                    mag[..., 0:2 * h:2], mag[..., 1:2 * h:2] = both, both
            slack = 1e-6 * self.mscale * mag
            if self.kv8 and p != "q":
                scale = float(self.k_scale if p == "k" else self.v_scale)
                y = np.clip(want / scale, -448, 448)
                slack = slack / scale + 2.0 ** -24 * np.abs(y)
                got = oracle.sampling.e4m3_to_f64(got_t.cpu().numpy())
                best = np.abs(oracle.sampling.e4m3_to_f64(oracle.e4m3_nearest(y)) - y)
                assert np.all(np.abs(got - y) <= best + 2 * slack), p
                continue
            got = _f64(host_bits(got_t))
            if p == "v":
                assert np.array_equal(host_bits(got_t), self.x[rows][:, self.heads[p]])
                continue
            assert np.array_equal(got[..., 2 * h:], x[..., 2 * h:]), f"{p}: the unrotated part"
            assert np.all(np.abs(got - want) <= slack + eps * np.abs(want)), \
                (p, float(np.max(np.abs(got - want))))


SHAPES = [(128, 128), (64, 64), (128, 64), (128, 32), (64, 20), (80, 80), (8, 2), (16, 16),
          (256, 96), (256, 256), (128, 30), (40, 38), (96, 48), (24, 16), (72, 64), (128, 120),
          (256, 250), (256, 2)]


@pytest.mark.parametrize("D,rot", SHAPES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kv8", [False, True])
def test_parity_on_ragged_rows(api, D, rot, layout, dtype, kv8):
    c = Case(api, [1, 5, 2, 9, 1, 3], 6, 2, D, rot, dtype, layout, kv8, seed=D + rot)
    api.spec_rope_rows(c.args())
    c.check()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("D,rot,layout", [(128, 128, "half"), (64, 20, "half"),
                                          (128, 64, "interleaved")])
@pytest.mark.parametrize("dtype,kv8", [("bf16", False), ("bf16", True), ("f32", False)])
def test_many_rows(api, D, rot, layout, dtype, kv8):
    """Enough rows for the arrangement of prompts (several rows per CTA, all
    heads in one), an odd count, lengths from none to hundreds."""
    c = Case(api, [0, 701, 1, 0, 16, 130, 0], 5, 1, D, rot, dtype, layout, kv8, seed=11,
             mscale=1.2079)
    api.spec_rope_rows(c.args())
    c.check()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("Hq,Hkv,parts", [(1, 1, "qkv"), (32, 32, "qkv"), (71, 1, "qkv"),
                                          (4, 2, "q"), (4, 2, "k"), (4, 2, "v"), (4, 2, "qk"),
                                          (4, 2, "kv"), (4, 2, "qv")])
@pytest.mark.parametrize("rows", [[1] * 8, [300, 400]])
def test_heads_and_absent_tensors(api, Hq, Hkv, parts, rows):
    c = Case(api, rows, Hq, Hkv, 64, 64, parts=parts, kv8=parts in ("v", "kv"), pad=3)
    api.spec_rope_rows(c.args())
    c.check()


@pytest.mark.parametrize("longest", [3, 90])
def test_many_sequences(api, longest):
    rng = np.random.default_rng(longest)
    rows = rng.integers(0, 4, 5000).tolist()
    rows[77] = longest
    c = Case(api, rows, 2, 1, 16, 8, seed=3)
    api.spec_rope_rows(c.args())
    c.check(rows=np.concatenate([np.arange(40), np.arange(c.live - 40, c.live)]))
    assert int(c.status.item()) == 0
    assert bool((c.out["q"] != 123).flatten(1).any(1).all())


@pytest.mark.parametrize("n", [1, 5, 2000])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_positions_near_and_far(api, n, layout):
    rng = np.random.default_rng(n)
    c = Case(api, [n], 3, 1, 128, 128, "f32", layout, seed=n)
    pos = np.concatenate([[0, 2 ** 31 - 1, -(2 ** 31) + 1, 1, -1],
                          rng.integers(-2 ** 31 + 1, 2 ** 31, max(0, n - 5))])[:n].astype(np.int64)
    api.spec_rope_rows(c.args(positions=dev(pos)))
    c.check(positions=pos, rows=np.arange(min(n, 64)))
    assert int(c.status.item()) == 0


def test_positions_out_of_range_are_skipped(api):
    c = Case(api, [4], 2, 1, 64, 64)
    pos = np.array([3, 2 ** 31, -(2 ** 31), 9], dtype=np.int64)
    api.spec_rope_rows(c.args(positions=dev(pos)))
    c.check(positions=pos, rows=[0, 3])
    assert int(c.status.item()) == oracle.DEV_BAD_LENGTH
    for p in "qkv":
        assert bool((c.out[p][1:3] == 123).all())


@pytest.mark.parametrize("how", ["order", "long", "past", "negative", "length"])
def test_inconsistent_sequences_are_skipped(api, how):
    c = Case(api, [2, 2, 2], 2, 1, 64, 64, extra_rows=2)
    cu, kv = c.cu.copy(), c.kv_len.copy()
    skipped = {"order": [2, 3, 4, 5], "long": [4, 5], "past": [4, 5], "negative": [0, 1],
               "length": [2, 3]}[how]
    if how == "order":
        cu[2] = 1                       # sequence 1 ends before it starts, 2 is then too long
    elif how == "long":
        cu[3] = 7                       # 3 rows where the bound is 2
    elif how == "past":
        cu[3] = 9
    elif how == "negative":
        cu[0] = -1
    else:
        kv[1] = -3
    api.spec_rope_rows(c.args(cu_q=dev(cu), kv_len=dev(kv), max_q_rows=8 if how == "past" else 2))
    torch.cuda.synchronize()
    assert int(c.status.item()) == oracle.DEV_BAD_LENGTH
    c.check(rows=[r for r in range(6) if r not in skipped])
    for p in "qkv":
        assert bool((c.out[p][skipped] == 123).all()), (how, p)


@pytest.mark.parametrize("cu", [[0, 30, 10, 40, 60], [0, 20, 70, 71, 60], [-5, 20, 40, 50, 60],
                                [0, 20, 20, 20, 60], [0, 0, 0, 0, 0]])
def test_rows_that_search_their_sequence(api, cu):
    """A bound of 60 rows on four sequences of 60 rows in all: rows of sequences
    that are consistent are right or (where cu_q does not ascend) untouched."""
    c = Case(api, [20, 20, 10, 10], 3, 1, 64, 64, seed=6)
    a = np.array(cu)
    good = (a[:-1] >= 0) & (a[1:] >= a[:-1]) & (a[1:] <= 60)
    pos = np.zeros(60, dtype=np.int64)
    owner = np.full(60, -1)
    for i in range(4):
        if good[i]:
            owner[a[i]:a[i + 1]] = i
            pos[a[i]:a[i + 1]] = c.kv_len[i] + np.arange(a[i + 1] - a[i])
    api.spec_rope_rows(c.args(cu_q=dev(a.astype(np.int32)), max_q_rows=60))
    torch.cuda.synchronize()
    assert int(c.status.item()) == (0 if good.all() else oracle.DEV_BAD_LENGTH)
    touched = (c.out["v"] != 123).flatten(1).any(1).cpu().numpy()
    assert not touched[owner < 0].any()
    if good.all():
        assert touched[owner >= 0].all()
    if (np.bincount(np.concatenate([np.arange(a[i], a[i + 1]) for i in range(4) if good[i]] + [[0]])
                    .astype(int)) <= 2).all() and touched.any():
        alone = [r for r in np.flatnonzero(touched)
                 if sum(good[i] and a[i] <= r < a[i + 1] for i in range(4)) == 1]
        c.check(positions=pos, rows=alone)


def test_rows_behind_the_last_sequence_stay(api):
    for rows in ([2, 3], [400, 500]):
        c = Case(api, rows, 4, 2, 128, 128, extra_rows=9)
        api.spec_rope_rows(c.args(max_q_rows=c.max_rows + 4))
        c.check()
        for p in "qkv":
            assert bool((c.out[p][c.live:] == 123).all())
        assert int(c.status.item()) == 0


@pytest.mark.parametrize("D,rot,layout", [(128, 128, "half"), (64, 20, "half"), (80, 70, "half"),
                                          (256, 250, "half"), (64, 40, "interleaved")])
@pytest.mark.parametrize("rows", [[3, 1], [700, 20]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_equals_out_of_place(api, D, rot, layout, rows, dtype):
    c = Case(api, rows, 9, 3, D, rot, dtype, layout, seed=8)
    api.spec_rope_rows(c.args())
    c.check()
    own = {p: c.dx[:, c.heads[p]].contiguous() for p in "qkv"}
    a = api.rope_args(own["q"], own["k"], own["v"], own["q"], own["k"], own["v"], c.turns,
                      cu_q=dev(c.cu), kv_len=dev(c.kv_len), max_q_rows=c.max_rows, layout=layout)
    api.spec_rope_rows(a)
    torch.cuda.synchronize()
    for p in "qkv":
        assert torch.equal(own[p], c.out[p]), p


def test_gradients_go_back_by_negated_positions(api):
    """d/dx of sum(g * rope(x, t)) is rope(g, -t): the formula's transpose (pinned against
    differences on the oracle), and a rotation there and back restores x."""
    rng = np.random.default_rng(12)
    x, g = rng.standard_normal((2, 37, 4, 64)).astype(np.float32)
    pos = rng.integers(0, 2 ** 20, 37).astype(np.int64)
    turns, m = api.rope_turns(48, scaling="yarn", factor=4.0, trained_len=4096)
    dx, dg, y, back = dev(x), dev(g), *(torch.empty(37, 4, 64, device="cuda") for _ in range(2))
    for src, dst, p in ((dx, y, pos), (dg, back, -pos)):
        api.spec_rope_rows(api.rope_args(src, None, None, dst, None, None, turns, mscale=m,
                                         positions=dev(p)))
    torch.cuda.synchronize()
    lhs = float((y.double() * dg.double()).sum())
    rhs = float((back.double() * dx.double()).sum())
    # every term of either sum is off by at most 1e-6 m (|a| + |b|) |g|
    assert abs(lhs - rhs) <= 2e-6 * m * 2 * float((dx.abs().double() * dg.abs().double()).sum() +
                                                  dx.abs().double().sum())
    again = torch.empty_like(y)
    api.spec_rope_rows(api.rope_args(y, None, None, again, None, None, turns, positions=dev(-pos)))
    torch.cuda.synchronize()
    rot = again[..., :48] / m
    assert float((rot - dx[..., :48]).abs().max()) <= 2 * 1e-6 * 2 * float(dx.abs().max()) * 2


def test_special_values(api):
    c = Case(api, [2], 1, 1, 64, 32, kv8=True, k_scale=1.0, v_scale=1.0)
    v = c.dx[:, c.heads["v"]]
    v[0, 0, :8] = torch.tensor([500.0, -1e30, float("inf"), -float("inf"), float("nan"), 0.0, -0.0,
                                448.0])
    q = c.dx[:, c.heads["q"]]
    q[0, 0, 40:44] = torch.tensor([float("nan"), float("inf"), -0.0, 1e-40])   # the copied part
    before = host_bits(q)[0, 0, 32:].copy()
    api.spec_rope_rows(c.args())
    torch.cuda.synchronize()
    got = c.out["v"][0, 0, :8].tolist()
    assert got[:4] == [0x7E, 0xFE, 0x7E, 0xFE] and got[4] & 0x7F == 0x7F
    assert got[5:] == [0x00, 0x80, 0x7E]
    assert np.array_equal(host_bits(c.out["q"])[0, 0, 32:], before)


def test_captured_and_replayed_on_another_stream(api):
    c = Case(api, [3, 6, 1], 4, 2, 128, 128, kv8=True, seed=21)
    a = c.args()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        api.spec_rope_rows(a)
    rng = np.random.default_rng(5)
    for _ in range(2):
        c.x = _draw(rng, c.x.shape, "bf16")
        c.dx.copy_(dev(c.x))
        graph.replay()
        c.check()
    with torch.cuda.stream(side):
        for p in "qkv":
            c.out[p].zero_()
        api.spec_rope_rows(a)
    side.synchronize()
    c.check()
    other = c.args()
    api.spec_rope_rows(other, stream=side)
    side.synchronize()
    c.check()


def test_offsets_past_32_bits(api):
    """q of 2.2 G elements: the last rows are right."""
    R, H, D = 270_000, 64, 128
    q = torch.zeros(R, H, D, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(2)
    x = f32_to_bf16_bits(rng.standard_normal((3, H, D), dtype=np.float32))
    q[-3:] = dev(x)
    turns, _ = api.rope_turns(D)
    pos = torch.arange(R, device="cuda", dtype=torch.int64)
    api.spec_rope_rows(api.rope_args(q, None, None, q, None, None, turns, positions=pos))
    torch.cuda.synchronize()
    want = oracle.rope_rows(_f64(x), [R - 3, R - 2, R - 1], oracle.rope_frequencies(D)[0])
    got = bf16_bits_to_f32(host_bits(q[-3:])).astype(np.float64)
    assert np.all(np.abs(got - want) <= 1e-5 + 2.0 ** -8 * np.abs(want))
    assert float(q[:-3].abs().max()) == 0.0


def test_torch_call_refusals(api):
    x = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    turns, _ = api.rope_turns(64)
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    kv = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(4, dtype=torch.int64, device="cuda")
    ok = dict(cu_q=cu, kv_len=kv, max_q_rows=4)
    o = torch.empty_like(x)
    codes = torch.empty(4, 2, 64, dtype=torch.uint8, device="cuda")
    bad = [
        lambda: api.rope_args(None, None, None, None, None, None, turns, **ok),
        lambda: api.rope_args(x, None, None, None, None, None, turns, **ok),
        lambda: api.rope_args(x, None, None, o, None, None, turns),
        lambda: api.rope_args(x, None, None, o, None, None, turns, positions=pos, **ok),
        lambda: api.rope_args(x, None, None, o, None, None, turns, positions=pos.int()),
        lambda: api.rope_args(x, None, None, o, None, None, turns, positions=pos[:3]),
        lambda: api.rope_args(x, None, None, o, None, None, turns, layout="other", **ok),
        lambda: api.rope_args(x, None, None, codes, None, None, turns, **ok),
        lambda: api.rope_args(x, None, None, o.float(), None, None, turns, **ok),
        lambda: api.rope_args(x.half(), None, None, o.half(), None, None, turns, **ok),
        lambda: api.rope_args(x, x, x, o, codes, o, turns, **ok),
        lambda: api.rope_args(x, x, x[:, :1], o, o, o[:, :1], turns, **ok),
        lambda: api.rope_args(x[:1].expand(4, 2, 64), None, None, o, None, None, turns, **ok),
        lambda: api.rope_args(x.transpose(0, 1), None, None, o, None, None, turns, **ok),
        lambda: api.rope_args(x, None, None, o, None, None, turns.int(), **ok),
        lambda: api.rope_args(x, None, None, o[:, :1], None, None, turns, **ok),
        lambda: api.rope_args(x, None, None, o, None, None, turns, cu_q=cu.long(), kv_len=kv,
                              max_q_rows=4),
        lambda: api.rope_args(x, None, None, o, None, None, turns, cu_q=cu, kv_len=kv.repeat(2),
                              max_q_rows=4),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.parametrize("D,rot", [(64, 20), (128, 30), (40, 38), (72, 64), (256, 250), (24, 2), (64, 8), (128, 120)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_copied_elements_keep_any_bits(api, D, rot, layout, dtype):
    """Every bit pattern (NaN payloads, infinities, subnormals) behind the rotated part."""
    c = Case(api, [3, 70], 5, 2, D, rot, dtype, layout, seed=rot)
    rng = np.random.default_rng(D)
    word = np.uint16 if dtype == "bf16" else np.uint32
    x = c.x.view(word).copy()
    tail = rng.integers(0, 2 ** (8 * word().itemsize), x[..., rot:].shape, dtype=np.uint64).astype(word)
    nan = rng.random(tail.shape) < 0.3              # exponent all ones, some payload
    tail[nan] |= word(0x7F80 if dtype == "bf16" else 0x7F800000)
    x[..., rot:] = tail
    c.x = x.view(c.x.dtype)
    c.dx.copy_(dev(c.x))
    api.spec_rope_rows(c.args())
    torch.cuda.synchronize()
    for p in "qk":
        got = host_bits(c.out[p]).view(word)
        assert np.array_equal(got[..., rot:], tail[:, c.heads[p]]), p
        x[..., rot:] = 0                            # the turned part as always
    c.x = x.view(c.x.dtype)
    for p in "qk":
        c.out[p][..., rot:] = 0
    c.out["v"].copy_(dev(c.x)[:, c.heads["v"]])
    c.check()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_cos_and_sin_are_as_exact_as_fp32_has_them(api, layout):
    """Rows of (1, 0) pairs come out as (cos, sin).  The angle's only rounding is that of
    its distance x from the nearest quarter turn (2^-24 of pi |x|, which moves the value
    by that times its derivative), and sincospif is within 2 ulp (2^-22 of the value): near
    a half turn, where rounding the whole angle would cost 9e-8, the sine is good to its
    last bits."""
    R, pairs = 4096, 8
    rng = np.random.default_rng(17)
    f = rng.integers(0, 2 ** 63, pairs, dtype=np.uint64)
    f[0] = (1 << 63) + (1 << 46) + 12345        # a half turn and a little
    f[1] = (1 << 62) - (1 << 45) + 777          # a quarter turn less a little
    f[2] = (1 << 63) - (1 << 40) - 1
    f[3] = (1 << 61) + (1 << 47) + 99           # between the quarters
    f[4] = 1 << 62                              # quarter turns exactly
    pos = np.concatenate([np.arange(R - 8), [2 ** 31 - 1, -(2 ** 31) + 1, -1, -2, -3, -4, -5, 2 ** 30]])
    x = torch.zeros(R, 1, 2 * pairs, device="cuda")
    if layout == "half":
        x[..., :pairs] = 1.0
    else:
        x[..., 0::2] = 1.0
    y = torch.empty_like(x)
    api.spec_rope_rows(api.rope_args(x, None, None, y, None, None, dev(f.view(np.int64)), layout=layout,
                                     positions=dev(pos.astype(np.int64))))
    torch.cuda.synchronize()
    got = y[:, 0].cpu().numpy().astype(np.float64)
    cos, sin = (got[:, :pairs], got[:, pairs:]) if layout == "half" else (got[:, 0::2], got[:, 1::2])
    for p in range(pairs):
        part = [int(t) * int(f[p]) % 2 ** 64 for t in pos]
        quarter = [(v + 2 ** 61 >> 62) % 4 for v in part]
        rest = np.array([(v - (q << 62) + 2 ** 63) % 2 ** 64 - 2 ** 63 for v, q in zip(part, quarter)],
                        dtype=np.float64) * 2.0 ** -63              # half turns, at most 1 / 4
        assert np.abs(rest).max() <= 0.25
        s0, c0 = np.sin(np.pi * rest), np.cos(np.pi * rest)
        q = np.array(quarter)
        want_s = np.choose(q, [s0, c0, -s0, -c0])
        want_c = np.choose(q, [c0, -s0, -c0, s0])
        moved = np.pi * np.abs(rest) * 2.0 ** -24
        for g, w, d in ((sin[:, p], want_s, want_c), (cos[:, p], want_c, want_s)):
            assert np.all(np.abs(g - w) <= 2.0 ** -22 * np.abs(w) + moved * np.abs(d)), p


def test_no_rows_from_torch(api):
    """Calls with nothing to turn do nothing, by positions and by sequences."""
    turns, _ = api.rope_turns(64)
    x = torch.zeros(0, 2, 64, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for kw in (dict(positions=torch.zeros(0, dtype=torch.int64, device="cuda")),
               dict(cu_q=cu, kv_len=cu[:2], max_q_rows=4),
               dict(cu_q=cu[:1], kv_len=cu[:0], max_q_rows=1)):
        api.spec_rope_rows(api.rope_args(x, x, x, x, x, x, turns, dev_status=status, **kw))
    torch.cuda.synchronize()
    assert int(status.item()) == 0


def _prompt_rows(more=37):
    """More rows than pairs of rows can fill the SMs with, so that a CTA takes several
    rows side by side: 16, 8 or 4 by the heads and their columns, or still 2."""
    return 8 * torch.cuda.get_device_properties(0).multi_processor_count + more


def _ends_and_middle(n):
    return np.unique(np.concatenate([np.arange(33), n // 2 + np.arange(33), np.arange(n - 40, n)]))


WIDE = [(64, 64, "half"), (80, 80, "half"), (64, 24, "half"), (64, 20, "half"), (64, 22, "half"), (40, 36, "half"), (256, 250, "half"),
        (64, 64, "interleaved"), (80, 80, "interleaved"), (64, 20, "interleaved"), (72, 50, "interleaved")]


@pytest.mark.parametrize("D,rot,layout", WIDE)
@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (14, 7), (40, 5), (80, 5)])
@pytest.mark.parametrize("dtype,kv8", [("bf16", False), ("bf16", True), ("f32", False), ("f32", True)])
def test_rows_side_by_side(api, D, rot, layout, Hq, Hkv, dtype, kv8):
    """All ways a CTA shares its threads among rows, heads and columns, in even and odd
    numbers; sequences by slots (all about as long) and searched (a long one among
    short ones), rows behind the last one untouched."""
    n = _prompt_rows()
    for rows in ([n - n // 2, n // 2], [n - 63, 0, 1, 50, 12]):
        c = Case(api, rows, Hq, Hkv, D, rot, dtype, layout, kv8, seed=D + Hq, extra_rows=3, mscale=1.1)
        api.spec_rope_rows(c.args())
        c.check(rows=_ends_and_middle(n))
        assert int(c.status.item()) == 0
        for p in "qkv":
            untouched = 0xAB if kv8 and p != "q" else 123
            assert bool((c.out[p][n:] == untouched).all())
            assert bool((c.out[p][:n] != untouched).flatten(1).any(1).all())


@pytest.mark.parametrize("D,rot,layout", WIDE)
@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (14, 7), (40, 5)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_side_by_side_in_place_and_by_positions(api, D, rot, layout, Hq, Hkv, dtype):
    n = _prompt_rows(5)
    c = Case(api, [n], Hq, Hkv, D, rot, dtype, layout, seed=rot)
    api.spec_rope_rows(c.args())
    c.check(rows=_ends_and_middle(n))
    own = {p: c.dx[:, c.heads[p]].contiguous() for p in "qkv"}
    pos = dev(np.array(oracle.row_positions(c.cu, c.kv_len), dtype=np.int64))
    api.spec_rope_rows(api.rope_args(own["q"], own["k"], own["v"], own["q"], own["k"], own["v"], c.turns,
                                     positions=pos, layout=layout))
    torch.cuda.synchronize()
    for p in "qkv":
        assert torch.equal(own[p], c.out[p]), p


def test_rows_side_by_side_out_of_range(api):
    """Among many rows, those of bad positions and of bad sequences stay as they are."""
    n = _prompt_rows()
    c = Case(api, [n], 3, 1, 64, 64, seed=1)
    pos = np.arange(n, dtype=np.int64)
    bad = np.arange(7, n, 97)
    pos[bad] = np.where(bad % 2, 2 ** 31, -2 ** 40)
    api.spec_rope_rows(c.args(positions=dev(pos)))
    keep = np.setdiff1d(_ends_and_middle(n), bad)
    c.check(positions=pos, rows=keep)
    assert int(c.status.item()) == oracle.DEV_BAD_LENGTH
    assert bool((c.out["q"][torch.from_numpy(bad).cuda()] == 123).all())
    c = Case(api, [n // 4] * 4, 3, 1, 64, 64, seed=2)
    kv = c.kv_len.copy()
    kv[2] = -1
    api.spec_rope_rows(c.args(kv_len=dev(kv)))
    m = n // 4
    c.check(rows=np.concatenate([np.arange(2 * m - 20, 2 * m), np.arange(3 * m, 3 * m + 20)]))
    assert int(c.status.item()) == oracle.DEV_BAD_LENGTH
    for p in "qkv":
        assert bool((c.out[p][2 * m:3 * m] == 123).all())
