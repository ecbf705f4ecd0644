"""GPU parity of the paged 4-bit cache (spec_kv4_append, spec_kv4_read,
spec_kv4_attn) with the float64 oracle.

Tolerances.
 append: the stored element y is within `err` of the exact one (test_gpu_norm_rope.py).  The
  scale is the nearest E4M3 to a quotient within 2^-23 (its factor 6 f and itself
  rounded) of max / (6 f), the maximum within err; the code the nearest E2M1 to y over
  the unit that was stored, within err / unit and 2^-23 of the exact quotient.  So the
  distance of the code to the exact quotient is at most the nearest code's plus twice that.
 attn: the weights e^(s - max) have a relative error of 2^-11 (f16), 2^-21 (exp2 and the
  scaled score's rounding) and that of the score: D + 8 roundings of 2^-24 of the sum of
  |q k| (times the scale), twice, for numerator and denominator.  Weights below f16's
  normal range lose up to 2^-25 each (the running maximum is a score of the row, so weights
  relative to it are no smaller than relative to the true maximum).  fp32 sums over n
  tokens: n 2^-24 of the sum of magnitudes.  The output is rounded by half a step of bf16."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host_bits
from test_gpu_norm_rope import Case as RowCase
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

CAPACITY, BAD_LENGTH, TIMEOUT, BAD_PARAM = 1, 16, 32, 64


@pytest.fixture(scope="module")
def api():
    import speculative_decoding_verify_09_gb300 as pkg
    pkg.build()
    return pkg.load()


def paged(rng, lens, page, spare=3):
    """(table with -1 where no token is, pages in the pool)."""
    need = [-(-int(n) // page) for n in lens]
    total = sum(need) + spare
    ids = rng.permutation(total)
    table = np.full((len(lens), max(max(need, default=0), 1)), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    return table, total


def filled(rng, total, Hkv, page, D, k_scale=0.5, v_scale=0.25):
    """Pages of normal K and V as uint8 [total, Hkv, page / 16, 18 D]."""
    pages = np.empty((total, Hkv, page // 16, 18 * D), np.uint8)
    for which, f in ((0, k_scale), (1, v_scale)):
        codes, scales = oracle.kv4_quantize(rng.standard_normal((total, Hkv, page // 16, 16, D)), f)
        at = 9 * D * which
        both = codes[..., 0::2] | codes[..., 1::2] << 4
        pages[..., at:at + 8 * D] = both.reshape(*pages.shape[:3], -1)
        pages[..., at + 8 * D:at + 9 * D] = scales.reshape(*pages.shape[:3], -1)
    return pages


# ------------------------------------------------------------------ append
class Append(RowCase):
    def __init__(self, api, rows, Hq, Hkv, D, rot, page=64, k_scale=0.5, v_scale=0.25, far=200, **kw):
        super().__init__(api, rows, Hq, Hkv, D, rot, far=far, **kw)
        rng = np.random.default_rng(3)
        self.page, self.f = page, (np.float32(k_scale), np.float32(v_scale))
        self.table, total = paged(rng, self.kv_len + np.array(rows), page)
        self.cache = api.Kv4Cache(total, Hkv, D, page_size=page, k_scale=k_scale, v_scale=v_scale)
        self.cache.pages.random_(0, 256, generator=torch.Generator("cuda").manual_seed(1))
        self.before = self.cache.pages.cpu().numpy()

    def append(self, **kw):
        w = {p: None if x is None else dev(x) for p, x in self.weight.items()}
        q = dict(q=self.dx[:, self.heads["q"]], q_out=self.out["q"]) if "q" in self.parts else {}
        kw = dict(table=dev(self.table), cu_q=dev(self.cu), kv_len=dev(self.kv_len)) | kw
        return self.api.kv4_append_args(
            self.cache, kw.pop("table"), kw.pop("cu_q"), kw.pop("kv_len"), self.dx[:, self.heads["k"]],
            self.dx[:, self.heads["v"]], max_q_rows=self.max_rows, turns=self.turns, q_weight=w["q"],
            k_weight=w["k"], eps=self.eps, weight_offset=self.offset, layout=self.layout,
            mscale=self.mscale, dev_status=self.status, **q, **kw)

    def check_pages(self, skip=()):
        """Every stored row, and every other byte of the pool as it was."""
        from test_gpu_norm_rope import turned
        torch.cuda.synchronize()
        got = self.cache.pages.cpu().numpy()
        expect = self.before.copy()
        pos = oracle.row_positions(self.cu, self.kv_len)
        for i in range(len(self.cu) - 1):
            for r in range(self.cu[i], self.cu[i + 1]):
                for which, p in ((0, "k"), (1, "v")):
                    x = oracle.to_f64(self.x[r:r + 1, self.heads[p]])
                    y, err = turned(x, self.weight["k"], self.eps, self.offset, [pos[r]], self.freqs,
                                    self.layout, self.mscale) if p == "k" else (x, np.zeros_like(x))
                    for h in range(x.shape[1]):
                        if (r, h, p) in skip or r in skip:
                            continue
                        codes, scales = oracle.kv4_load(got, self.table[i:i + 1], self.page, 0, pos[r] + 1, h,
                                                        which)
                        self.check_row(codes[-1], scales[-1], y[0, h], err[0, h], float(self.f[which]),
                                       exact=p == "v")
                        oracle.kv4_store(expect, self.table, self.page, i, pos[r], h, which, codes[-1],
                                         scales[-1])
        assert np.array_equal(got, expect), "bytes beside the rows changed"

    def check_row(self, codes, scales, y, err, f, exact):
        if exact and np.log2(f) % 1 == 0 and self.dtype == "bf16":
            want = oracle.kv4_quantize(y, f)
            assert np.array_equal(codes, want[0]) and np.array_equal(scales, want[1])
            return
        y, err = y.reshape(-1, 16), err.reshape(-1, 16)
        e4 = oracle.sampling.e4m3_to_f64
        s = np.minimum(np.abs(y).max(-1) / (6 * f), 448)
        slack = err.max(-1) / (6 * f) + 2.0 ** -23 * s
        best = np.abs(e4(oracle.e4m3_nearest(s)) - s)
        assert np.all(np.abs(e4(scales) - s) <= best + 2 * slack)
        unit = e4(scales)[:, None] * f
        q = np.where(unit > 0, np.clip(y / np.where(unit > 0, unit, 1), -6, 6), 0)
        slack = np.where(unit > 0, err / np.where(unit > 0, unit, 1), 0) + 2.0 ** -23 * np.abs(q)
        best = np.abs(oracle.e2m1_to_f64(oracle.e2m1_nearest(q)) - q)
        assert np.all(np.abs(oracle.e2m1_to_f64(codes.reshape(-1, 16)) - q) <= best + 2 * slack)


@pytest.mark.parametrize("layout,rot", [("half", 128), ("half", 64), ("half", 48), ("half", 20),
                                        ("interleaved", 128), ("interleaved", 22), ("half", 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,page,f", [(128, 64, (0.5, 0.25)), (64, 16, (1.0, 2.0)), (128, 48, (0.3, 0.7)),
                                      (64, 4096, (2.0 ** -20, 2.0 ** 20))])
def test_append(api, layout, rot, dtype, D, page, f):
    c = Append(api, [1, 5, 0, 20], 4, 2, D, min(rot, D), page, *f, dtype=dtype, layout=layout, mscale=1.25,
               extra_rows=1, parts="q", seed=rot + D)
    api.spec_kv4_append(c.append())
    c.check()
    c.check_pages()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("rows,Hq,Hkv,norms", [([1] * 8, 32, 32, ""), ([300, 2], 0, 1, "k"),
                                               ([9] * 16, 8, 8, "qk"), ([1], 7, 7, "q")])
def test_append_rows_and_heads(api, rows, Hq, Hkv, norms):
    c = Append(api, rows, Hq, Hkv, 64, 64, 32, norms=norms, parts="q" if Hq else "")
    api.spec_kv4_append(c.append())
    c.check()
    c.check_pages()


def test_append_twice_overwrites(api):
    """Rows of rejected drafts stay behind the length, the next step writes over them."""
    c = Append(api, [6, 6], 2, 2, 64, 64, 16, parts="q")
    api.spec_kv4_append(c.append())
    c.check_pages()
    c.before = c.cache.pages.cpu().numpy()
    c.kv_len += np.array([1, 4], np.int32)
    c.table, total = np.pad(c.table, ((0, 0), (0, 1)), constant_values=-1), c.cache.num_pages
    free = [p for p in range(total) if p not in c.table]
    for i in range(2):
        for at in range(-(-(int(c.kv_len[i]) + 6) // 16)):
            if c.table[i, at] < 0:
                c.table[i, at] = free.pop()
    api.spec_kv4_append(c.append())
    c.check_pages()


def test_append_special_values(api):
    """Zeros, blocks too small for a scale, saturation, infinities; a NaN takes its 16 elements."""
    c = Append(api, [3], 2, 1, 64, 0, 16, 1.0, 1.0, dtype="f32", norms="", parts="q")
    x = np.zeros((3, 4, 64), np.float32)
    x[0, 2, :16], x[0, 2, 16:32] = 1e-4, 1e9
    x[0, 3, 5], x[0, 3, 20], x[0, 3, 33] = np.inf, -np.inf, np.nan
    x[0, 3, 48:] = np.arange(16) - 7.5
    x[1, 2:, :] = -0.0
    x[2, 2, 3] = np.nan
    c.x = x
    c.dx.copy_(torch.from_numpy(x))
    api.spec_kv4_append(c.append())
    torch.cuda.synchronize()
    got = c.cache.pages.cpu().numpy()
    n = int(c.kv_len[0])
    for which, h in ((0, 2), (1, 3)):
        codes, scales = oracle.kv4_load(got, c.table, 16, 0, n + 3, 0, which)
        for r in range(3):
            want = oracle.kv4_quantize(x[r, h].astype(np.float64), 1.0)
            assert np.array_equal(scales[n + r], want[1]), (which, r)
            nan = np.repeat(want[1] == 0x7F, 16)
            assert np.array_equal(codes[n + r][~nan], want[0][~nan]), (which, r)


def test_append_problems(api):
    """Each sequence's problem is its own: bad length, behind the table, bad pages; q all the same."""
    c = Append(api, [4, 4, 4, 4, 4], 2, 2, 64, 64, 16, far=20, parts="q")
    c.kv_len[:] = [3, -1, 14, 14, 20]
    c.table = np.array([[0, -1], [1, 2], [3, -1], [4, 9999], [5, 6]], np.int32)
    c.cache = api.Kv4Cache(8, 2, 64, page_size=16, k_scale=0.5, v_scale=0.25)
    c.before = c.cache.pages.cpu().numpy()
    api.spec_kv4_append(c.append())
    torch.cuda.synchronize()
    assert int(c.status.item()) == BAD_LENGTH | BAD_PARAM
    bad = list(range(4, 8))
    c.check(rows=[r for r in range(20) if r not in bad])
    assert bool((c.out["q"][4:8] == 123.0).all())
    c.check_pages(skip=set(bad) | {10, 11, 14, 15})
    c.status.zero_()
    c.kv_len[:] = [30, 0, 0, 0, 0]                       # rows 2 and 3 of the first behind the table
    c.table = np.array([[0, 1], [2, 2], [3, 3], [4, 4], [5, 5]], np.int32)
    c.before = c.cache.pages.cpu().numpy()
    api.spec_kv4_append(c.append())
    torch.cuda.synchronize()
    assert int(c.status.item()) == CAPACITY
    c.check_pages(skip={2, 3})
    c.check()


def test_append_and_attention_far_in_a_large_pool(api):
    """Pages whose bytes begin behind 2^32."""
    D, Hkv, page = 128, 8, 64
    page_bytes = Hkv * 4 * 18 * D
    total = (1 << 32) // page_bytes + 40
    rows = [2, 3]
    c = Append(api, rows, 16, Hkv, D, 128, page, far=150, parts="q")
    pages = torch.zeros(total, Hkv, 4, 18 * D, dtype=torch.uint8, device="cuda")
    c.cache = api.Kv4Cache(total, Hkv, D, page_size=page, k_scale=0.5, v_scale=0.25, pages=pages)
    rng = np.random.default_rng(0)
    need = c.table.shape[1] * 2
    top = np.arange(total - need, total)
    far = c.table.copy()
    small = np.full_like(far, -1)
    ids = iter(rng.permutation(need))
    for i in range(2):
        for at in range(-(-(int(c.kv_len[i]) + rows[i]) // page)):
            small[i, at] = next(ids)
            far[i, at] = top[small[i, at]]
    fill = filled(rng, need, Hkv, page, D)
    pages[total - need:] = dev(fill)
    api.spec_kv4_append(c.append(table=dev(far)))
    torch.cuda.synchronize()
    c.before, c.table = fill, small
    tail = pages[total - need:]
    assert not bool(pages[:need].any())
    big, c.cache = c.cache, api.Kv4Cache(need, Hkv, D, page_size=page, pages=tail)
    c.check_pages()
    q = c.out["q"]
    out = torch.empty_like(q)
    args = api.kv4_attn_args(big, dev(far), dev(c.cu), dev(c.kv_len), q, out, max_q_rows=3)
    api.spec_kv4_attn(args, api.kv4_workspace(args))
    torch.cuda.synchronize()
    close(out, q, tail.cpu().numpy(), small, page, c.cu, c.kv_len)


# -------------------------------------------------------------------- read
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
@pytest.mark.parametrize("D,page,Hkv,rows", [(128, 64, 2, [1, 70, 0, 3]), (64, 16, 5, [40]),
                                             (128, 48, 1, [1] * 30), (64, 32, 16, [9] * 20)])
def test_read(api, dtype, D, page, Hkv, rows):
    rng = np.random.default_rng(D + len(rows))
    kv_len = rng.integers(0, 100, len(rows)).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    R = int(cu[-1])
    table, total = paged(rng, kv_len + np.array(rows), page)
    pages = rng.integers(0, 256, (total, Hkv, page // 16, 18 * D)).astype(np.uint8)
    f, to = (0.5, 0.25), (np.float32(0.125), np.float32(0.03))
    cache = api.Kv4Cache(total, Hkv, D, page_size=page, k_scale=f[0], v_scale=f[1], pages=dev(pages))
    fill = 0x2B if dtype == torch.uint8 else 123.0
    out = [torch.full((R + 2, Hkv, D), fill, dtype=dtype, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.spec_kv4_read(api.kv4_read_args(cache, dev(table), dev(cu), dev(kv_len), *out,
                                        max_q_rows=max(rows), k_scale=float(to[0]), v_scale=float(to[1]),
                                        dev_status=status))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for which in range(2):
        got = host_bits(out[which])
        assert (got[R:] == host_bits(torch.full((1,), fill, dtype=dtype))[0]).all()
        for i in range(len(rows)):
            for h in range(Hkv):
                n, L = rows[i], int(kv_len[i])
                codes, scales = oracle.kv4_load(pages, table, page, i, L + n, h, which)
                want = oracle.kv4_values(codes[L:], scales[L:], f[which])
                x = got[cu[i]:cu[i + 1], h]
                if dtype == torch.uint8:
                    y = np.clip(want / float(to[which]), -448, 448)
                    nan = np.isnan(want)
                    assert ((x[nan] & 0x7F) == 0x7F).all()
                    e4 = oracle.sampling.e4m3_to_f64
                    y, x = y[~nan], x[~nan]
                    best = np.abs(e4(oracle.e4m3_nearest(y)) - y)
                    assert np.all(np.abs(e4(x) - y) <= best + 2 * 2.0 ** -24 * np.abs(y))
                else:
                    assert np.array_equal(oracle.to_f64(x), want, equal_nan=True)


@pytest.mark.parametrize("f,to", [((0.3, 1.7), (0.3, 0.1)), ((64.0, 2.0 ** -9), (1.0, 1.0)),
                                  ((2.0 ** -30, 2.0 ** 30), (2.0 ** -33, 2.0 ** 27)),
                                  ((0.5, 0.5), (2.0 ** -6, 2.0 ** 5))])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
def test_read_scales(api, f, to, dtype):
    """Factors that do and do not fit f16, and quotients of them that are no powers of two.  Values:
    one rounding of fp32 (and one of bf16); codes: the quotient of a value so rounded, rounded."""
    rng = np.random.default_rng(5)
    D, Hkv, page, n = 64, 3, 16, 40
    pages = rng.integers(0, 256, (3, Hkv, 1, 18 * D)).astype(np.uint8)
    cache = api.Kv4Cache(3, Hkv, D, page_size=page, k_scale=f[0], v_scale=f[1], pages=dev(pages))
    table = np.array([[2, 0, 1]], np.int32)
    out = [torch.zeros(n, Hkv, D, dtype=dtype, device="cuda") for _ in range(2)]
    api.spec_kv4_read(api.kv4_read_args(cache, dev(table), dev(np.array([0, n], np.int32)),
                                        dev(np.array([5], np.int32)), *out, max_q_rows=n, k_scale=to[0],
                                        v_scale=to[1]))
    torch.cuda.synchronize()
    e4 = oracle.sampling.e4m3_to_f64
    for which in range(2):
        got = host_bits(out[which])
        for h in range(Hkv):
            codes, scales = oracle.kv4_load(pages, table, page, 0, 5 + n, h, which)
            want = oracle.kv4_values(codes[5:], scales[5:], float(np.float32(f[which])))
            nan = np.isnan(want)
            if dtype == torch.uint8:
                y = np.clip(want / float(np.float32(to[which])), -448, 448)[~nan]
                assert ((got[:, h][nan] & 0x7F) == 0x7F).all()
                best = np.abs(e4(oracle.e4m3_nearest(y)) - y)
                assert np.all(np.abs(e4(got[:, h][~nan]) - y) <= best + 2 * 3 * 2.0 ** -24 * np.abs(y))
                continue
            got_h = oracle.to_f64(got[:, h])
            assert np.isnan(got_h[nan]).all()
            eps = 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0)
            assert np.all(np.abs(got_h - want)[~nan] <= eps * (1 + 2.0 ** -20) * np.abs(want)[~nan])
            if np.log2(f[which]) % 1 == 0:
                assert np.array_equal(got_h, want, equal_nan=True)


def test_read_parts_and_problems(api):
    rng = np.random.default_rng(2)
    D, Hkv, page = 64, 2, 16
    pages = filled(rng, 6, Hkv, page, D)
    cache = api.Kv4Cache(6, Hkv, D, page_size=page, k_scale=0.5, v_scale=0.25, pages=dev(pages))
    table = np.array([[0, 1], [2, 77], [3, 4]], np.int32)
    cu, kv_len = np.array([0, 4, 8, 12], np.int32), np.array([30, 14, 2], np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((12, Hkv, D), 5.0, device="cuda")
    for which, pair in ((0, (out, None)), (1, (None, out))):
        out.fill_(5.0)
        status.zero_()
        api.spec_kv4_read(api.kv4_read_args(cache, dev(table), dev(cu), dev(kv_len), *pair, max_q_rows=4,
                                            dev_status=status))
        torch.cuda.synchronize()
        assert int(status.item()) == CAPACITY | BAD_PARAM
        got = out.cpu().numpy()
        for r in range(12):
            i, pos = r // 4, int(kv_len[r // 4]) + r % 4
            if r in (2, 3, 6, 7):
                assert (got[r] == 5.0).all()
                continue
            for h in range(Hkv):
                codes, scales = oracle.kv4_load(pages, table, page, i, pos + 1, h, which)
                assert np.array_equal(got[r, h], oracle.kv4_values(codes[-1], scales[-1], (0.5, 0.25)[which]))


# --------------------------------------------------------------- attention
def close(out, q, pages, table, page, cu, kv_len, scale=0.0, f=(0.5, 0.25), rows=None):
    bits = host_bits(q)
    want, mag, small, reach = oracle.kv4_attention(bits, pages, table, page, cu, kv_len, scale, *f)
    D = q.shape[2]
    n = np.concatenate([int(kv_len[i]) + 1 + np.arange(cu[i + 1] - cu[i]) for i in range(len(cu) - 1)] or [[]])
    R = len(n)
    weight = 2.0 ** -11 + 2.0 ** -21 + 2 * (D + 8) * 2.0 ** -24 * reach[:R] + n[:, None] * 2.0 ** -24
    tol = 2.0 ** -8 * np.abs(want[:R]) + 1.01 * (weight[..., None] * mag[:R] + 2.0 ** -25 * small[:R])
    got = oracle.to_f64(host_bits(out))[:R]
    live = np.arange(R) if rows is None else np.asarray(rows)
    bad = ~(np.abs(got - want[:R]) <= tol)[live]
    assert not bad.any(), (live[np.argwhere(bad)[0][0]], np.argwhere(bad)[:3], got[live][bad][:4],
                           want[:R][live][bad][:4])


class Attn:
    def __init__(self, api, kv_len, rows, Hq, Hkv, D, page=64, seed=0, garbage=0xFF, extra_rows=0, pad=0):
        rng = np.random.default_rng(seed)
        self.api, self.page = api, page
        self.kv_len, self.rows = np.array(kv_len, np.int32), list(rows)
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        lens = [n + r if r else 0 for n, r in zip(kv_len, rows)]
        self.table, total = paged(rng, lens, page)
        self.pages = filled(rng, total, Hkv, page, D)
        if garbage is not None:        # whatever no token needs: NaN scales, codes of +-6
            used = np.zeros((total, page), bool)
            for i, n in enumerate(lens):
                for t in range(n):
                    used[self.table[i, t // page], t % page] = True
            wild = np.full(D, 15, np.uint8), np.full(D // 16, garbage, np.uint8)
            for p, t in np.argwhere(~used):
                for h in range(Hkv):
                    for which in (0, 1):
                        oracle.kv4_store(self.pages, np.array([[p]]), page, 0, t, h, which, *wild)
        self.cache = api.Kv4Cache(total, Hkv, D, page_size=page, k_scale=0.5, v_scale=0.25,
                                  pages=dev(self.pages))
        R = int(self.cu[-1]) + extra_rows
        x = f32_to_bf16_bits(rng.standard_normal((R, Hq + pad, D), dtype=np.float32))
        self.q = dev(x).view(torch.bfloat16)[:, :Hq]
        self.out = torch.full((R, Hq, D), 123.0, dtype=torch.bfloat16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.max_rows = max(max(rows), 1)

    def args(self, **kw):
        t = kw.pop("table", None)
        return self.api.kv4_attn_args(self.cache, dev(self.table) if t is None else t, dev(self.cu),
                                      dev(self.kv_len), self.q, self.out,
                                      max_q_rows=kw.pop("max_q_rows", self.max_rows),
                                      dev_status=self.status, **kw)

    def run(self, ws=None, **kw):
        a = self.args(**kw)
        self.api.spec_kv4_attn(a, ws or self.api.kv4_workspace(a))
        torch.cuda.synchronize()

    def check(self, rows=None, **kw):
        close(self.out, self.q.contiguous(), self.pages, self.table, self.page, self.cu, self.kv_len,
              rows=rows, **kw)
        assert bool((self.out[int(self.cu[-1]):] == 123.0).all())


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("Hq,Hkv,rows", [
    (4, 4, [1, 1, 1, 1]), (4, 4, [6, 1, 3, 0]), (8, 2, [3, 4, 1, 2]), (8, 1, [2, 1, 2, 1]),
    (8, 2, [6, 5, 0, 1]), (4, 1, [9, 8, 2, 7]), (3, 1, [16, 1, 5, 2]), (12, 4, [5, 5, 5, 5]),
    (16, 1, [5, 1, 2, 4]), (2, 2, [40, 3, 1, 33])])
@pytest.mark.parametrize("page", [16, 48, 64])
def test_attention_rows(api, D, Hq, Hkv, rows, page):
    c = Attn(api, [0, 70, 31, 200], rows, Hq, Hkv, D, page, seed=Hq + rows[0], extra_rows=2, pad=1)
    c.run()
    c.check()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("page", [16, 32, 128])
def test_attention_lengths(api, D, page):
    """Every length around the slabs', tiles' and pages' ends, single rows."""
    lens = list(range(0, 68)) + [95, 96, 97, 127, 128, 129, 255, 256, 257, 511, 512, 513]
    c = Attn(api, lens, [1] * len(lens), 2, 1, D, page, seed=page)
    c.run()
    c.check()


@pytest.mark.parametrize("Hq,Hkv,lens,rows", [
    (1, 1, [20000], [1]), (24, 1, [17000], [1]), (5, 1, [14000], [1]), (16, 1, [13000, 0], [2, 1]),
    (4, 1, [9000, 1], [4, 2]), (8, 1, [5000], [3]), (32, 32, [600, 1500], [1, 6]),
    (8, 8, [3001, 10, 0, 700], [2, 5, 1, 3])])
def test_attention_cut_segments(api, Hq, Hkv, lens, rows):
    """Long segments over many CTAs, several segments in one."""
    c = Attn(api, lens, rows, Hq, Hkv, 128, 64, garbage=None)
    c.run()
    c.check()
    first = c.out.clone()
    ws = api.kv4_workspace(c.args())
    for _ in range(3):                  # the joins go in order: the same bits every time
        c.out.fill_(0)
        c.run(ws)
        assert torch.equal(c.out, first)


@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 1), (128, 8), (128, 12)])
def test_attention_of_the_largest_batch(api, D, Hq):
    """768 sequences, most of a few tokens, some without rows."""
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 40, 768)
    lens[100], rows = 900, rng.integers(0, 3, 768)
    c = Attn(api, lens, rows, Hq, 1, D, 16, garbage=None)
    c.run()
    c.check()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("g", [64, 256])
def test_attention_many_query_heads(api, g):
    c = Attn(api, [50, 300], [2, 1], g, 1, 64, 16)
    c.run()
    c.check()


@pytest.mark.parametrize("Hq,rows,bound", [(8, [600, 3], 1024), (2, [1024, 0], 1024)])
def test_attention_of_long_blocks(api, Hq, rows, bound):
    """Hundreds of parts (of which the host's bound allows more than there are)."""
    c = Attn(api, [40, 70], rows, Hq, 1, 64, 16)
    c.run(max_q_rows=bound)
    c.check()
    assert int(c.status.item()) == 0


def test_attention_scales_at_fp32s_ends(api):
    """A scale that underflows with the factor weighs all tokens alike, and masks hold."""
    c = Attn(api, [37], [3], 2, 1, 128, 16)
    c.cache.k_scale = 2.0 ** -64
    c.run(scale=2.0 ** -126)
    close(c.out, c.q.contiguous(), c.pages, c.table, 16, c.cu, c.kv_len, scale=2.0 ** -126,
          f=(2.0 ** -64, 0.25))


def test_attention_large_scores(api):
    """Scores that grow along the sequence and overflow exp without a maximum."""
    c = Attn(api, [500, 90], [2, 3], 4, 2, 128, 64)
    c.q *= 30
    c.run(scale=2.0)
    c.check(scale=2.0)


def test_attention_of_infinite_and_nan_queries(api):
    """Stay with their row and head."""
    c = Attn(api, [100], [4], 4, 2, 128)
    c.q[1, 2, 5], c.q[2, 0, 0], c.q[3, 3, 9] = float("nan"), float("inf"), 1e30
    c.run()
    got = c.out.float()
    for r, h in ((1, 2), (2, 0), (3, 3)):
        assert not bool(got[r, h].isfinite().any())
        c.q[r, h], c.out[r, h] = 0, 0
    assert bool(c.out.float().isfinite().all())
    keep = c.out.clone()
    c.run()
    for r, h in ((1, 2), (2, 0), (3, 3)):
        c.out[r, h] = 0
    assert torch.equal(keep, c.out)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("L", [0, 15, 40, 63])
def test_nan_in_a_later_draft_does_not_reach_earlier_rows(api, D, L):
    """Block token 3's K in one head, block token 2's V in some elements of another."""
    c = Attn(api, [L, 9], [6, 2], 4, 2, D, 16)
    nan = np.full(D // 16, 0x7F, np.uint8)
    codes, scales = oracle.kv4_load(c.pages, c.table, 16, 0, L + 4, 0, 0)
    oracle.kv4_store(c.pages, c.table, 16, 0, L + 3, 0, 0, codes[-1], nan)
    codes, scales = oracle.kv4_load(c.pages, c.table, 16, 0, L + 3, 1, 1)
    scales = scales[-1].copy()
    scales[1] = 0xFF
    oracle.kv4_store(c.pages, c.table, 16, 0, L + 2, 1, 1, codes[-1], scales)
    c.cache.pages.copy_(dev(c.pages))
    c.run()
    got = c.out.float().cpu().numpy()
    assert np.isnan(got[3:6, 0:2]).all() and np.isfinite(got[:3, 0:2]).all()
    assert np.isnan(got[2:6, 2:4, 16:32]).all() and np.isfinite(got[:2, 2:4]).all()
    assert np.isfinite(np.delete(got[2:6, 2:4], slice(16, 32), axis=-1)).all()
    c.check(rows=[0, 1, 6, 7])


def test_nan_in_a_seen_token_reaches_every_row(api):
    c = Attn(api, [40], [3], 2, 2, 128)
    codes, scales = oracle.kv4_load(c.pages, c.table, 64, 0, 11, 1, 1)
    scales = scales[-1].copy()
    scales[7] = 0x7F
    oracle.kv4_store(c.pages, c.table, 64, 0, 10, 1, 1, codes[-1], scales)
    c.cache.pages.copy_(dev(c.pages))
    c.run()
    got = c.out.float().cpu().numpy()
    assert np.isnan(got[:, 1, 112:]).all()
    got[:, 1, 112:] = 0
    assert np.isfinite(got).all()


def test_attention_problems(api):
    """Each sequence's problem is its own."""
    c = Attn(api, [100, 20, 30, 50, 200], [2, 2, 2, 2, 2], 4, 2, 128, 16, garbage=None)
    want = c.table.copy()
    c.table[2, 1] = c.cache.num_pages            # needed page outside the pool
    c.table[3, 0] = -2
    c.kv_len[1] = -5
    c.run()
    assert int(c.status.item()) == BAD_LENGTH | BAD_PARAM
    assert bool((c.out[2:4] == 123.0).all())
    assert bool(c.out[4:8].isnan().all())
    c.table = want
    c.kv_len[1] = 20
    c.check(rows=[0, 1, 8, 9])
    c.status.zero_()
    c.kv_len[1] = 16 * c.table.shape[1] - 1      # passes the table by a token
    c.out.fill_(123.0)
    c.run()
    assert int(c.status.item()) == CAPACITY
    assert bool((c.out[2:4] == 123.0).all())
    c.kv_len[1] = 20
    c.check(rows=[0, 1, 4, 5, 6, 7, 8, 9])
    c.status.zero_()
    c.cu[2] = c.cu[1] - 1                        # sequence 1 ends before it begins, 2 has too many rows
    c.out.fill_(123.0)
    c.run()
    assert int(c.status.item()) == BAD_LENGTH
    assert bool((c.out[2:6] == 123.0).all()) and not bool((c.out[6:] == 123.0).any())


def test_attention_of_no_rows(api):
    c = Attn(api, [5, 0, 7], [0, 0, 0], 2, 1, 64, extra_rows=3)
    c.run()
    assert bool((c.out == 123.0).all()) and int(c.status.item()) == 0


def test_strided_table_and_shared_pages(api):
    """Two sequences over the same prefix pages, in a wider table."""
    c = Attn(api, [128, 128], [1, 1], 4, 2, 128, 64, garbage=None)
    c.table[1, :2] = c.table[0, :2]
    wide = torch.full((2, 9), -7, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = dev(c.table)
    c.run(table=wide[:, :c.table.shape[1]])
    c.check()


def test_tables_far_wider_than_the_lengths(api):
    """Bounds at which the list of tiles could hold hundreds of millions of units."""
    c = Attn(api, [70 * i for i in range(20)], [3, 1, 2, 0] * 5, 8, 1, 64, 4096, garbage=None)
    wide = torch.full((20, 1 << 18), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = dev(c.table)
    c.run(table=wide)
    c.check()
    assert int(c.status.item()) == 0


def test_one_workspace_for_many_shapes(api):
    """Larger and smaller calls in turn, counters at zero in between."""
    cases = [Attn(api, [700, 20], [2, 5], 8, 2, 128, garbage=None), Attn(api, [3000], [1], 1, 1, 64, garbage=None),
             Attn(api, [90] * 30, [9] * 30, 16, 4, 128, 16, garbage=None)]
    args = [c.args() for c in cases]
    ws = max((api.kv4_workspace(a) for a in args), key=lambda w: w.nbytes)
    for a in args + args[::-1] + args:
        api.spec_kv4_attn(a, ws)
    torch.cuda.synchronize()
    for c in cases:
        c.check()
    assert not bool(ws.buf[ws.ptr - ws.buf.data_ptr():][:4 * 24 * 192].any())


def test_two_graphs_share_a_workspace_with_eager_calls(api):
    cases = [Attn(api, [700, 20], [2, 5], 8, 2, 128, garbage=None), Attn(api, [2000], [4], 4, 1, 128, garbage=None)]
    args = [c.args() for c in cases]
    ws = max((api.kv4_workspace(a) for a in args), key=lambda w: w.nbytes)
    graphs = []
    for a in args:
        api.spec_kv4_attn(a, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.spec_kv4_attn(a, ws)
        graphs.append(g)
    for c in cases:
        c.out.fill_(0)
    for g in graphs + graphs:
        g.replay()
        api.spec_kv4_attn(args[0], ws)
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_two_streams_with_a_workspace_each(api):
    cases = [Attn(api, [1500, 300], [2, 5], 8, 8, 128, seed=s, garbage=None) for s in range(2)]
    args = [c.args() for c in cases]
    ws = [api.kv4_workspace(a) for a in args]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, w, s in zip(args, ws, streams):
            api.spec_kv4_attn(a, w, stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_waits_that_run_out_return_with_a_status(api):
    """At one poll waits run out while their copies are in flight; the call ends, the status says
    so, and after the bound is restored and the workspace zeroed all is as before."""
    B, Hkv, D, page, L = 4, 8, 128, 64, 20000
    n = -(-(L + 1) // page)
    cache = api.Kv4Cache(B * n, Hkv, D, page_size=page)
    slabs = cache.pages.view(-1, 2, 9 * D)
    slabs[..., :8 * D].random_(0, 256, generator=torch.Generator("cuda").manual_seed(2))
    slabs[..., 8 * D:] = 0x38
    table = torch.randperm(B * n, device="cuda").to(torch.int32).view(B, n)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    kv_len = torch.full((B,), L, dtype=torch.int32, device="cuda")
    q = torch.randn(B, 2 * Hkv, D, device="cuda").bfloat16()
    out, status = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    a = api.kv4_attn_args(cache, table, cu, kv_len, q, out, max_q_rows=1, dev_status=status)
    ws = api.kv4_workspace(a)
    api.spec_kv4_attn(a, ws)
    want = out.clone()
    assert int(status.item()) == 0 and bool(want.isfinite().all())
    seen = False
    try:
        api.sv_set_wait_limit(1)
        for _ in range(3):
            status.zero_()
            api.spec_kv4_attn(a, ws)
            torch.cuda.synchronize()                 # returns: no wait is endless
            seen |= int(status.item()) == TIMEOUT
    finally:
        api.sv_set_wait_limit(0)
    assert seen, "a one-poll bound never ran out"
    ws.zero()
    status.zero_()
    out.zero_()
    api.spec_kv4_attn(a, ws)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(out, want)


def test_torch_checks(api):
    c = Attn(api, [20], [1], 2, 1, 64)
    i32 = torch.int32
    with pytest.raises(ValueError, match="dtype"):
        api.kv4_attn_args(c.cache, dev(c.table), dev(c.cu), dev(c.kv_len), c.q.float(), c.out, max_q_rows=1)
    with pytest.raises(ValueError, match="table"):
        api.kv4_attn_args(c.cache, dev(c.table)[0], dev(c.cu), dev(c.kv_len), c.q, c.out, max_q_rows=1)
    with pytest.raises(ValueError, match="table"):
        api.kv4_attn_args(c.cache, torch.zeros(1, 4, dtype=i32, device="cuda").t(), dev(c.cu),
                          dev(c.kv_len), c.q, c.out, max_q_rows=1)
    with pytest.raises(ValueError, match="out"):
        api.kv4_attn_args(c.cache, dev(c.table), dev(c.cu), dev(c.kv_len), c.q, c.out[:, :1], max_q_rows=1)
    with pytest.raises(ValueError, match="kv_len"):
        api.kv4_attn_args(c.cache, dev(c.table), dev(c.cu), dev(c.cu), c.q, c.out, max_q_rows=1)
    k = torch.zeros(1, 2, 64, device="cuda")
    with pytest.raises(ValueError, match="cache of 1 heads"):
        api.kv4_append_args(c.cache, dev(c.table), dev(c.cu), dev(c.kv_len), k, k, max_q_rows=1)
    with pytest.raises(ValueError, match="q_weight"):
        api.norm_rope_args(k, None, None, k, None, None, q_weight=torch.zeros(32, device="cuda"),
                           cu_q=dev(c.cu), kv_len=dev(c.kv_len), max_q_rows=1)
