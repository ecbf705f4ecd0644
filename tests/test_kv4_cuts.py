"""How spec_kv4_attn cuts its list of tiles (csrc/kv4_cuts.inl), compiled for the host and compared
with the same cutting in integers of any size: shares of CTAs and runs of warps ascend from 0 to the
end of the list, at lists up to the largest that the calls accept.

The list: sequences, their KV heads, parts of 8 NB rows, and of each HEAD units and one per tile.  Costs
(NB > 1): 6 a unit of HEAD and 3 + 2 columns a tile, or 1 each where the sum could pass 2^32."""
import bisect
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILE, HEAD, LEAST, SNAP = 32, 2, 4, 8
WARPS = {1: 16, 2: 12, 3: 8}
TOKENS = (1 << 31) - 16                # the most that a table accepted by the calls holds

DRIVER = r"""
#include "kv4_cuts.inl"
using namespace sv;
struct Params { int batch, g, weighted; };
template <int NB>
static int cuts(int batch, int heads, int g, int weighted, int grid, int warps, const int *rows, const int *len,
                int *start, uint32_t *cost, int *ends, int *runs) {
  const Params P{batch, g, weighted};
  const TileList<NB, Params> list{P, start, rows, len, cost};
  start[0] = 0, cost[0] = 0;
  for (int i = 0; i < batch; ++i) {
    const Amount n = rows[i] ? list.amount_of(rows[i], rows[i] + len[i], heads) : Amount{0, 0};
    start[i + 1] = start[i] + n.units, cost[i + 1] = cost[i] + n.cost;
  }
  if (start[batch] == 0) return 0;
  const int ctas = list.ctas_of(start[batch], grid);
  for (int x = 0; x <= ctas; ++x) ends[x] = list.share_from(x, ctas).unit;
  for (int x = 0; x < ctas; ++x)
    for (int y = 0; y <= warps; ++y)
      runs[x * (warps + 1) + y] = list.run_from(list.share_from(x, ctas), list.share_from(x + 1, ctas), y, warps);
  return ctas;
}
extern "C" int cut(int nb, int batch, int heads, int g, int weighted, int grid, int warps, const int *rows,
                   const int *len, int *start, uint32_t *cost, int *ends, int *runs) {
  auto f = nb == 1 ? cuts<1> : nb == 2 ? cuts<2> : cuts<3>;
  return f(batch, heads, g, weighted, grid, warps, rows, len, start, cost, ends, runs);
}
extern "C" void place(int nb, int batch, int g, const int *rows, const int *len, const int *start, int v, int *p) {
  const Params P{batch, g, 0};
  const TileList<1, Params> one{P, start, rows, len, nullptr};
  const TileList<2, Params> two{P, start, rows, len, nullptr};
  const TileList<3, Params> three{P, start, rows, len, nullptr};
  const Place at = nb == 1 ? one.locate(v) : nb == 2 ? two.locate(v) : three.locate(v);
  p[0] = at.i, p[1] = at.unit, p[2] = at.at, p[3] = at.tiles;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    at = tmp_path_factory.mktemp("cuts")
    (at / "cuts.cpp").write_text(DRIVER)
    csrc = os.path.join(ROOT, "speculative_decoding_verify_09_gb300", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-Wall", "-Werror", "-shared", "-fPIC",
                        "-I", csrc, "-o", str(at / "cuts.so"), str(at / "cuts.cpp")], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(at / "cuts.so"))


def ints(x):
    return np.ascontiguousarray(x, np.int32)


def ptr(x):
    return x.ctypes.data_as(ctypes.c_void_p)


class List:
    """The list and its cuts in Python's integers.  bound: tokens that the tables hold."""

    def __init__(self, rows, lens, heads, g, bound=None, max_rows=None):
        self.rows, self.lens, self.heads, self.g = list(map(int, rows)), list(map(int, lens)), heads, g
        max_rows = max_rows or max(self.rows)
        blocks = -(-max_rows * g // 8)
        parts = 1 if blocks <= 3 else (blocks + 1) // 2
        self.nb = -(-blocks // parts)
        parts = -(-blocks // self.nb)
        units = len(rows) * heads * parts
        bound = bound or max(n + r for n, r in zip(self.lens, self.rows))
        tiles = -(-bound // TILE)
        assert max_rows <= 1024 and max_rows * g <= 16384 and units <= 65536
        assert bound < 1 << 31 and units * (tiles + HEAD) < 1 << 31, "the calls refuse this"
        self.weighted = units * ((3 + 2 * self.nb) * tiles + 6 * HEAD) < 1 << 32
        self.start, self.cost = [0], [0]
        for i in range(len(rows)):
            segs = self.segments(i)
            self.start.append(self.start[-1] + heads * sum(HEAD + t for t, _ in segs))
            self.cost.append(self.cost[-1] + heads * sum(self.seg_cost(s) for s in segs))

    def segments(self, i):
        """(tiles, cost of one) of the parts of a KV head."""
        n = self.rows[i] * self.g
        if n == 0:
            return []
        tiles = -(-(self.lens[i] + self.rows[i]) // TILE)
        columns = [min(self.nb, -(-(n - at) // 8)) for at in range(0, n, 8 * self.nb)]
        return [(tiles, 3 + 2 * c if self.weighted else 1) for c in columns]

    def head_cost(self):
        return 6 * HEAD if self.weighted else HEAD

    def seg_cost(self, seg):
        return self.head_cost() + seg[0] * seg[1]

    def unit_at(self, v):
        """(sequence, unit of it, place in it, tiles) of list entry v."""
        i = bisect.bisect_right(self.start, v) - 1
        each = HEAD + self.segments(i)[0][0]
        return i, (v - self.start[i]) // each, (v - self.start[i]) % each, each - HEAD

    def cut_at(self, x):
        """(unit, place in its segment, units left of that, costs before and after) at cost x."""
        i = bisect.bisect_right(self.cost, x) - 1
        segs = self.segments(i)
        h, into = divmod(x - self.cost[i], sum(map(self.seg_cost, segs)))
        part = 0
        while into >= self.seg_cost(segs[part]):
            if part == 0 and segs[0] == segs[-2 if len(segs) > 1 else 0]:      # (full parts are alike)
                part = min(into // self.seg_cost(segs[0]), len(segs) - 1)
                into -= part * self.seg_cost(segs[0])
            else:
                into -= self.seg_cost(segs[part])
                part += 1
        tiles, one = segs[part]
        before = self.head_cost()
        at = into * HEAD // before if into < before else HEAD + (into - before) // one
        unit = self.start[i] + (h * len(segs) + part) * (HEAD + tiles) + at
        return unit, at, HEAD + tiles - at, into, self.seg_cost(segs[part]) - into

    def shares(self, ctas):
        """(unit, cost) of the shares' begins and of the end."""
        total, out = self.start[-1], []
        for x in range(ctas + 1):
            if self.nb == 1:
                v = total // ctas * x + min(x, total % ctas)
                if 0 < v < total:
                    _, _, at, tiles = self.unit_at(v)
                    left = HEAD + tiles - at
                    v += -at if at <= min(left, SNAP) else left if left <= SNAP else 0
                out.append((v, 0))
                continue
            sum_, v = self.cost[-1], 0 if x == 0 else total
            c = sum_ // ctas * x + min(x, sum_ % ctas)
            if 0 < x < ctas:
                v, at, left, into, rest = self.cut_at(c)
                if at <= min(left, SNAP):
                    v, c = v - at, c - into
                elif left <= SNAP:
                    v, c = v + left, c + rest
            out.append((v, c))
        return out

    def runs(self, a, b, warps):
        if self.nb == 1:
            return [a[0] + (b[0] - a[0]) * y // warps for y in range(warps + 1)]
        inner = [min(b[0], max(a[0], self.cut_at(a[1] + (b[1] - a[1]) * y // warps)[0])) if b[1] > a[1] else b[0]
                 for y in range(1, warps)]
        return [a[0], *inner, b[0]]

    def check(self, host, grid=152):
        B, warps = len(self.rows), WARPS[self.nb]
        start, cost, ends = np.zeros(B + 1, np.int32), np.zeros(B + 1, np.uint32), np.zeros(grid + 1, np.int32)
        runs = np.zeros((grid, warps + 1), np.int32)
        rows, lens = ints(self.rows), ints(self.lens)
        ctas = host.cut(self.nb, B, self.heads, self.g, int(self.weighted), grid, warps, ptr(rows), ptr(lens),
                        ptr(start), ptr(cost), ptr(ends), ptr(runs))
        assert start.tolist() == self.start
        if self.start[-1] == 0:
            return
        assert self.nb == 1 or cost.tolist() == self.cost
        assert ctas == max(1, min(grid, self.start[-1] // LEAST))
        ends, runs = ends[:ctas + 1], runs[:ctas]
        # in the list, in order, no share of a segment's inside without a unit
        assert ends[0] == 0 and ends[-1] == self.start[-1] and (np.diff(ends) >= 0).all(), ends
        assert (runs[:, 0] == ends[:-1]).all() and (runs[:, -1] == ends[1:]).all()
        assert (np.diff(runs, axis=1) >= 0).all()
        for x in np.flatnonzero(np.diff(ends) == 0):
            assert ends[x] == self.start[-1] or self.unit_at(int(ends[x]))[2] == 0, "a share without units"
        want = self.shares(ctas)
        assert ends.tolist() == [v for v, _ in want]
        for x in range(ctas):
            assert runs[x].tolist() == self.runs(want[x], want[x + 1], warps), x
        p = np.zeros(4, np.int32)
        for v in {int(v) for v in runs.reshape(-1)[::7] if v < self.start[-1]} | {0, self.start[-1] - 1}:
            host.place(self.nb, B, self.g, ptr(rows), ptr(lens), ptr(start), v, ptr(p))
            assert tuple(p) == self.unit_at(v), v


@pytest.mark.parametrize("grid", [1, 2, 152, 192])
@pytest.mark.parametrize("rows,g,tokens", [
    # parts times 7 times tiles from below 2^31 to 2^32: costs of one KV head
    (1024, 16, 9_000_000), (1024, 16, 9_580_000), (1024, 16, 9_586_981), (1024, 16, 9_590_000),
    (1024, 16, 12_000_000), (1024, 16, 19_100_000), (1024, 16, 19_170_000), (1024, 16, 19_180_000),
    (1024, 1, 154_000_000), (1000, 1, 300_000_000), (10, 8, 1_999_999_967), (9, 8, TOKENS - 40),
    # the most of few rows: one, two and three columns
    (1, 1, TOKENS - 48), (1, 16, TOKENS - 48), (3, 8, TOKENS - 48), (3, 6, TOKENS - 48), (2, 9, TOKENS - 48)])
def test_one_long_head(host, rows, g, tokens, grid):
    """Quotients of costs at and above 2^31."""
    List([rows], [tokens], 1, g).check(host, grid)


@pytest.mark.parametrize("rows,g", [(1, 1), (3, 6), (1, 16), (10, 8), (17, 1)])
@pytest.mark.parametrize("keys", range(TOKENS - 18, TOKENS + 1, 3))
def test_the_longest_sequences(host, rows, g, keys):
    """Lengths that, rounded up to tiles, pass 2^31."""
    List([rows], [keys - rows], 1, g).check(host)


@pytest.mark.parametrize("rows,lens,heads,g", [
    ([1024, 3, 0, 1024], [9_000_000, 5, 0, 9_100_000], 1, 16), ([1, 1024], [0, 19_000_000], 1, 16),
    ([1024, 1], [19_000_000, 0], 1, 16), ([24] * 7, [9_000_000] * 7, 8, 1), ([16] * 20, [5_000_000] * 20, 2, 8),
    ([700] * 3, [50_000_000] * 3, 1, 1), ([1] * 768, [60_000] * 768, 8, 8), ([2] * 700, [9_000] * 700, 8, 12)])
def test_several_long_sequences(host, rows, lens, heads, g):
    for grid in (7, 152):
        List(rows, lens, heads, g).check(host, grid)


@pytest.mark.parametrize("seed", range(40))
def test_ragged_lists(host, seed):
    rng = np.random.default_rng(seed)
    B = int(rng.integers(1, 60))
    g, heads = int(rng.choice([1, 2, 3, 4, 7, 8, 16])), int(rng.choice([1, 2, 5, 8]))
    rows = rng.integers(0, 10, B)
    rows[0] = max(rows[0], 1)
    lens = np.floor(np.exp(rng.uniform(0, np.log(rng.choice([40, 900, 20000])), B))).astype(int) - 1
    wide = 1 << 30 if seed % 4 == 3 and B * heads * g < 60 else None
    List(rows, lens, heads, g, bound=None if wide is None else wide // (B * heads * g)).check(host)
