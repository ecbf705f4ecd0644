// How spec_kv4_attn's list of tiles is cut into shares for CTAs and runs for their
// warps.  Integers only, and host code compiles this as well.
//
// A segment is (sequence, KV head, part of the block's rows); its units are kHead and
// one for each tile of its tokens.  Sequences follow one another in the list, their
// heads, parts and tiles in this order.  Where parts have several columns of 8 rows
// (NB > 1) the cuts are equal in cost, not in units.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SV_BOTH __host__ __device__ __forceinline__
#else
#define SV_BOTH inline
#endif

namespace sv {

namespace {

constexpr int kTile = 32;                            // tokens
// Units that a segment costs beside its tiles (32 ragged sequences of 2 to 9 rows of 4 heads and 13
// small ragged sequences 1: 62.3 and 6.7 us, 2: 58.6 and 6.7, 4: 57.9 and 7.0).
constexpr int kHead = 2;
// Units of a CTA's share at least (the small sequences 6.7 us, with 16 7.5), and by how many it may
// end early or late to end with a segment (0: the same small sequences 8.3 us, 8: 6.7; 16: shares
// so unequal that 8 sequences of 32 heads take 19.2 us instead of 18.5).
constexpr int kLeast = 4;
constexpr int kSnap = 8;

// Units of the list, and what they cost.
struct Amount {
  int units;
  uint32_t cost;
};

// Where a share begins.
struct Cut {
  int unit;
  uint32_t cost;
};

// Sequence, unit (head * parts + part) and place in it of a list entry.
struct Place {
  int i, unit, at, tiles;
};

SV_BOTH float quick_quotient(float a, float b) {     // within 2^-21 of a / b
#ifdef __CUDA_ARCH__
  return __fdividef(a, b);
#else
  return a / b;
#endif
}

SV_BOTH int less_of(int a, int b) { return a < b ? a : b; }
SV_BOTH int more_of(int a, int b) { return a > b ? a : b; }

// a / d where that is below 2^16: by floats it is off by one at most.  (Costs go up to 2^32: their
// remainder takes 33 bits and a sign.)
SV_BOTH int quotient(uint32_t a, uint32_t d) {
  const uint32_t q = static_cast<uint32_t>(quick_quotient(static_cast<float>(a), static_cast<float>(d)));
  const int64_t rem = static_cast<int64_t>(a) - static_cast<int64_t>(static_cast<uint64_t>(q) * d);
  return static_cast<int>(q) + (rem < 0 ? -1 : rem >= static_cast<int64_t>(d) ? 1 : 0);
}

// x * y / n for y up to n (a few), without a product that passes x's type.
template <typename T>
SV_BOTH T share_of(T x, T y, T n) { return x / n * y + x % n * y / n; }

// Params: batch, g (query heads of a KV head), weighted (costs of tiles by their columns).
template <int NB, typename Params>
struct TileList {
  const Params &P;
  const int32_t *start;                              // [batch + 1] units before a sequence
  const int32_t *rows, *len;                         // [batch] block rows, and tokens before them
  const uint32_t *cost;                              // [batch + 1] costs before a sequence (NB > 1)

  // (unsigned: the longest sequences, rounded up, pass 2^31)
  SV_BOTH int tiles_of(int keys) const { return (static_cast<uint32_t>(keys) + (kTile - 1)) / kTile; }
  SV_BOTH int parts_of(int block_rows) const { return (block_rows * P.g + 8 * NB - 1) / (8 * NB); }

  // Costs of a tile with so many columns (two take 1.4 times as long as one; with equal costs the
  // ragged verify rows take 59.6 us instead of 58.6), of a segment beside its tiles, and of a
  // sequence's parts.
  struct Costs {
    int tiles, parts;
    uint32_t last_tile, full, head;                  // (full: a full part; head: all of a KV head)
  };
  SV_BOTH uint32_t tile_cost(int columns) const { return P.weighted ? 3u + 2u * columns : 1u; }
  SV_BOTH uint32_t head_cost() const { return P.weighted ? 6 * kHead : kHead; }
  SV_BOTH Costs costs_of(int block_rows, int keys) const {
    Costs c;
    c.tiles = tiles_of(keys);
    c.parts = parts_of(block_rows);
    c.last_tile = tile_cost((block_rows * P.g + 7) / 8 - (c.parts - 1) * NB);
    c.full = head_cost() + c.tiles * tile_cost(NB);
    c.head = (c.parts - 1) * c.full + head_cost() + c.tiles * c.last_tile;
    return c;
  }
  // All of a sequence that has rows.
  SV_BOTH Amount amount_of(int block_rows, int keys, int heads) const {
    return Amount{(tiles_of(keys) + kHead) * parts_of(block_rows) * heads,
                  NB == 1 ? 0 : costs_of(block_rows, keys).head * heads};
  }

  // The last sequence that begins at or before x, of those that have units.
  template <typename T>
  SV_BOTH int sequence_at(const T *before, T x) const {
    int lo = 0, hi = P.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  }
  SV_BOTH Place locate(int v) const {
    Place p;
    p.i = sequence_at(start, v);
    const int each = tiles_of(rows[p.i] + len[p.i]) + kHead, rem = v - start[p.i];
    // (a quotient below 2^17: by floats it is off by one at most)
    p.unit = static_cast<int>(quick_quotient(static_cast<float>(rem), static_cast<float>(each)));
    p.at = rem - p.unit * each;
    if (p.at < 0) --p.unit, p.at += each;
    if (p.at >= each) ++p.unit, p.at -= each;
    p.tiles = each - kHead;
    return p;
  }

  // The unit that a cost falls in, and its segment.
  struct Spot {
    int unit, at, left;                              // units; of the segment before and after
    uint32_t into, rest;                             // costs of the segment before and after
  };
  SV_BOTH Spot spot_of(uint32_t x) const {
    const int i = sequence_at(cost, x);
    const Costs k = costs_of(rows[i], rows[i] + len[i]);
    Spot s;
    s.into = x - cost[i];
    const int h = quotient(s.into, k.head);
    s.into -= h * k.head;
    const int part = k.parts == 1 ? 0 : less_of(k.parts - 1, quotient(s.into, k.full));
    s.into -= part * k.full;
    const uint32_t one = part == k.parts - 1 ? k.last_tile : tile_cost(NB);
    s.rest = head_cost() + k.tiles * one - s.into;
    const uint32_t tiles = s.into - head_cost();
    s.at = s.into < head_cost() ? (P.weighted ? s.into / 6 : s.into)
                                : kHead + (one == 1 ? tiles : one == 5 ? tiles / 5 : one == 7 ? tiles / 7 : tiles / 9);
    s.left = kHead + k.tiles - s.at;
    s.unit = start[i] + (h * k.parts + part) * (kHead + k.tiles) + s.at;
    return s;
  }

  // Shares of a list of `total` units, of which a grid can take so many.
  SV_BOTH int ctas_of(int total, int grid) const { return more_of(1, less_of(grid, total / kLeast)); }

  // Where share x (0 .. ctas) begins.  Shares are equal, but for ends that come within kSnap of a
  // segment's, which are moved there (a cut there would cost the joining of two CTAs' pieces).
  SV_BOTH Cut share_from(int x, int ctas) const {
    const int total = start[P.batch];
    if constexpr (NB == 1) {
      const int each = total / ctas, v = each * x + less_of(x, total - each * ctas);
      if (v <= 0 || v >= total) return Cut{v, 0};
      const Place p = locate(v);
      const int after = kHead + p.tiles - p.at;
      return Cut{p.at <= less_of(after, kSnap) ? v - p.at : after <= kSnap ? v + after : v, 0};
    } else {
      const uint32_t sum = cost[P.batch], each = sum / ctas, more = sum - each * ctas;
      Cut c{x == 0 ? 0 : total, each * x + (static_cast<uint32_t>(x) < more ? x : more)};
      if (x > 0 && x < ctas) {
        const Spot s = spot_of(c.cost);
        c.unit = s.unit;
        if (s.at <= less_of(s.left, kSnap)) c.unit -= s.at, c.cost -= s.into;
        else if (s.left <= kSnap) c.unit += s.left, c.cost += s.rest;
      }
      return c;
    }
  }

  // Where the run of warp y (0 .. warps) of the share between two cuts begins.
  SV_BOTH int run_from(const Cut &from, const Cut &to, int y, int warps) const {
    if constexpr (NB == 1) return from.unit + share_of(to.unit - from.unit, y, warps);
    if (y == 0) return from.unit;
    if (y == warps || to.cost <= from.cost) return to.unit;
    const uint32_t at = from.cost + share_of<uint32_t>(to.cost - from.cost, y, warps);
    return less_of(to.unit, more_of(from.unit, spot_of(at).unit));
  }
};

}  // namespace

}  // namespace sv
