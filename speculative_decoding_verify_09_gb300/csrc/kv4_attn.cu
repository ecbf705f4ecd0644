// Attention of ragged block rows over a paged cache in 4 bits (sm_103a).
// Contract: spec_kv4_attn in include/spec_kv4.h.
//
// softmax(scale q K^T) V with K and V as E2M1 codes times a scale per 16 elements.
// A token takes 18 D / 16 bytes per KV head, read once for all of the block's rows
// that share the head.  What stands against those bytes is the work per byte: every
// code becomes an f16 operand (one conversion and one product per two codes, and a
// byte moved down for three of four conversions) that a matrix instruction of 8 rows
// takes once.  E2M1 times E4M3 has six significant bits, so the operands are exact and
// only q (to f16: exact from 2^-17 on, and below that where it could show), the weights
// (to f16: 2^-11, below the output's 2^-8, or 2^-32 of the row's largest) and the fp32
// sums are rounded.
//
// Split: the tiles of 32 tokens of all (sequence, KV head, part of the rows) --
// segments -- are one list, cut into equal runs, one per warp of a persistent grid
// (one CTA per SM).  A warp streams its run through a ring of its own: a slab of 16
// tokens is 18 D contiguous bytes, K and V and their scales, so a tile is one or two
// bulk copies, which run ahead across segments; no warp waits for another before its
// run is done.  A segment that lies in one run is finished by its warp.  The pieces of
// the others are left in shared memory, joined there by the CTA, and, where a segment
// passes the CTA's runs, joined in the workspace, in order, by the last warp to leave a row's
// (runs per CTA instead, its warps taking tiles in turn and meeting at every segment's
// end: 160 us against 76 at 32 ragged GQA sequences).
//
// Operands: S^T = K q^T and O^T = V^T P^T, tokens (then elements) on M, rows on N,
// so a block of 1 row costs 8 columns, not 16 or more rows.  The order of a head's
// elements in a product is free: a lane takes 16 bytes in a row of a token's K (32
// elements) and the same elements of q; of V, 8 bytes in a row of four tokens'
// elements.  The weights' running maximum is kept within 2^8 of the true one, so
// the sums are rescaled seldom; its token's weight is 2^7, which uses f16's range.
// The 5th-generation tensor path is not used: single rows gain nothing by it, since the
// conversions stay.  Blocks of more than 8 rows would: 1024 bytes of f16 operands
// written to shared memory and read per token and head are 8 clocks (half with K in tensor
// memory) beside 4.2 of conversions done once, against 17.8 that the ragged rows below take.
//
// Bounds, D = 128, 8 KV heads, device time per call: 4 sequences of 128k tokens,
// single rows, 104 us = 5.8 TB/s (0.85 of the measured copy rate), 614 instructions a
// tile of 32 tokens issued at 2.6 of 4 per clock, the ALU pipe (conversions, byte
// moves) at 0.46; 16 and 24 rows take 151 and 208 us, 67 instructions more a tile for
// each 8 rows but 12 and 8 warps, and fewer registers free to overlap in.  Blocks of
// more rows go in parts, each of which converts the tokens anew: 32 ragged sequences
// of 2 to 9 rows of 4 heads take 59 us, 5 times the time of their bytes.  Short
// lists are bound by latency: 8 sequences of 32 heads over 512 to 2048 tokens 18.6 us,
// of which 4 us pass before the first copies (bounds, places, pages: one dependent
// load after the other), 2 until the first tile is there, 7 in tiles, the rest in the
// slowest warps and the joining.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "kv4.inl"
#include "kv4_cuts.inl"
#include "ops_host.inl"

namespace sv {

namespace {

constexpr int kMaxBatch = 768;                       // (16 or 20 bytes each in shared memory)
constexpr int kMaxParts = 1024;
constexpr int kMaxCtas = 192;                        // (sizes the workspace on any host)
constexpr int kCounters = 24 * kMaxCtas;             // first in the workspace, whatever the shape
constexpr int kMaxUnits = 65536;                     // sequences times KV heads times parts
// log2 the maximum may grow before sums are rescaled (0: 61.3 us, 8: 58.6), and of the weight that the
// maximum's token has.  Weights reach 2^15, which f16 holds; down to 2^-21 of the largest they keep
// f16's 11 bits, and those below 2^-32 of it are lost (with a weight of 1 for the maximum it was 2^-25, and
// 2^18 tokens of that size 0.8 % of the output).
constexpr float kLate = 8.0f, kUp = 7.0f;
// Maxima from here on are far: the fp32 rounding of a score, which the maximum is, differs from the exact
// product of the sum and its scale by more than an exponent may be off, so that products are rounded too.
constexpr float kFarMax = 0x1p22f;

// Warps and stages of a warp's ring; NB: 8-row columns of a part.  As many warps as registers
// allow (128, 168, 255 a thread; 12 instead of 16 warps with three stages: 116 us against 105
// at 128k tokens before other steps, 8 with four: 128), and two stages each, which keep 147 KB under way; a
// third one fits only where there are 8 warps.
template <int D, int NB>
struct Shape {
  static constexpr int kWarps = NB == 1 ? 16 : NB == 2 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = (NB == 3 ? 3 : 2) * (128 / D);
  static constexpr int kRows = 8 * NB;
  static constexpr int kStride = D + 4;              // floats between a slot's rows
  static constexpr int kTileBytes = 2 * slab_bytes(D);
  static constexpr size_t kRingOne = static_cast<size_t>(kStages) * kTileBytes;
  static constexpr size_t kSlotOne = static_cast<size_t>(kRows) * kStride * 4;
  static_assert(kSlotOne <= kRingOne, "a warp's last piece goes into its ring");
  static_assert(2 * kWarps <= 32, "a lane per piece");
  static constexpr size_t kRing = kWarps * kRingOne, kSlots = kWarps * kSlotOne;
  static constexpr size_t kSums = size_t{2} * kWarps * kRows * 8;
  static constexpr size_t kFixed = kRing + kSlots + kSums;
  static constexpr size_t bytes(int batch) { return kFixed + (static_cast<size_t>(batch) * (NB == 1 ? 4 : 5) + 2) * 4; }
};

struct Kv4AttnParams {
  Kv4View cache;
  int batch, Hq, g, max_q_rows;                      // g: query heads of a KV head
  int slab_shift;                                    // log2 of a page's slabs, or -1
  int weighted;                                      // costs of tiles by their columns (NB > 1)
  uint32_t g_inverse;                                // 2^32 / g rounded up: exact quotients of rows
                                                     // below 2^32 / g; 0: g is 1
  int64_t num_rows, q_stride;
  float scale_log2;                                  // of a score, k_scale and log2 e in it
  float scale_inverse;                               // 1 / scale_log2
  uint32_t scale_bits;                               // (SCALED) the same as an fp32 in [1, 2) and the power of
  int scale_power;                                   // two that it is multiplied by
  const int32_t *cu_q, *kv_len;
  const uint16_t *q;
  uint16_t *out;
  uint32_t *dev_status;
  uint32_t *counters;                                // [CTAs, rows] of the segment that a CTA begins and passes on
  float *part_o;                                     // [2 CTAs, rows, D]
  float2 *part_ml;                                   // [2 CTAs, rows] maximum, sum
  uint32_t spin_limit;
};

__device__ __forceinline__ void bar_init(uint32_t bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// Whether a phase is over (at once), or is within the time that a wait may sleep.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{.reg .pred p;\n"
               "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
               "selp.u32 %0, 1, 0, p;}\n"
               : "=r"(done) : "r"(bar), "r"(parity) : "memory");
  return done != 0;
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{.reg .pred p;\n"
               "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
               "selp.u32 %0, 1, 0, p;}\n"
               : "=r"(done) : "r"(bar), "r"(parity) : "memory");
  return done != 0;
}
// Waits for a phase; false after `limit` polls, of which the first does not sleep.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint32_t limit) {
  bool done = bar_test(bar, parity);
  for (uint32_t n = 1; !done && n < limit; ++n) done = bar_try(bar, parity);
  return done;
}

// Rows and tokens of a sequence; nothing to do: R = 0.
struct Sequence {
  int r0, R, L, keys;
};
__device__ __forceinline__ Sequence sequence_of(const Kv4AttnParams &P, int r0, int r1, int L, uint32_t *why) {
  Sequence s{0, 0, 0, 0};
  if (r0 < 0 || r1 < r0 || r1 > P.num_rows || r1 - r0 > P.max_q_rows || L < 0) {
    *why = SV_DEV_BAD_LENGTH;
  } else if (r1 > r0) {
    if (static_cast<int64_t>(L) + (r1 - r0) > static_cast<int64_t>(P.cache.max_pages) * P.cache.page_size)
      *why = SV_DEV_CAPACITY;
    else
      s = Sequence{r0, r1 - r0, L, L + (r1 - r0)};
  }
  return s;
}

// Tokens of a slab in the order of the products' rows: neighbours of a pair of lanes
// in different halves of 128 bytes.
__device__ __forceinline__ int token_of(int x) { return x ^ ((x >> 1) & 1); }

// A piece of a segment that its warp could not finish.
struct __align__(16) Piece {
  int seg;                                           // the segment's first unit; < 0: no piece
  int ends;                                          // 1: holds the segment's first tile, 2: its last
  int tiles;                                         // of the segment
  int rows, first_row, r0, h;                        // its rows: packed rows of a block at r0, KV head
};

// SCALED: a row and head of q whose largest element is below 2^15 is multiplied by the power of two that
// brings it there, on its way into f16, and its scores' scale is divided by that.
template <int D, int NB, bool SCALED>
__global__ void __launch_bounds__(Shape<D, NB>::kThreads, 1) kv4_attn_kernel(const Kv4AttnParams P) {
  using Sh = Shape<D, NB>;
  constexpr int W = Sh::kWarps, S = Sh::kStages, NT = Sh::kThreads, ROWS = Sh::kRows;
  constexpr int SLAB = slab_bytes(D), STEPS = D / 16, WORDS = D / 32, MT = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  float2 *s_ml = reinterpret_cast<float2 *>(smem + Sh::kRing + Sh::kSlots);  // [2 W, ROWS] maximum, sum
  int32_t *s_start = reinterpret_cast<int32_t *>(smem + Sh::kFixed);         // [batch + 1] units before
  int32_t *s_r0 = s_start + P.batch + 1, *s_rows = s_r0 + P.batch;           // [batch] of sequences with
  int32_t *s_len = reinterpret_cast<int32_t *>(s_rows + P.batch);            // units: first row, rows, tokens
  uint32_t *s_cost = reinterpret_cast<uint32_t *>(s_len + P.batch);          // [batch + 1] costs before (NB > 1)
  __shared__ __align__(8) uint64_t s_bar[W * S];
  __shared__ uint8_t s_bad[W * S];
  __shared__ Piece s_piece[2 * W];
  __shared__ int s_share[kMaxCtas + 1];
  const int tid = threadIdx.x, w = tid >> 5, l = tid & 31, r = l >> 2, c = l & 3;

  if (l < S) bar_init(smem_u32(&s_bar[w * S + l]));  // (a warp's barriers and pieces are its own)
  if (l < 2) s_piece[2 * w + l].seg = -1;
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  __syncwarp();
  wait_for_previous();

  // units (tiles, and kHead for each segment) before each sequence's first
  const int heads = P.cache.heads;
  const TileList<NB, Kv4AttnParams> list{P, s_start, s_rows, s_len, s_cost};
  auto head_of = [&](int unit, int parts) {          // unit / parts, exact: unit below 2^16
    return parts == 1 ? unit : static_cast<int>(__fdividef(static_cast<float>(unit) + 0.5f, static_cast<float>(parts)));
  };
  __shared__ Amount s_scan[W];
  auto enter = [&](int i) {                          // the sequence's data; its units
    uint32_t why = 0;
    const Sequence s = sequence_of(P, P.cu_q[i], P.cu_q[i + 1], P.kv_len[i], &why);
    if (why && blockIdx.x == 0) set_status(P.dev_status, why);
    s_r0[i] = s.r0, s_rows[i] = s.R, s_len[i] = s.L;
    return s.R == 0 ? Amount{0, 0} : list.amount_of(s.R, s.keys, heads);
  };
  auto inclusive = [&](int x) {                      // sums over a warp's lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (l >= o) x += y;
    }
    return x;
  };
  if (P.batch <= 32) {                               // every warp for itself: the same values, no barrier
    const Amount n = l < P.batch ? enter(l) : Amount{0, 0};
    const int inc = inclusive(n.units);
    if (l < P.batch) s_start[l] = inc - n.units;
    if (l == 31) s_start[P.batch] = inc;
    if constexpr (NB > 1) {
      const uint32_t cost = inclusive(n.cost);
      if (l < P.batch) s_cost[l] = cost - n.cost;
      if (l == 31) s_cost[P.batch] = cost;
    }
    __syncwarp();
  } else {
    const int each = (P.batch + NT - 1) / NT, i0 = min(P.batch, tid * each), i1 = min(P.batch, i0 + each);
    Amount mine{0, 0};
    for (int i = i0; i < i1; ++i) {
      const Amount n = enter(i);
      s_start[i] = n.units;
      mine.units += n.units;
      if constexpr (NB > 1) {
        s_cost[i] = n.cost;
        mine.cost += n.cost;
      }
    }
    const int inc = inclusive(mine.units);
    const uint32_t cost = NB > 1 ? inclusive(mine.cost) : 0;
    if (l == 31) s_scan[w] = Amount{inc, cost};
    __syncthreads();
    Amount before{inc - mine.units, cost - mine.cost}, all{0, 0};
    for (int i = 0; i < W; ++i) {
      const Amount x = s_scan[i];
      if (i < w) before.units += x.units, before.cost += x.cost;
      all.units += x.units, all.cost += x.cost;
    }
    for (int i = i0; i < i1; ++i) {
      const int n = s_start[i];
      s_start[i] = before.units;
      before.units += n;
      if constexpr (NB > 1) {
        const uint32_t x = s_cost[i];
        s_cost[i] = before.cost;
        before.cost += x;
      }
    }
    if (tid == 0) {
      s_start[P.batch] = all.units;
      if constexpr (NB > 1) s_cost[P.batch] = all.cost;
    }
    __syncthreads();
  }
  const int total = s_start[P.batch];
  if (total == 0) return;
  auto data_of = [&](int i) {
    const int R = s_rows[i], L = s_len[i];
    return Sequence{s_r0[i], R, L, L + R};
  };

  // A share's units go to the warps in runs of equal length (or cost).
  const int ctas = list.ctas_of(total, static_cast<int>(gridDim.x)), b = blockIdx.x;
  if (b >= ctas) return;
  // (a warp's lanes 0 and 1 find its own share's ends, the others part of the table for later)
  const int share = min(ctas, l < 2 ? b + l : 30 * w + l - 2);
  const Cut cut = list.share_from(share, ctas);
  if (l >= 2) s_share[share] = cut.unit;
  const Cut from{__shfl_sync(0xffffffffu, cut.unit, 0), __shfl_sync(0xffffffffu, cut.cost, 0)};
  const Cut to{__shfl_sync(0xffffffffu, cut.unit, 1), __shfl_sync(0xffffffffu, cut.cost, 1)};
  int v0, v1;
  if constexpr (NB == 1) {
    v0 = list.run_from(from, to, w, W), v1 = list.run_from(from, to, w + 1, W);
  } else {                                           // (lanes 0 and 1 find the run's ends)
    const int end = list.run_from(from, to, w + (l & 1), W);
    v0 = __shfl_sync(0xffffffffu, end, 0);
    v1 = __shfl_sync(0xffffffffu, end, 1);
  }
  static_assert(30 * W > kMaxCtas, "a table entry per lane");
  auto cta_of = [&](int v) {                         // the last share that starts at or before v
    int lo = 0, hi = ctas;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_share[mid] <= v) lo = mid; else hi = mid;
    }
    return lo;
  };

  // ---- this warp's copies: a lane finds the slabs of each of the next 32 units, in two steps
  // (their pages asked for, their addresses)
  const uint8_t *from0 = nullptr, *from1 = nullptr;  // slabs of this lane's tile (nullptr: not copied)
  bool from_bad = false, any_bad = false;            // pages outside the pool; any so far
  uint32_t open = 0;                                 // of these units: tiles not yet asked for
  int looked = v0;                                   // units looked at
  int issued = 0, taken = 0;                         // tiles asked for, and used
  Place ahead{0, 0, 0, 0};                           // this lane's unit, and the sequence it is of
  Sequence ahead_s{0, 0, 0, 0};
  int32_t page0 = 0, page1 = 0;                      // pages of the tile's slabs 2 n and 2 n + 1
  uint32_t slab0 = 0;                                // the first one's place in its page
  bool second = false;
  auto look_up = [&]() {
    const int v = looked + l;
    ahead = Place{0, 0, 0, 0};
    ahead_s = Sequence{0, 0, 0, 0};
    page0 = page1 = 0;
    slab0 = 0;
    second = false;
    if (v < v1) {
      ahead = list.locate(v);
      ahead_s = data_of(ahead.i);
      if (ahead.at >= kHead) {
        const uint32_t n = 2u * static_cast<uint32_t>(ahead.at - kHead), per = P.cache.slabs;
        const uint32_t at0 = P.slab_shift >= 0 ? n >> P.slab_shift : n / per;
        slab0 = n - at0 * per;
        second = static_cast<int>(n + 1) * kSlab < ahead_s.keys;
        const int32_t *row = P.cache.table + ahead.i * P.cache.table_stride + at0;
        page0 = row[0];
        page1 = slab0 + 1 == per && second ? row[1] : page0;
      }
    }
  };
  auto look_up_done = [&]() {
    const bool real = looked + l < v1 && ahead.at >= kHead;
    from0 = from1 = nullptr;
    from_bad = false;
    if (real) {
      const int parts = list.parts_of(ahead_s.R);
      const int64_t head = head_of(ahead.unit, parts) * head_bytes(P.cache);
      const int64_t page_bytes = P.cache.heads * head_bytes(P.cache);
      if (page0 < 0 || page0 >= P.cache.num_pages || page1 < 0 || page1 >= P.cache.num_pages) {
        set_status(P.dev_status, SV_DEV_BAD_PARAM);
        from_bad = true;
      } else {
        from0 = P.cache.pages + page0 * page_bytes + head + static_cast<int64_t>(slab0) * SLAB;
        if (second)
          from1 = slab0 + 1 < static_cast<uint32_t>(P.cache.slabs) ? from0 + SLAB
                                                                   : P.cache.pages + page1 * page_bytes + head;
      }
    }
    open = __ballot_sync(0xffffffffu, real);
    any_bad |= __any_sync(0xffffffffu, from_bad);
    looked += 32;
  };
  uint8_t *ring = smem + w * Sh::kRingOne;
  auto issue_open = [&]() {
    const int st = issued % S;
    if (l == __ffs(open) - 1) {
      const uint32_t bar = smem_u32(&s_bar[w * S + st]), to = smem_u32(ring + st * Sh::kTileBytes);
      s_bad[w * S + st] = from_bad;
      bar_expect(bar, (from0 != nullptr ? SLAB : 0) + (from1 != nullptr ? SLAB : 0));
      if (from0 != nullptr && from1 == from0 + SLAB) {
        bulk_copy(to, from0, 2 * SLAB, bar);
      } else {
        if (from0 != nullptr) bulk_copy(to, from0, SLAB, bar);
        if (from1 != nullptr) bulk_copy(to + SLAB, from1, SLAB, bar);
      }
    }
    open &= open - 1;
    ++issued;
  };
  auto issue = [&]() {
    while (open == 0) {
      if (looked >= v1) return;
      look_up();
      look_up_done();
    }
    issue_open();
  };
  // the segment of list entry v, and this lane's part of its rows of q
  struct Segment { Place p; Sequence s; int h, part, rows; };
  auto complete = [&](Segment &x) {
    const int parts = list.parts_of(x.s.R);
    x.h = head_of(x.p.unit, parts);
    x.part = x.p.unit - x.h * parts;
    x.rows = min(ROWS, x.s.R * P.g - x.part * ROWS);
  };
  auto token_row = [&](int row) {                    // of the block, of packed row `row`
    return P.g_inverse ? static_cast<int>(__umulhi(static_cast<uint32_t>(row), P.g_inverse)) : row;
  };
  auto q_row = [&](const Segment &x, int n) {
    const int row = x.part * ROWS + n, j = token_row(row), hh = row - j * P.g;
    return P.q + (x.s.r0 + j) * P.q_stride + static_cast<int64_t>(x.h * P.g + hh) * D + c * (D / 4);
  };
  uint4 q[NB][WORDS];
  auto fetch_q = [&](const Segment &x) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const uint4 *src = reinterpret_cast<const uint4 *>(q_row(x, 8 * nb + r));
#pragma unroll
      for (int y = 0; y < WORDS; ++y) q[nb][y] = 8 * nb + r < x.rows ? src[y] : make_uint4(0, 0, 0, 0);
    }
  };
  bool dead = false;                                 // a wait ran out: nothing more is asked for

  for (int v = v0; v < v1;) {
    // ---- a segment's tiles in this run
    Segment here;
    if (v == v0) {                                   // the first unit is lane 0's; q before the copies
      look_up();
      here.p = Place{__shfl_sync(0xffffffffu, ahead.i, 0), __shfl_sync(0xffffffffu, ahead.unit, 0),
                     __shfl_sync(0xffffffffu, ahead.at, 0), __shfl_sync(0xffffffffu, ahead.tiles, 0)};
      here.s = Sequence{__shfl_sync(0xffffffffu, ahead_s.r0, 0), __shfl_sync(0xffffffffu, ahead_s.R, 0),
                        __shfl_sync(0xffffffffu, ahead_s.L, 0), __shfl_sync(0xffffffffu, ahead_s.keys, 0)};
      complete(here);
      fetch_q(here);
      look_up_done();
      static_assert(32 / (kHead + 1) >= S, "32 units hold the first stages' tiles");
#pragma unroll 1
      for (int x = 0; x < S && open != 0; ++x) issue_open();
    } else {
      here.p = list.locate(v);
      here.s = data_of(here.p.i);
      complete(here);
      fetch_q(here);
    }
    const Place p = here.p;
    const Sequence s = here.s;
    const int h = here.h, rows = here.rows, first_row = here.part * ROWS;   // of the block's R * g rows
    const int seg = v - p.at, end = min(v1, seg + kHead + p.tiles);
    const int tile0 = max(0, p.at - kHead), tile1 = end - seg - kHead;
    const bool starts = p.at <= kHead, stops = end == seg + kHead + p.tiles;
    v = end;
    if (tile1 <= tile0) continue;

    // (SCALED) [ROWS] the scale of each column's scores; the place is the run's last piece's later
    float *s_scale = reinterpret_cast<float *>(s_ml + (2 * w + 1) * ROWS);
    if constexpr (SCALED) {
      __syncwarp();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        uint32_t top = 0;                              // the row's largest element, without its sign
#pragma unroll
        for (int x = 0; x < WORDS; ++x)
          for (const uint32_t two : {q[nb][x].x, q[nb][x].y, q[nb][x].z, q[nb][x].w})
            top = __vmaxu2(top, two & 0x7FFF7FFFu);
        top = max(top & 0xFFFFu, top >> 16);
        for (int d = 1; d < 4; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int power = min(126, max(0, 142 - static_cast<int>(top >> 7)));    // (infinities and NaN: 0)
        const uint32_t f = (127 + power) * 0x800080u;
#pragma unroll
        for (int x = 0; x < WORDS; ++x)
          for (uint32_t *two : {&q[nb][x].x, &q[nb][x].y, &q[nb][x].z, &q[nb][x].w}) *two = mul_bf16x2(*two, f);
        // (a normal number: 0 or infinity times a masked score of -inf or a score of 0 were NaN)
        if (c == 0)
          s_scale[8 * nb + r] = __uint_as_float(
              P.scale_bits + (static_cast<uint32_t>(min(max(P.scale_power - power, -126), 126)) << 23));
      }
      __syncwarp();
    }
    uint32_t qf[NB][STEPS][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int x = 0; x < WORDS; ++x) {
        qf[nb][2 * x][0] = bf16x2_to_f16x2(q[nb][x].x);
        qf[nb][2 * x][1] = bf16x2_to_f16x2(q[nb][x].y);
        qf[nb][2 * x + 1][0] = bf16x2_to_f16x2(q[nb][x].z);
        qf[nb][2 * x + 1][1] = bf16x2_to_f16x2(q[nb][x].w);
      }
    int lim[NB][2];                                  // the last token that this lane's columns see
    float m[NB][2], mu[NB][2], sum[NB][2], o[MT][NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        lim[nb][x] = s.L + min(token_row(first_row + 8 * nb + 2 * c + x), s.R - 1);
        m[nb][x] = -INFINITY;
        mu[nb][x] = sum[nb][x] = 0.0f;
      }
#pragma unroll
      for (int x = 0; x < MT; ++x) o[x][nb][0] = o[x][nb][1] = o[x][nb][2] = o[x][nb][3] = 0.0f;
    }
    bool far = false;                                // a maximum is
    int nan_from = 0x7fffffff;                       // block token whose V has NaN in this lane's elements
    // (columns that have no rows are not computed)
    auto run_tiles = [&](auto columns) {
      constexpr int NC = decltype(columns)::value;
      for (int tile = tile0; tile < tile1; ++tile, ++taken) {
        const int st = taken % S;
        if (!dead &&
            !__all_sync(0xffffffffu, bar_wait(smem_u32(&s_bar[w * S + st]), (taken / S) & 1, P.spin_limit))) {
          dead = true;
          if (l == 0) set_status(P.dev_status, SV_DEV_TIMEOUT);
          for (int x = taken; x < issued; ++x)         // copies in flight write this CTA's memory
            bar_wait(smem_u32(&s_bar[w * S + x % S]), (x / S) & 1, 1u << 22);
        }
        if (dead || (any_bad && s_bad[w * S + st])) {
#pragma unroll
          for (int nb = 0; nb < NC; ++nb) sum[nb][0] = sum[nb][1] = NAN;
          __syncwarp();
          if (!dead) issue();
          continue;
        }
        const uint8_t *stage = ring + st * Sh::kTileBytes;
        const int key0 = tile * kTile;
        const bool edge = key0 + kTile - 1 > s.L;      // tokens that some row does not see
        if (edge) {
          // Tokens behind the last hold anything: V's scales there become 0.  So do a block token's
          // that are NaN, to keep them from the rows before it (a weight of 0 would not do that);
          // the rows that see it get their NaN at the end.  A lane takes a token.
          const int key = key0 + l;
          uint8_t *scales = ring + st * Sh::kTileBytes + (l >> 4) * SLAB + slab_v(D) + 8 * D + (l & 15) * (D / 16);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const bool nan = key > s.L && key < s.keys && (scales[x] & 0x7Fu) == 0x7Fu;
            if (nan || key >= s.keys) scales[x] = 0;
            const uint32_t who = __ballot_sync(0xffffffffu, nan);
            if (who != 0 && x == (D == 128 ? r : r >> 1)) nan_from = min(nan_from, key0 + __ffs(who) - 1);
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
        }

        // ---- S^T = K q^T
        float sc[2][NC][4];
#pragma unroll
        for (int sl = 0; sl < 2; ++sl) {
#pragma unroll
          for (int nb = 0; nb < NC; ++nb) sc[sl][nb][0] = sc[sl][nb][1] = sc[sl][nb][2] = sc[sl][nb][3] = 0.0f;
          const uint8_t *slab = stage + sl * SLAB;
          const int ka = token_of(r), kb = ka + 8;
          uint32_t wa[WORDS], wb[WORDS], fa[2], fb[2]; // codes of two tokens; scales, twice each
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4 *>(slab + ka * 64 + c * 16);
            const uint4 y = *reinterpret_cast<const uint4 *>(slab + kb * 64 + c * 16);
            wa[0] = x.x, wa[1] = x.y, wa[2] = x.z, wa[3] = x.w;
            wb[0] = y.x, wb[1] = y.y, wb[2] = y.z, wb[3] = y.w;
            const uint32_t sa = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(slab + slab_k_scales(D) + ka * 8 + c * 2));
            const uint32_t sb = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(slab + slab_k_scales(D) + kb * 8 + c * 2));
            fa[0] = __byte_perm(sa, sa, 0x1010), fa[1] = __byte_perm(sa, sa, 0x3232);
            fb[0] = __byte_perm(sb, sb, 0x1010), fb[1] = __byte_perm(sb, sb, 0x3232);
          } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(slab + ka * 32 + c * 8);
            const uint2 y = *reinterpret_cast<const uint2 *>(slab + kb * 32 + c * 8);
            wa[0] = x.x, wa[1] = x.y;
            wb[0] = y.x, wb[1] = y.y;
            const uint32_t sa = slab[slab_k_scales(D) + ka * 4 + c], sb = slab[slab_k_scales(D) + kb * 4 + c];
            fa[0] = fa[1] = e4m3x2_to_f16x2(sa | sa << 8);
            fb[0] = fb[1] = e4m3x2_to_f16x2(sb | sb << 8);
          }
#pragma unroll
          for (int x = 0; x < WORDS; ++x) {
            uint32_t ha[4], hb[4];
            e2m1x8_to_f16x2(wa[x], ha);
            e2m1x8_to_f16x2(wb[x], hb);
            const uint32_t pa = fa[2 * x / WORDS], pb = fb[2 * x / WORDS];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t a[4] = {mul_f16x2(ha[2 * y], pa), mul_f16x2(hb[2 * y], pb),
                                     mul_f16x2(ha[2 * y + 1], pa), mul_f16x2(hb[2 * y + 1], pb)};
#pragma unroll
              for (int nb = 0; nb < NC; ++nb)
                mma_f16(sc[sl][nb], a, qf[nb][2 * x + y][0], qf[nb][2 * x + y][1]);
            }
          }
        }

        // ---- weights
        float scale[NC][2];                            // of this lane's columns
#pragma unroll
        for (int nb = 0; nb < NC; ++nb) {
          scale[nb][0] = scale[nb][1] = P.scale_log2;
          if constexpr (SCALED) {
            const float2 two = *reinterpret_cast<const float2 *>(s_scale + 8 * nb + 2 * c);
            scale[nb][0] = two.x, scale[nb][1] = two.y;
          }
        }
        if (edge) {
#pragma unroll
          for (int sl = 0; sl < 2; ++sl) {
            const int key = key0 + sl * kSlab + token_of(r);
#pragma unroll
            for (int nb = 0; nb < NC; ++nb)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (key + (x >> 1) * 8 > lim[nb][x & 1]) sc[sl][nb][x] = -INFINITY;
          }
        }
        bool grows = far;
#pragma unroll
        for (int nb = 0; nb < NC; ++nb)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            grows |= fmaxf(fmaxf(sc[0][nb][x], sc[0][nb][2 + x]), fmaxf(sc[1][nb][x], sc[1][nb][2 + x])) *
                         scale[nb][x] > m[nb][x] + kLate;
        if (__any_sync(0xffffffffu, grows)) {
          far = false;
#pragma unroll
          for (int nb = 0; nb < NC; ++nb)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float top = fmaxf(fmaxf(sc[0][nb][x], sc[0][nb][2 + x]), fmaxf(sc[1][nb][x], sc[1][nb][2 + x]));
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
              const float now = fmaxf(m[nb][x], top * scale[nb][x]);
              const float f = now == -INFINITY ? 1.0f : fast_exp2(m[nb][x] - now);
              m[nb][x] = now;
              mu[nb][x] = now == -INFINITY ? 0.0f : now - kUp;
              far |= fabsf(mu[nb][x]) >= kFarMax;
              sum[nb][x] *= f;
#pragma unroll
              for (int y = 0; y < MT; ++y) {
                o[y][nb][x] *= f;
                o[y][nb][2 + x] *= f;
              }
            }
          far = __any_sync(0xffffffffu, far);
          if (far) {                                   // scores less their maximum, which is 0 then
#pragma unroll
            for (int nb = 0; nb < NC; ++nb)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float top = m[nb][x] == -INFINITY ? 0.0f : m[nb][x];
                const float inverse = SCALED ? 1.0f / scale[nb][x] : P.scale_inverse;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  float &s = sc[y >> 1][nb][2 * (y & 1) + x];
                  s = __fmul_rn(__fsub_rn(__fmul_rn(s, scale[nb][x]), top), inverse);
                }
                mu[nb][x] = -kUp;
              }
          }
        }
        uint32_t pf[2][NC][2];
#pragma unroll
        for (int sl = 0; sl < 2; ++sl)
#pragma unroll
          for (int nb = 0; nb < NC; ++nb) {
            float e[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              e[x] = fast_exp2(fmaf(sc[sl][nb][x], scale[nb][x & 1], -mu[nb][x & 1]));
              sum[nb][x & 1] += e[x];
            }
            pf[sl][nb][0] = movmatrix_trans(pack_f16x2(e[0], e[1]));
            pf[sl][nb][1] = movmatrix_trans(pack_f16x2(e[2], e[3]));
          }

        // ---- O^T += V^T P^T
#pragma unroll
        for (int sl = 0; sl < 2; ++sl) {
          const uint8_t *slab = stage + sl * SLAB + slab_v(D);
          uint32_t v[4][D / 64], s4[4];                // four tokens' codes and scales
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int tok = token_of(2 * c + (x & 1)) + (x >> 1) * 8;
            if constexpr (D == 128) {
              const uint2 y = *reinterpret_cast<const uint2 *>(slab + tok * 64 + r * 8);
              v[x][0] = y.x, v[x][1] = y.y;
              s4[x] = slab[8 * D + tok * 8 + r];
            } else {
              v[x][0] = *reinterpret_cast<const uint32_t *>(slab + tok * 32 + r * 4);
              s4[x] = slab[8 * D + tok * 4 + (r >> 1)];
            }
          }
          const uint32_t f01 = e4m3x2_to_f16x2(s4[0] | s4[1] << 8), f23 = e4m3x2_to_f16x2(s4[2] | s4[3] << 8);
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            constexpr uint32_t kLow = 0x0F0F0F0Fu;
            uint32_t a0[4], a1[4], a2[4], a3[4];       // even elements of two tokens, odd ones
            e2m1x8_to_f16x2((v[0][x] & kLow) | (v[1][x] << 4 & ~kLow), a0);
            e2m1x8_to_f16x2((v[0][x] >> 4 & kLow) | (v[1][x] & ~kLow), a1);
            e2m1x8_to_f16x2((v[2][x] & kLow) | (v[3][x] << 4 & ~kLow), a2);
            e2m1x8_to_f16x2((v[2][x] >> 4 & kLow) | (v[3][x] & ~kLow), a3);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t a[4] = {mul_f16x2(a0[y], f01), mul_f16x2(a1[y], f01), mul_f16x2(a2[y], f23),
                                     mul_f16x2(a3[y], f23)};
#pragma unroll
              for (int nb = 0; nb < NC; ++nb) mma_f16(o[4 * x + y][nb], a, pf[sl][nb][0], pf[sl][nb][1]);
            }
          }
        }
        __syncwarp();
        issue();
      }
    };
    const int columns = (rows + 7) / 8;
    if (NB >= 2 && columns == 1)
      run_tiles(std::integral_constant<int, 1>());
    else if (NB >= 3 && columns == 2)
      run_tiles(std::integral_constant<int, 2>());
    else
      run_tiles(std::integral_constant<int, NB>());

    // ---- its sums: rows that this warp has seen whole are done, others a piece
    if (__any_sync(0xffffffffu, nan_from != 0x7fffffff)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int y = 0; y < MT; ++y)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (lim[nb][x & 1] >= nan_from) o[y][nb][x] = NAN;
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum[nb][x] += __shfl_xor_sync(0xffffffffu, sum[nb][x], d);
    if (starts && stops) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int n = 8 * nb + 2 * c + x;
          if (n >= rows) continue;
          const int j = token_row(first_row + n), hh = first_row + n - j * P.g;
          const float f = P.cache.v_scale / sum[nb][x];
          uint32_t pair[MT];
#pragma unroll
          for (int y = 0; y < MT; ++y) pair[y] = pack_bf16x2(o[y][nb][x] * f, o[y][nb][2 + x] * f);
          uint4 *to = reinterpret_cast<uint4 *>(
              P.out + (static_cast<int64_t>(s.r0 + j) * P.Hq + h * P.g + hh) * D + r * (D / 8));
#pragma unroll
          for (int y = 0; y < MT; y += 4) to[y / 4] = make_uint4(pair[y], pair[y + 1], pair[y + 2], pair[y + 3]);
        }
      continue;
    }
    // (the last piece of a run goes where its ring was)
    const int e = 2 * w + (end == v1 ? 1 : 0);
    float *slot = reinterpret_cast<float *>(end == v1 ? ring : smem + Sh::kRing + w * Sh::kSlotOne);
    __syncwarp();
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int n = 8 * nb + 2 * c + x;
        if (n >= rows) continue;
        if (r == 0) s_ml[e * ROWS + n] = make_float2(m[nb][x], sum[nb][x]);
        float4 *to = reinterpret_cast<float4 *>(slot + n * Sh::kStride + r * (D / 8));
#pragma unroll
        for (int y = 0; y < MT; y += 2)
          to[y / 2] = make_float4(o[y][nb][x], o[y][nb][2 + x], o[y + 1][nb][x], o[y + 1][nb][2 + x]);
      }
    if (l == 0)
      s_piece[e] = Piece{seg, (starts ? 1 : 0) | (stops ? 2 : 0), p.tiles, rows, first_row, s.r0, h};
  }

  // ---- the pieces joined: those of a segment are neighbours in the list of 2 W
  __syncthreads();
  const int my_seg = l < 2 * W ? s_piece[l].seg : -1;
  const uint32_t there = __ballot_sync(0xffffffffu, my_seg >= 0);
  if (there == 0) return;
  const uint32_t below = there & ((1u << l) - 1);
  const int prev_seg = __shfl_sync(0xffffffffu, my_seg, below ? 31 - __clz(below) : l);
  uint32_t leaders = __ballot_sync(0xffffffffu, my_seg >= 0 && (below == 0 || prev_seg != my_seg));
  constexpr int E = D / 32;                          // elements of a lane
  auto store_row = [&](const Piece &of, int n, const float (&x)[E], float total_sum) {
    const int row = of.first_row + n, j = token_row(row), hh = row - j * P.g;
    const float f = P.cache.v_scale / total_sum;
    uint32_t *to = reinterpret_cast<uint32_t *>(
        P.out + (static_cast<int64_t>(of.r0 + j) * P.Hq + of.h * P.g + hh) * D + E * l);
    if constexpr (E == 4)
      *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f));
    else
      *to = pack_bf16x2(x[0] * f, x[1] * f);
  };
  auto add = [&](float (&x)[E], float f, const float *from) {        // E neighbouring floats
    if constexpr (E == 4) {
      const float4 y = *reinterpret_cast<const float4 *>(from);
      x[0] = fmaf(f, y.x, x[0]), x[1] = fmaf(f, y.y, x[1]), x[2] = fmaf(f, y.z, x[2]), x[3] = fmaf(f, y.w, x[3]);
    } else {
      const float2 y = *reinterpret_cast<const float2 *>(from);
      x[0] = fmaf(f, y.x, x[0]), x[1] = fmaf(f, y.y, x[1]);
    }
  };
  int jobs = 0, passing = 0;                         // rows handed out; segments that pass this CTA
  int open0 = 0, open1 = 0;                          // (their first pieces)
  int left = 0, left_which = 0, left_row = 0;        // rows left in the workspace by this warp; lane n has the n-th
  while (leaders) {
    const int lead = __ffs(leaders) - 1;
    leaders &= leaders - 1;
    const uint32_t group = there & ~((1u << lead) - 1) & (leaders ? (1u << (__ffs(leaders) - 1)) - 1 : ~0u);
    const Piece head = s_piece[lead];
    const bool whole = (head.ends & 1) && (s_piece[31 - __clz(group)].ends & 2);
    const int slot = 2 * b + (head.ends & 1);
    for (int n = (w + W - jobs % W) % W; n < head.rows; n += W) {
      const bool on = group >> l & 1;
      const float2 ml = on ? s_ml[l * ROWS + n] : make_float2(-INFINITY, 0.0f);
      const float top = warp_max(ml.x), base = top == -INFINITY ? 0.0f : top;
      const float f = fast_exp2(ml.x - base), all = warp_sum(f * ml.y);
      float x[E] = {};
      for (uint32_t rest = group; rest; rest &= rest - 1) {
        const int e = __ffs(rest) - 1;
        const float *from = reinterpret_cast<const float *>(
            e & 1 ? smem + (e >> 1) * Sh::kRingOne : smem + Sh::kRing + (e >> 1) * Sh::kSlotOne);
        add(x, __shfl_sync(0xffffffffu, f, e), from + n * Sh::kStride + E * l);
      }
      if (whole) {
        store_row(head, n, x, all);
      } else {
        float *to = P.part_o + (static_cast<int64_t>(slot) * ROWS + n) * D + E * l;
#pragma unroll
        for (int y = 0; y < E; y += 2) *reinterpret_cast<float2 *>(to + y) = make_float2(x[y], x[y + 1]);
        if (l == 0) P.part_ml[slot * ROWS + n] = make_float2(top, all);
        if (l == left) left_which = passing, left_row = n;
        ++left;
      }
    }
    jobs += head.rows;
    if (!whole) {
      if (passing == 0) open0 = lead; else open1 = lead;         // (the first and the last one)
      ++passing;
    }
  }
  if (passing == 0) return;

  // ---- segments of several CTAs.  Each is known by the CTA that its first tile is in, and goes no
  // further back than that.  A row's pieces are joined, in order, by the last warp to leave one,
  // a lane per piece for the weights.
  const Piece &lane_piece = s_piece[(l & 1) == 0 ? open0 : open1];
  const int lane_cta = cta_of(lane_piece.seg + kHead + (l & 2 ? lane_piece.tiles - 1 : 0));
  const int from_a = __shfl_sync(0xffffffffu, lane_cta, 0), from_b = __shfl_sync(0xffffffffu, lane_cta, 1);
  const int pass_a = __shfl_sync(0xffffffffu, lane_cta, 2) - from_a,         // CTAs after the first
            pass_b = __shfl_sync(0xffffffffu, lane_cta, 3) - from_b;
  struct __align__(8) Some { float x[E]; };
  auto place_of = [&](int c0, int x, int n) { return static_cast<int64_t>(2 * (c0 + x) + (x == 0 ? 1 : 0)) * ROWS + n; };
  auto part = [&](int c0, int x, int n) {
    const float *from = P.part_o + place_of(c0, x, n) * D + E * l;
    Some v;
#pragma unroll
    for (int z = 0; z < E; z += 2) {
      const float2 two = __ldcg(reinterpret_cast<const float2 *>(from + z));
      v.x[z] = two.x, v.x[z + 1] = two.y;
    }
    return v;
  };
  __threadfence();                                   // (each lane's writes, before the warp's counts)
  __syncwarp();
  bool last = false;
  if (l < left) {
    const uint32_t others = left_which ? pass_b : pass_a;
    last = atomicInc(P.counters + (left_which ? from_b : from_a) * ROWS + left_row, others) == others;
    __threadfence();
  }
  __syncwarp();
  for (uint32_t todo = __ballot_sync(0xffffffffu, last); todo; todo &= todo - 1) {
    const int who = __ffs(todo) - 1, which = __shfl_sync(0xffffffffu, left_which, who),
              n = __shfl_sync(0xffffffffu, left_row, who);
    const int c0 = which ? from_b : from_a, count = (which ? pass_b : pass_a) + 1;
    constexpr int kFirst = 3;                        // sums under way together with the weights
    auto weight = [&](int y) {                       // maximum and sum of piece y + lane
      return y + l < count ? __ldcg(&P.part_ml[place_of(c0, y + l, n)]) : make_float2(-INFINITY, 0.0f);
    };
    float2 ml = weight(0);
    Some v[kFirst];
#pragma unroll
    for (int y = 0; y < kFirst; ++y)
      if (y < count) v[y] = part(c0, y, n);
    float top = ml.x;
    for (int y = 32; y < count; y += 32) top = fmaxf(top, weight(y).x);
    top = warp_max(top);
    const float base = top == -INFINITY ? 0.0f : top;
    float f = fast_exp2(ml.x - base), all = f * ml.y;
    float x[E] = {};
#pragma unroll
    for (int y = 0; y < kFirst; ++y)
      if (y < count) add(x, __shfl_sync(0xffffffffu, f, y), v[y].x);
    for (int y0 = 0; y0 < count; y0 += 32) {
      if (y0 > 0) {
        ml = weight(y0);
        f = fast_exp2(ml.x - base);
        all = fmaf(f, ml.y, all);
      }
#pragma unroll 8
      for (int y = y0 == 0 ? kFirst : 0; y < min(32, count - y0); ++y)
        add(x, __shfl_sync(0xffffffffu, f, y), part(c0, y0 + y, n).x);
    }
    store_row(s_piece[which ? open1 : open0], n, x, warp_sum(all));
  }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Columns of 8 rows that a part has (1 to 3), and parts of the largest block.
struct Plan {
  int nb, parts;
  size_t part_o, part_ml, bytes;                     // offsets in the workspace, and its size
};
Plan plan_of(const sv_kv4_attn_args &a) {
  Plan p;
  const int rows = a.max_q_rows * (a.num_q_heads / a.cache.num_kv_heads), blocks = (rows + 7) / 8;
  // Two columns a part, or three in one: a third costs a third of the warps (128k tokens of 8
  // heads: 16 rows 151 us, 24 rows 208 us, but 36 rows or fewer, ragged, 59 us in parts of two
  // and 73 us in parts of three).
  p.parts = blocks <= 3 ? 1 : (blocks + 1) / 2;
  p.nb = (blocks + p.parts - 1) / p.parts;
  p.parts = (blocks + p.nb - 1) / p.nb;
  p.part_o = kCounters * sizeof(uint32_t);
  p.part_ml = p.part_o + align256(size_t{2} * kMaxCtas * 8 * p.nb * a.cache.head_dim * sizeof(float));
  p.bytes = p.part_ml + align256(size_t{2} * kMaxCtas * 8 * p.nb * sizeof(float2));
  return p;
}

template <int D, int NB, bool SCALED>
cudaError_t launch_shape(const Kv4AttnParams &P, int ctas, cudaStream_t s) {
  using Sh = Shape<D, NB>;
  static SharedLimit limit(Sh::bytes(kMaxBatch));
  return launch_after_previous(kv4_attn_kernel<D, NB, SCALED>, limit, dim3(ctas), Sh::kThreads, Sh::bytes(P.batch),
                               s, P);
}
template <int D, bool SCALED>
cudaError_t launch_rows(int nb, const Kv4AttnParams &P, int ctas, cudaStream_t s) {
  return nb == 1   ? launch_shape<D, 1, SCALED>(P, ctas, s)
         : nb == 2 ? launch_shape<D, 2, SCALED>(P, ctas, s)
                   : launch_shape<D, 3, SCALED>(P, ctas, s);
}

sv_status check_attn4(const sv_kv4_attn_args *a, bool tensors) {
  const char *who = "kv4_attn";
  if (!a) return record_error(SV_ERR_INVALID, "%s: null arguments", who);
  sv_kv4_cache cache = a->cache;
  alignas(16) static unsigned char none[16];
  static const int32_t no_table[1] = {0};
  if (!tensors) cache.pages = none, cache.table = no_table;
  const sv_status st = check_cache(&cache, who);
  if (st != SV_OK) return st;
  if (a->batch < 0 || a->batch > kMaxBatch)
    return record_error(SV_ERR_UNSUPPORTED, "%s: batch %d outside [0, %d]", who, a->batch, kMaxBatch);
  const int Hkv = cache.num_kv_heads;
  if (a->num_q_heads < Hkv || a->num_q_heads % Hkv || a->num_q_heads / Hkv > 256)
    return record_error(SV_ERR_INVALID, "%s: heads Hq=%d Hkv=%d (need Hq %% Hkv == 0, Hq / Hkv <= 256)",
                        who, a->num_q_heads, Hkv);
  if (a->dtype != SV_BF16) return record_error(SV_ERR_UNSUPPORTED, "%s: dtype %d (built: bf16)", who, a->dtype);
  if (a->reserved != 0) return record_error(SV_ERR_INVALID, "%s: reserved must be 0", who);
  if (a->max_q_rows < 1 || a->max_q_rows > 1024)
    return record_error(SV_ERR_INVALID, "%s: max_q_rows %d outside [1, 1024]", who, a->max_q_rows);
  if (a->num_rows < 0 || a->num_rows >= (int64_t{1} << 31))
    return record_error(SV_ERR_INVALID, "%s: num_rows %lld", who, static_cast<long long>(a->num_rows));
  if (!std::isfinite(a->scale) || a->scale < 0.0f)
    return record_error(SV_ERR_INVALID, "%s: scale must be finite and >= 0", who);
  const Plan p = plan_of(*a);
  const int64_t units = static_cast<int64_t>(a->batch) * Hkv * p.parts;
  if (p.parts > kMaxParts || units > kMaxUnits)
    return record_error(SV_ERR_UNSUPPORTED, "%s: %d sequences x %d KV heads x %d parts of rows", who,
                        a->batch, Hkv, p.parts);
  const int64_t tokens = static_cast<int64_t>(cache.max_pages) * cache.page_size;
  if (tokens >= (int64_t{1} << 31) || units * ((tokens + kTile - 1) / kTile + kHead) >= (int64_t{1} << 31))
    return record_error(SV_ERR_UNSUPPORTED, "%s: tables of %d pages of %d tokens", who, cache.max_pages,
                        cache.page_size);
  const int64_t width = static_cast<int64_t>(a->num_q_heads) * cache.head_dim;
  if (a->q_stride != 0 && (a->q_stride < width || a->q_stride % 8 || a->q_stride > (int64_t{1} << 40)))
    return record_error(SV_ERR_INVALID, "%s: q row stride %lld (a multiple of 8, at least %lld)", who,
                        static_cast<long long>(a->q_stride), static_cast<long long>(width));
  if (!tensors || a->batch == 0 || a->num_rows == 0) return SV_OK;
  if (!a->cu_q || !a->kv_len) return record_error(SV_ERR_INVALID, "%s: null cu_q or kv_len", who);
  if (!a->q || !a->out || !is_aligned16(a->q) || !is_aligned16(a->out))
    return record_error(SV_ERR_INVALID, "%s: q or out null or not 16-byte aligned", who);
  if (a->q == a->out) return record_error(SV_ERR_INVALID, "%s: out is q", who);
  return SV_OK;
}

}  // namespace

}  // namespace sv

extern "C" {

SV_API size_t sv_kv4_workspace_bytes(const sv_kv4_attn_args *a) {
  using namespace sv;
  return check_attn4(a, false) == SV_OK ? plan_of(*a).bytes : 0;
}

SV_API sv_status spec_kv4_attn(const sv_kv4_attn_args *a, void *ws, size_t ws_bytes, void *stream) {
  using namespace sv;
  const char *who = "kv4_attn";
  const sv_status st = check_attn4(a, true);
  if (st != SV_OK) return st;
  const Plan p = plan_of(*a);
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 || ws_bytes < p.bytes)
    return record_error(SV_ERR_WORKSPACE, "%s: workspace null, not 256-byte aligned or below %zu bytes", who, p.bytes);
  if (a->batch == 0 || a->num_rows == 0) return SV_OK;
  const int sms = device_sms();
  if (sms <= 0) return record_error(SV_ERR_CUDA, "%s: no current CUDA device", who);
  Kv4AttnParams P{};
  P.cache = view_of(a->cache);
  P.batch = a->batch;
  P.Hq = a->num_q_heads;
  P.g = a->num_q_heads / a->cache.num_kv_heads;
  P.slab_shift = -1;
  for (int x = 0; x <= 8; ++x)
    if (P.cache.slabs == 1 << x) P.slab_shift = x;
  P.g_inverse = P.g == 1 ? 0 : static_cast<uint32_t>(((uint64_t{1} << 32) + P.g - 1) / P.g);
  P.max_q_rows = a->max_q_rows;
  const int64_t units = static_cast<int64_t>(P.batch) * P.cache.heads * p.parts,
                tiles = (static_cast<int64_t>(P.cache.max_pages) * P.cache.page_size + kTile - 1) / kTile;
  P.weighted = units * ((3 + 2 * p.nb) * tiles + 6 * kHead) < (int64_t{1} << 32);
  P.num_rows = a->num_rows;
  P.q_stride = a->q_stride ? a->q_stride : static_cast<int64_t>(P.Hq) * a->cache.head_dim;
  const double scale = a->scale != 0.0f ? a->scale : 1.0 / std::sqrt(static_cast<double>(a->cache.head_dim));
  const double all = scale * P.cache.k_scale * 1.4426950408889634;
  // An element of q below 2^-17 is off by up to 2^-25 in f16: by D scale k_scale 2^-25 of a row's largest
  // code * scale in a score, all of them together.  From here on its row is scaled (four sequences of
  // 128k tokens 105.5 us against 104.4, ragged verify rows 60.3 against 58.9).
  const bool scaled = scale * P.cache.k_scale * a->cache.head_dim > 16.0;
  // (kept a normal number: 0 or infinity times a masked score of -inf or a score of 0 were NaN)
  P.scale_log2 = static_cast<float>(std::min(std::max(all, 0x1p-126), 0x1p127));
  P.scale_inverse = 1.0f / P.scale_log2;
  if (scaled) {
    const int power = std::ilogb(all);
    const float one = static_cast<float>(std::ldexp(all, -power));
    P.scale_power = power;                           // (one may be 2: its bits add up all the same)
    std::memcpy(&P.scale_bits, &one, sizeof one);
  }
  P.cu_q = a->cu_q;
  P.kv_len = a->kv_len;
  P.q = static_cast<const uint16_t *>(a->q);
  P.out = static_cast<uint16_t *>(a->out);
  P.dev_status = a->dev_status;
  P.counters = static_cast<uint32_t *>(ws);
  P.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + p.part_o);
  P.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(ws) + p.part_ml);
  const uint32_t limit = attention_wait_limit();
  P.spin_limit = limit ? limit : 1u << 22;
  const int ctas = std::min(sms, kMaxCtas);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->cache.head_dim == 128
                            ? scaled ? launch_rows<128, true>(p.nb, P, ctas, s) : launch_rows<128, false>(p.nb, P, ctas, s)
                        : scaled ? launch_rows<64, true>(p.nb, P, ctas, s) : launch_rows<64, false>(p.nb, P, ctas, s);
  if (e != cudaSuccess) return record_error(SV_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return SV_OK;
}

SV_API int32_t sv_kv4_version(void) { return SV_KV4_VERSION; }

SV_API size_t sv_kv4_struct_size(int32_t which) {
  switch (which) {
    case 0: return sizeof(sv_kv4_cache);
    case 1: return sizeof(sv_norm_args);
    case 2: return sizeof(sv_norm_rope_args);
    case 3: return sizeof(sv_kv4_append_args);
    case 4: return sizeof(sv_kv4_read_args);
    case 5: return sizeof(sv_kv4_attn_args);
    default: return 0;
  }
}

}  // extern "C"
