// RMS norms of q and k heads and rotary positions in one pass over ragged rows
// (sm_103a), to contiguous rows or, K and V as 4-bit codes, into a paged cache;
// and rows read back out of the pages.  Contracts: spec_norm_rope_rows,
// spec_kv4_append and spec_kv4_read in include/spec_kv4.h.
//
// A head's D elements lie with D / 16 neighbouring lanes (rounded up to a power of
// two), 16 each as 8 pairs (a, b), so that its sum of squares and the largest
// magnitude of 16 elements are a few shuffles away and nothing is read twice.  Where
// the members of a pair are a multiple of 8 apart a lane holds 8 elements and the 8
// partners of these; where they are neighbours, 8 elements of each half of the head (so
// that neighbouring lanes have neighbouring 16 bytes: 16384 rows of 48 heads 64 us, with
// 16 elements in a row 81); for other distances the partner is fetched through shared
// memory.  Arithmetic is done on two floats at a
// time.  Angles as in rope.cu: the position times the turn fraction modulo 2^64, a
// quarter turn taken off, the rest rounded once.
//
// Bounds: prompts are bound by DRAM: 32768 bf16 rows of 48 heads of 128 (q and k normed and
// rotated) 121 us, 6.6 TB/s, 0.98 of the measured copy rate; 17936 rows of 32 + 2 x 8 heads
// into pages 66 us, 0.87, with instructions next; read back as bf16 0.80 of that rate, as
// E4M3 0.58 (25 bytes moved per 16 elements: instructions and latency weigh more).
// Blocks of a few rows take 2.3 to 6.7 us: the launch and one chain of dependent loads.
#include <algorithm>
#include <cmath>

#include "kv4.inl"
#include "kv4_quotient.inl"
#include "ops_host.inl"
#include "rows.inl"

namespace sv {

namespace {

constexpr int kNT = 256;
constexpr int kPad = 20;                             // floats between lanes in the exchange

enum Output { kRows, kCodes8, kPages };              // k and v: as they came, E4M3, E2M1 in pages
// How pairs lie with a lane: a = 8 elements, b = the 8 that are half further on; a and b
// neighbours in two runs of 8 elements; 16 elements in a row, partners elsewhere.
enum Layout { kPaired, kNeighbours, kFar };

struct NormRopeParams {
  int batch, max_q_rows, Hq, Hkv, D, half;           // half: pairs that are turned
  int nq, nk, heads;                                 // q heads, k heads, all heads of a row
  int lane_shift, row_shift, pairs;                  // log2 lanes of a head, threads of a row
  int heads_per_cta;
  int by_row;
  int64_t num_rows, slots;
  int64_t q_stride, k_stride, v_stride;
  float mscale, k_scale, v_scale, k_inverse, v_inverse;
  float2 k_sixth, v_sixth;                           // 1 / (6 scale): rounded down, and the rest
  float eps, weight_offset, inverse_D;
  const float *q_weight, *k_weight;
  const uint64_t *turns;
  const int32_t *cu_q, *kv_len;
  const int64_t *positions;
  const void *q, *k, *v;
  void *q_out, *k_out, *v_out;
  Kv4View cache;
  uint32_t *dev_status;
};

// The last of the batch's sequences that begins at or before row `slot`, found by a warp
// in two loads one after the other (a binary search takes one for each bit of the batch).
__device__ __forceinline__ int search_sequence(const int32_t *cu_q, int batch, int64_t slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0, step = (batch + 31) / 32;
  while (true) {
    const int at = lo + lane * step;
    const uint32_t not_behind = __ballot_sync(0xffffffffu, at < batch && cu_q[at] <= slot);
    lo += not_behind ? (31 - __clz(not_behind)) * step : 0;
    if (step == 1) return lo;
    step = (step + 31) / 32;
  }
}

// find_row (rows.inl) for a warp whose lanes ask for the same slot.
template <typename Params>
__device__ __forceinline__ bool find_row_by_warp(const Params &P, int64_t slot, int64_t &row, int64_t &pos,
                                                 bool &bad, int &seq) {
  if (!P.by_row) return find_row(P, slot, row, pos, bad, &seq);
  bad = false;
  if (slot >= P.slots) return false;
  seq = search_sequence(P.cu_q, P.batch, slot);
  const int r0 = P.cu_q[seq], r1 = P.cu_q[seq + 1], L = P.kv_len[seq], j = static_cast<int>(slot) - r0;
  if (!good_sequence(P, seq)) {
    bad = true;
    return false;
  }
  if (j < 0 || j >= r1 - r0) return false;
  row = slot;
  pos = static_cast<int64_t>(L) + j;
  return true;
}

// Two floats in a register pair, worked on at once.
typedef unsigned long long F2;
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_get(F2 x, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Scale of 16 elements whose largest magnitude is m: the E4M3 of m / (6 factor), and unit = scale *
// factor, what a code of 1 stands for.  The quotient is m times 1 / (6 factor) in two parts, which
// rounds it to fp32 as a division would: by one part it is off by a step, and then meets a tie of
// two scales that the quotient misses, or the other way round.  (Both parts are positive, so that an
// infinite m stays infinite.)
__device__ __forceinline__ uint32_t scale_code(float m, float2 sixth, float factor, float &unit) {
  const uint32_t s = e4m3x2_of(__fmaf_rn(m, sixth.x, __fmul_rn(m, sixth.y)), 0.0f) & 0xFFu;
  unit = __fmul_rn(e4m3_to_f32(s), factor);
  return s;
}
struct One {
  typedef float T;
  static __device__ __forceinline__ float fma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
};
struct Two {
  typedef F2 T;
  static __device__ __forceinline__ F2 mul(F2 a, F2 b) { return f2_mul(a, b); }
  static __device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) { return f2_fma(a, b, c); }
};
// Codes of x / unit.  A saturated scale (or NaN) may come with quotients that overflow: these are
// divided.
__device__ __forceinline__ uint32_t codes_of(const F2 (&x)[4], float unit, uint32_t scale) {
  float y[8];
  if (scale - 1u < 0x7Du) {
    float near;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(near) : "f"(unit));
    const float inv = refined_reciprocal<One>(-unit, near, 1.0f);
    const F2 inv2 = f2(inv, inv), neg = f2(-unit, -unit);
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_get(corrected_quotient<Two>(x[i], neg, inv2), y[2 * i], y[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      f2_get(x[i], lo, hi);
      y[2 * i] = scale == 0 ? 0.0f : __fdiv_rn(lo, unit);
      y[2 * i + 1] = scale == 0 ? 0.0f : __fdiv_rn(hi, unit);
    }
  }
  return e2m1x8_of(y);
}
__device__ __forceinline__ float largest(const F2 (&x)[4]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_get(x[i], lo, hi);
    m = max_nan(fabsf(lo), fabsf(hi), m);
  }
  return m;
}

// 16 elements as they lie in memory (two runs of 8) and as pairs: a[i], b[i] hold members
// 2 i and 2 i + 1 of the runs, or (neighbours) the even and the odd elements.
template <bool NEIGHBOURS>
__device__ __forceinline__ void split(const Vec<uint16_t, 8> (&v)[2], F2 (&a)[4], F2 (&b)[4]) {
  const uint32_t x[4] = {v[0].raw.a.x, v[0].raw.a.y, v[0].raw.a.z, v[0].raw.a.w};
  const uint32_t y[4] = {v[1].raw.a.x, v[1].raw.a.y, v[1].raw.a.z, v[1].raw.a.w};
  auto low = [](uint32_t z) { return __uint_as_float(z << 16); };
  auto high = [](uint32_t z) { return __uint_as_float(z & 0xFFFF0000u); };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (NEIGHBOURS) {
      const uint32_t z0 = i < 2 ? x[2 * i] : y[2 * i - 4], z1 = i < 2 ? x[2 * i + 1] : y[2 * i - 3];
      a[i] = f2(low(z0), low(z1));
      b[i] = f2(high(z0), high(z1));
    } else {
      a[i] = f2(low(x[i]), high(x[i]));
      b[i] = f2(low(y[i]), high(y[i]));
    }
  }
}
template <bool NEIGHBOURS>
__device__ __forceinline__ void split(const Vec<float, 8> (&v)[2], F2 (&a)[4], F2 (&b)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (NEIGHBOURS) {
      const float *from = i < 2 ? v[0].e + 4 * i : v[1].e + 4 * i - 8;
      a[i] = f2(from[0], from[2]);
      b[i] = f2(from[1], from[3]);
    } else {
      a[i] = f2(v[0].e[2 * i], v[0].e[2 * i + 1]);
      b[i] = f2(v[1].e[2 * i], v[1].e[2 * i + 1]);
    }
  }
}
// The other way: runs x and y of 8 elements.
template <bool NEIGHBOURS>
__device__ __forceinline__ void runs(const F2 (&a)[4], const F2 (&b)[4], float (&x)[8], float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a0, a1, b0, b1;
    f2_get(a[i], a0, a1);
    f2_get(b[i], b0, b1);
    if constexpr (NEIGHBOURS) {
      float *to = i < 2 ? x + 4 * i : y + 4 * i - 8;
      to[0] = a0, to[1] = b0, to[2] = a1, to[3] = b1;
    } else {
      x[2 * i] = a0, x[2 * i + 1] = a1;
      y[2 * i] = b0, y[2 * i + 1] = b1;
    }
  }
}

// Back into a vector of the rows' type.
__device__ __forceinline__ void join(Vec<uint16_t, 8> &v, const float (&x)[8]) {
  v.raw.a = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void join(Vec<float, 8> &v, const float (&x)[8]) { v.set(x); }

// CTAs per SM that the registers are capped for: copies under way are what prompts need (32768 bf16
// rows of 48 heads of 128 take 123 us at 4 CTAs, 126 at 3), but with pages 4 cost local memory:
// 17936 rows 69 us against 66, 576 rows 7.0 against 6.7.
template <typename T, Output OUT, Layout LAYOUT>
constexpr int kCtas = LAYOUT == kFar || sizeof(T) == 4 ? 2 : OUT == kPages ? 3 : 4;

// A lane asks for its 16 elements of kStages - 1 heads ahead, into places of its own in shared memory
// (32768 rows of 48 heads with 3 stages 121 us, 4 123, 6 129; 17936 rows into pages 67, 66, 69; with
// one head ahead in registers, and none from one kind of heads to the next, 134 and 79).
template <typename T, Output OUT>
constexpr int kStages = OUT == kPages && sizeof(T) == 2 ? 4 : 3;
template <typename T, Output OUT>
constexpr size_t kRing = kStages<T, OUT> * sizeof(T) * kNT * 16;     // bytes
// Past L1, where neighbouring lanes take neighbouring 16 bytes; else what is left of a sector is
// found there by the next copy (16384 rows of 48 heads, past it or not: 66 and 72 us; fp32 172
// and 130).
template <bool PAST_L1>
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
  if constexpr (PAST_L1)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }

template <typename T, Output OUT, Layout LAYOUT>
__global__ void __launch_bounds__(kNT, kCtas<T, OUT, LAYOUT>) norm_rope_kernel(const NormRopeParams P) {
  constexpr bool kSide = LAYOUT == kNeighbours;
  constexpr bool kPastL1 = LAYOUT != kFar && sizeof(T) == 2;
  constexpr int S = kStages<T, OUT>, CHUNKS = static_cast<int>(sizeof(T));        // 16 bytes of a stage that a lane has
  extern __shared__ __align__(16) uint8_t s_ring[];  // [stages][chunks][threads] of 16 bytes
  float *s_swap = reinterpret_cast<float *>(s_ring + kRing<T, OUT>);                   // (kFar) the exchange
  float *s_turn = s_swap + (LAYOUT == kFar ? kNT * kPad : 0);        // [rows][cos, sin][pairs], [q, k][16 lanes] weights
  const int row_threads = 1 << P.row_shift, lanes = 1 << P.lane_shift;
  const int rl = threadIdx.x >> P.row_shift, t = threadIdx.x & (row_threads - 1);
  const int hl = t >> P.lane_shift, c = t & (lanes - 1), hstep = row_threads >> P.lane_shift;
  const int h_begin = blockIdx.y * P.heads_per_cta;
  const int h_end = min(P.heads, h_begin + P.heads_per_cta);
  wait_for_previous();

  int64_t row = 0, pos = 0;
  int seq = 0;
  bool bad;
  const bool live = find_row_by_warp(P, static_cast<int64_t>(blockIdx.x) * (kNT >> P.row_shift) + rl, row,
                                     pos, bad, seq);
  if (bad && t == 0 && blockIdx.y == 0) set_status(P.dev_status, SV_DEV_BAD_LENGTH);
  if (P.by_row && blockIdx.y == 0)                   // (a bad sequence need not be found by a row)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNT + threadIdx.x; i < P.batch;
         i += static_cast<int64_t>(gridDim.x) * kNT)
      if (!good_sequence(P, static_cast<int>(i))) set_status(P.dev_status, SV_DEV_BAD_LENGTH);

  // this lane's column: two runs of 8 elements of a head, and how many of its pairs turn
  const bool wide = kSide && P.D % 16 == 0;          // (neighbours, in runs of both halves of a head)
  auto run_of = [&](int c, int second) {
    if (LAYOUT == kPaired && 8 * c < P.half) return 8 * c + second * P.half;         // the runs are a pair's members
    if (LAYOUT == kPaired) return 2 * P.half + 16 * (c - P.half / 8) + 8 * second;
    return wide ? 8 * c + second * (P.D / 2) : 16 * c + 8 * second;
  };
  const int o0 = run_of(c, 0), o1 = run_of(c, 1);
  const bool column = live && o0 < (wide ? P.D / 2 : P.D), both = column && o1 < P.D;
  const bool apart = (LAYOUT == kPaired && 8 * c < P.half) || wide;  // runs of two times 16 elements
  auto turning_of = [&](int run) {                   // how many of 4 pairs do
    return LAYOUT == kPaired ? (8 * c < P.half ? 4 : 0) : min(4, max(0, P.half - run / 2));
  };
  const int turning[2] = {turning_of(o0), turning_of(o1)};

  Kv4Spot spot{};
  if (OUT == kPages && live) spot = find_page(P.cache, seq, pos);

  // the kinds' first heads and their tensors: q, k, v
  auto first_of = [&](int kind) { return kind == 0 ? 0 : kind == 1 ? P.nq : P.nq + P.nk; };
  auto source = [&](int kind) {
    return kind == 0   ? static_cast<const T *>(P.q) + row * P.q_stride
           : kind == 1 ? static_cast<const T *>(P.k) + row * P.k_stride
                       : static_cast<const T *>(P.v) + row * P.v_stride;
  };
  auto range = [&](int kind, int &begin, int &end) {  // heads of a kind that this CTA has
    const int k0 = first_of(kind);
    begin = max(h_begin, k0) - k0, end = min(h_end, kind == 2 ? P.heads : first_of(kind + 1)) - k0;
  };
  // This lane's elements of the next heads in order: into its own places of a stage
  int f_kind = h_begin < P.nq ? 0 : h_begin < P.nq + P.nk ? 1 : 2, f_hb, f_end;
  range(f_kind, f_hb, f_end);
  const T *f_in = source(f_kind) + (f_hb + hl) * P.D;
  auto fetch = [&](int stage) {
    if (f_hb >= f_end && first_of(f_kind) + f_end < h_end) {         // the next kind that has heads here
      do range(++f_kind, f_hb, f_end);
      while (f_hb >= f_end);
      f_in = source(f_kind) + (f_hb + hl) * P.D;
    }
    if (column && f_hb + hl < f_end) {
      const uint32_t to = smem_u32(s_ring) + (stage * CHUNKS * kNT + threadIdx.x) * 16;
#pragma unroll
      for (int x = 0; x < CHUNKS / 2; ++x) {
        copy16<kPastL1>(to + x * kNT * 16, f_in + o0 + x * 4);
        if (both) copy16<kPastL1>(to + (CHUNKS / 2 + x) * kNT * 16, f_in + o1 + x * 4);
      }
    }
    f_hb += hstep;
    f_in += hstep * P.D;
    copies_end();
  };
  fetch(0);
  int stage = 0;

  // cos and sin of the row's pairs, by the threads that share the row; the weights in the order
  // of the columns' a and b
  float *s_cos = s_turn + rl * 2 * P.pairs, *s_sin = s_cos + P.pairs;
  float *s_weight = s_turn + (kNT >> P.row_shift) * 2 * P.pairs;
  const bool any_turn = P.half > 0 && h_begin < P.nq + P.nk;
  if (live && any_turn) {
    for (int p = t; p < P.half; p += row_threads) {
      const uint64_t part = static_cast<uint64_t>(pos) * P.turns[p];
      const uint64_t quarter = (part + (uint64_t{1} << 61)) >> 62;
      const int64_t rest = static_cast<int64_t>(part - (quarter << 62));
      float sr, cr;
      sincospif(__ll2float_rn(rest) * 0x1p-63f, &sr, &cr);
      const float sn = quarter & 1 ? cr : sr, cs = quarter & 1 ? sr : cr;
      s_cos[p] = ((quarter + 1) & 2 ? -cs : cs) * P.mscale;
      s_sin[p] = (quarter & 2 ? -sn : sn) * P.mscale;
    }
  }
  const bool norms = P.q_weight != nullptr || P.k_weight != nullptr;
  if (norms) {
    for (int x = threadIdx.x; x < 32 * lanes; x += kNT) {          // [kind][a, b][lanes][8]
      const float *weight = x < 16 * lanes ? P.q_weight : P.k_weight;
      const int y = x & (16 * lanes - 1), second = y >= 8 * lanes, col = (y & (8 * lanes - 1)) >> 3, i = y & 7;
      const int at = kSide ? run_of(col, i >> 2) + 2 * (i & 3) + second : run_of(col, second) + i;
      s_weight[x] = weight != nullptr && at < P.D ? weight[at] + P.weight_offset : 1.0f;
    }
  }
  uint8_t *slab = nullptr;                           // of the row's token, KV head 0
  if (OUT == kPages && live) {
    uint32_t why = 0;
    slab = find_slab(P.cache, spot, &why);
    if (why && t == 0 && blockIdx.y == 0) set_status(P.dev_status, why);
  }
  if (f_hb < f_end || first_of(f_kind) + f_end < h_end) {            // (else there is nothing more)
#pragma unroll
    for (int x = 1; x < S - 1; ++x) fetch(x);
  } else {
#pragma unroll
    for (int x = 1; x < S - 1; ++x) copies_end();
  }
  __syncthreads();
  if (!live) return;                                 // (all threads of a warp share a row)

  // the pairs of this column (those that do not turn read others' and are not touched)
  const int p0 = kSide ? o0 / 2 : 8 * c, p1 = kSide ? o1 / 2 : 8 * c + 4;
  const bool all_turn = __all_sync(0xffffffffu, turning[0] + turning[1] == 8 || !column);
  const int token = static_cast<int>(pos) & (kSlab - 1);

  for (int kind = 0; kind < 3; ++kind) {
    int begin, end;
    range(kind, begin, end);
    if (begin >= end) continue;
    const bool is_q = kind == 0, turns = kind < 2 && any_turn;
    const bool normed = kind == 0 ? P.q_weight != nullptr : kind == 1 && P.k_weight != nullptr;
    const bool changed = turns || normed;
    const float factor = kind == 1 ? P.k_scale : P.v_scale, inverse = kind == 1 ? P.k_inverse : P.v_inverse;
    const float2 sixth = kind == 1 ? P.k_sixth : P.v_sixth;
    const float4 *w4 = reinterpret_cast<const float4 *>(s_weight + (is_q ? 0 : 16 * lanes)) + 2 * c;
    const int64_t out = is_q ? row * P.Hq * P.D : row * P.Hkv * P.D;
    T *to = static_cast<T *>(is_q ? P.q_out : kind == 1 ? P.k_out : P.v_out) + out + (begin + hl) * P.D;
    uint8_t *to8 = static_cast<uint8_t *>(kind == 1 ? P.k_out : P.v_out) + out + (begin + hl) * P.D;
    const int64_t next_head = OUT == kPages ? hstep * head_bytes(P.cache) : 0;
    uint8_t *codes = nullptr, *scales = nullptr;     // of this lane's elements from o0 on
    if (OUT == kPages && !is_q && slab != nullptr) {
      uint8_t *page = slab + (begin + hl) * head_bytes(P.cache) + (kind == 1 ? 0 : slab_v(P.D));
      codes = page + token * (P.D / 2) + o0 / 2;
      scales = page + slab_k_scales(P.D) + token * (P.D / 16) + o0 / 16;
    }
#pragma unroll 1
    for (int hb = begin; hb < end; hb += hstep) {
      const bool on = column && hb + hl < end;
      fetch((stage + S - 1) % S);
      asm volatile("cp.async.wait_group %0;\n" ::"n"(S - 1) : "memory");
      Vec<T, 8> cur[2];
      {
        const uint8_t *at = s_ring + (stage * CHUNKS * kNT + threadIdx.x) * 16;
#pragma unroll
        for (int x = 0; x < CHUNKS / 2; ++x) {
          reinterpret_cast<uint4 *>(&cur[0])[x] = *reinterpret_cast<const uint4 *>(at + x * kNT * 16);
          const uint4 second = *reinterpret_cast<const uint4 *>(at + (CHUNKS / 2 + x) * kNT * 16);
          reinterpret_cast<uint4 *>(&cur[1])[x] = both ? second : make_uint4(0, 0, 0, 0);
        }
      }
      stage = (stage + 1) % S;
      F2 a[4], b[4];
      if (changed || OUT == kCodes8 || OUT == kPages) split<kSide>(cur, a, b);
      if (normed) {
        F2 s = f2_mul(a[0], a[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s = f2_fma(a[i], a[i], s);
#pragma unroll
        for (int i = 0; i < 4; ++i) s = f2_fma(b[i], b[i], s);
        float s0, s1;
        f2_get(s, s0, s1);
        s0 = on ? s0 + s1 : 0.0f;
        for (int o = lanes >> 1; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        const float r = rsqrtf(fmaf(s0, P.inverse_D, P.eps));
        const F2 r2 = f2(r, r);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float4 wa = w4[x], wb = w4[2 * lanes + x];
          a[2 * x] = f2_mul(f2_mul(a[2 * x], r2), f2(wa.x, wa.y));
          a[2 * x + 1] = f2_mul(f2_mul(a[2 * x + 1], r2), f2(wa.z, wa.w));
          b[2 * x] = f2_mul(f2_mul(b[2 * x], r2), f2(wb.x, wb.y));
          b[2 * x + 1] = f2_mul(f2_mul(b[2 * x + 1], r2), f2(wb.z, wb.w));
        }
      }
      if (turns && LAYOUT == kFar) {                 // partners through shared memory
        float x[8], y[8];
        runs<false>(a, b, x, y);
        float *mine = s_swap + threadIdx.x * kPad, *head = s_swap + (threadIdx.x - c) * kPad;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          mine[i] = x[i];
          mine[8 + i] = y[i];
        }
        __syncwarp();
        auto turned = [&](float own, int e) {
          if (e >= 2 * P.half) return own;
          const bool first = e < P.half;
          const int p = first ? e : e - P.half, o = first ? e + P.half : p;
          const float other = head[(o >> 4) * kPad + (o & 15)];
          return first ? own * s_cos[p] - other * s_sin[p] : own * s_cos[p] + other * s_sin[p];
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = turned(x[i], o0 + i);
          y[i] = turned(y[i], o1 + i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = f2(x[2 * i], x[2 * i + 1]);
          b[i] = f2(y[2 * i], y[2 * i + 1]);
        }
      } else if (turns) {
        if (all_turn || turning[0] + turning[1] > 0) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float4 cx = *reinterpret_cast<const float4 *>(s_cos + (n ? p1 : p0));
            const float4 sx = *reinterpret_cast<const float4 *>(s_sin + (n ? p1 : p0));
            const F2 cs[2] = {f2(cx.x, cx.y), f2(cx.z, cx.w)}, sn[2] = {f2(sx.x, sx.y), f2(sx.z, sx.w)};
            const F2 minus[2] = {f2(-sx.x, -sx.y), f2(-sx.z, -sx.w)};
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const int i = 2 * n + m;
              const F2 x = f2_fma(a[i], cs[m], f2_mul(b[i], minus[m]));
              const F2 y = f2_fma(b[i], cs[m], f2_mul(a[i], sn[m]));
              if (all_turn) {
                a[i] = x;
                b[i] = y;
              } else {
                float a0, a1, b0, b1, x0, x1, y0, y1;
                f2_get(a[i], a0, a1);
                f2_get(b[i], b0, b1);
                f2_get(x, x0, x1);
                f2_get(y, y0, y1);
                const bool on0 = 2 * m < turning[n], on1 = 2 * m + 1 < turning[n];
                a[i] = f2(on0 ? x0 : a0, on1 ? x1 : a1);
                b[i] = f2(on0 ? y0 : b0, on1 ? y1 : b1);
              }
            }
          }
        }
      }
      if (OUT == kPages && !is_q) {                  // (all lanes: shuffles)
        if constexpr (kSide) {
          float x[8], y[8];
          runs<true>(a, b, x, y);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = f2(x[2 * i], x[2 * i + 1]);
            b[i] = f2(y[2 * i], y[2 * i + 1]);
          }
        }
        float m0 = largest(a), m1 = largest(b);
        const float n0 = __shfl_xor_sync(0xffffffffu, m0, 1), n1 = __shfl_xor_sync(0xffffffffu, m1, 1);
        const float all = max_nan(m0, m1);
        m0 = apart ? max_nan(m0, n0) : all;
        m1 = apart ? max_nan(m1, n1) : all;
        if (on && slab != nullptr) {
          float u0;
          const uint32_t s0 = scale_code(m0, sixth, factor, u0);
          if (apart) {
            float u1;
            const uint32_t s1 = scale_code(m1, sixth, factor, u1);
            *reinterpret_cast<uint32_t *>(codes) = codes_of(a, u0, s0);
            *reinterpret_cast<uint32_t *>(codes + (o1 - o0) / 2) = codes_of(b, u1, s1);
            if (c % 2 == 0) {                        // one lane of those that share 16 elements
              *scales = static_cast<uint8_t>(s0);
              scales[(o1 - o0) / 16] = static_cast<uint8_t>(s1);
            }
          } else {
            *reinterpret_cast<uint2 *>(codes) = make_uint2(codes_of(a, u0, s0), codes_of(b, u0, s0));
            *scales = static_cast<uint8_t>(s0);
          }
        }
        codes += next_head;
        scales += next_head;
      } else if (OUT == kCodes8 && !is_q) {
        if (on) {
          float x[8], y[8];
          runs<kSide>(a, b, x, y);
          store_codes(to8 + o0, x, factor, inverse);
          if (both) store_codes(to8 + o1, y, factor, inverse);
        }
        to8 += hstep * P.D;
      } else {
        if (on) {
          if (changed) {                             // (else the bits stay)
            float x[8], y[8];
            runs<kSide>(a, b, x, y);
            join(cur[0], x);
            join(cur[1], y);
          }
          cur[0].store(to + o0);
          if (both) cur[1].store(to + o1);
        }
        to += hstep * P.D;
      }
    }
  }
}

// ---------------------------------------------------------------- read
struct ReadParams {
  int batch, max_q_rows, D, row_shift;
  int by_row;
  int64_t num_rows, slots;
  float k_scale, v_scale, k_inverse, v_inverse;      // E4M3 outputs
  uint32_t k_short, v_short;                         // f16x2 of what a product of code and scale is to be
                                                     // multiplied by, where that may be done to the scale
                                                     // in f16 (below), else 0
  const int32_t *cu_q, *kv_len;
  const int64_t *positions;                          // nullptr
  void *k_out, *v_out;
  Kv4View cache;
  uint32_t *dev_status;
};

// A thread takes 16 bytes of a row of the output at a time (of fp32 32), 8 elements (4 bytes of
// codes, a scale that two threads share) or 16, so that a warp writes whole lines, of kReads K and
// V heads each, all asked for before the first is written (17936 rows of 8 heads as E4M3 14.8 us;
// K before V 15.6, and 8 elements at a time 16.6; kReads 4 with E4M3 20.3, but 8192 rows of 32 as
// bf16 31.9 us against 33.2 with 2).
template <typename T>
constexpr int kItem = sizeof(T) == 1 ? 16 : 8;
template <typename T>
constexpr int kReadsOf = sizeof(T) == 2 ? 4 : 2;
template <typename T>
__global__ void __launch_bounds__(kNT, sizeof(T) == 1 ? 5 : 4) kv4_read_kernel(const ReadParams P) {
  const int row_threads = 1 << P.row_shift;
  const int rl = threadIdx.x >> P.row_shift, t = threadIdx.x & (row_threads - 1);
  wait_for_previous();
  int64_t row = 0, pos = 0;
  int seq = 0;
  bool bad;
  const bool live = find_row_by_warp(P, static_cast<int64_t>(blockIdx.x) * (kNT >> P.row_shift) + rl, row,
                                     pos, bad, seq);
  if (bad && t == 0 && blockIdx.y == 0) set_status(P.dev_status, SV_DEV_BAD_LENGTH);
  if (P.by_row && blockIdx.y == 0)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNT + threadIdx.x; i < P.batch;
         i += static_cast<int64_t>(gridDim.x) * kNT)
      if (!good_sequence(P, static_cast<int>(i))) set_status(P.dev_status, SV_DEV_BAD_LENGTH);
  if (!live) return;
  uint32_t why = 0;
  const uint8_t *slab = find_slab(P.cache, find_page(P.cache, seq, pos), &why);
  if (why && t == 0 && blockIdx.y == 0) set_status(P.dev_status, why);
  if (slab == nullptr) return;
  const int token = static_cast<int>(pos) & (kSlab - 1);
  constexpr int N = kItem<T>, WORDS = N / 8, kReads = kReadsOf<T>;
  const int shift = (P.D == 128 ? 4 : 3) - (N == 16);                // log2 of the items of a head
  const int heads = P.cache.heads, g = t & ((1 << shift) - 1);
  const int each = row_threads >> shift, step = each * gridDim.y;    // heads at once: of a slice, of all
  const int64_t head = head_bytes(P.cache);
  const int scale_at = slab_k_scales(P.D) + token * (P.D / 16) + (N == 16 ? g : g >> 1), code_at = token * (P.D / 2) + N / 2 * g;
  const int h0 = blockIdx.y * each + (t >> shift);
  const uint8_t *at = slab + h0 * head;
  const int64_t to = (row * heads + h0) * P.D + N * g;
  const bool both[2] = {P.k_out != nullptr, P.v_out != nullptr};
  for (int h = h0, done = 0; h < heads; h += kReads * step, done += kReads * step) {
    uint32_t codes[2][kReads][WORDS], scale[2][kReads];
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v)
#pragma unroll
      for (int u = 0; u < kReads; ++u)
        if (both[is_v] && h + u * step < heads) {
          const uint8_t *from = at + (done + u * step) * head + (is_v ? slab_v(P.D) : 0);
          if constexpr (WORDS == 2) {
            const uint2 two = *reinterpret_cast<const uint2 *>(from + code_at);
            codes[is_v][u][0] = two.x, codes[is_v][u][1] = two.y;
          } else {
            codes[is_v][u][0] = *reinterpret_cast<const uint32_t *>(from + code_at);
          }
          scale[is_v][u] = from[scale_at];
        }
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v) {
      const float factor = is_v ? P.cache.v_scale : P.cache.k_scale;
      const float to_scale = is_v ? P.v_scale : P.k_scale, inverse = is_v ? P.v_inverse : P.k_inverse;
      const uint32_t brief = is_v ? P.v_short : P.k_short;
#pragma unroll
      for (int u = 0; u < kReads; ++u) {
        if (!both[is_v] || h + u * step >= heads) continue;
        T *out = static_cast<T *>(is_v ? P.v_out : P.k_out) + to + (done + u * step) * P.D;
        uint32_t s = e4m3x2_to_f16x2(scale[is_v][u] | scale[is_v][u] << 8);
        if (brief != 0) s = mul_f16x2(s, brief);
        uint32_t y[4 * WORDS];
#pragma unroll
        for (int n = 0; n < WORDS; ++n) {
          uint32_t pair[4];
          e2m1x8_to_f16x2(codes[is_v][u][n], pair);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[4 * n + i] = mul_f16x2(pair[i], s);    // exact
        }
        if constexpr (sizeof(T) == 1) {
          if (brief != 0) {
            uint32_t z[2 * WORDS];
#pragma unroll
            for (int i = 0; i < 2 * WORDS; ++i) z[i] = f16x2_to_e4m3x2(y[2 * i]) | f16x2_to_e4m3x2(y[2 * i + 1]) << 16;
            *reinterpret_cast<uint4 *>(out) = make_uint4(z[0], z[1], z[2], z[3]);
            continue;
          }
        }
        float x[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          x[2 * i] = f16_bits_to_f32(y[i] & 0xFFFFu);
          x[2 * i + 1] = f16_bits_to_f32(y[i] >> 16);
        }
        if (brief == 0) {
#pragma unroll
          for (int i = 0; i < N; ++i) x[i] = __fmul_rn(x[i], factor);
        }
        if constexpr (sizeof(T) == 1) {
          store_codes(out, x, to_scale, inverse);
        } else if constexpr (sizeof(T) == 4) {
          // two lanes (of one head) write one's 32 bytes, then the other's: whole sectors at a time
          // (8192 rows of 32 heads 57 us, with halves of sectors 73)
          const bool odd = threadIdx.x & 1;
          const uint32_t pair = 3u << (threadIdx.x & 30);
          float4 own = odd ? make_float4(x[4], x[5], x[6], x[7]) : make_float4(x[0], x[1], x[2], x[3]);
          float4 got = odd ? make_float4(x[0], x[1], x[2], x[3]) : make_float4(x[4], x[5], x[6], x[7]);
          got.x = __shfl_xor_sync(pair, got.x, 1);
          got.y = __shfl_xor_sync(pair, got.y, 1);
          got.z = __shfl_xor_sync(pair, got.z, 1);
          got.w = __shfl_xor_sync(pair, got.w, 1);
          *reinterpret_cast<float4 *>(out - (odd ? 4 : 0)) = odd ? got : own;
          *reinterpret_cast<float4 *>(out + (odd ? 4 : 8)) = odd ? own : got;
        } else {
          Vec<T, 8> v;
          v.set(x);
          v.store(out);
        }
      }
    }
  }
}

float exact_inverse(float x) {                       // 1 / x where x is a power of two, else 0
  int e;
  const float inv = 1.0f / x;
  return std::frexp(x, &e) == 0.5f && std::isnormal(inv) ? inv : 0.0f;
}

float2 sixth_of(float x) {                           // 1 / (6 x), x > 0, as two positive numbers
  const double all = 1.0 / (6.0 * static_cast<double>(x));
  float down = static_cast<float>(all);
  if (down >= all) down = std::nextafter(down, 0.0f);
  return make_float2(down, static_cast<float>(all - down));
}

// f16x2 of `x` if it is a power of two in [2^-5, 2^5], else 0.  A scale (2^-9 .. 448, four
// significant bits) times such an x is exact in f16, and so is that times a code: six bits
// from 2^-15 on, or beyond f16's range where E4M3 saturates all the same.
uint32_t short_factor(float x) {
  int e;
  if (std::frexp(x, &e) != 0.5f || e < -4 || e > 6) return 0;
  const uint32_t h = static_cast<uint32_t>(e - 1 + 15) << 10;
  return h | h << 16;
}

// Shared memory behind the ring: the exchange, and what all layouts have (at most: 8 rows of 132
// pairs, 16 lanes of weights).
constexpr size_t swap_bytes(Layout layout) { return layout == kFar ? kNT * kPad * sizeof(float) : 0; }
constexpr size_t turn_bytes(int rows, int pairs, int lanes) {
  return (static_cast<size_t>(rows) * 2 * pairs + 32 * lanes) * sizeof(float);
}

template <typename T, Output OUT, Layout LAYOUT>
cudaError_t launch_rows(dim3 grid, size_t turns, cudaStream_t s, const NormRopeParams &P) {
  constexpr size_t before = kRing<T, OUT> + swap_bytes(LAYOUT);
  static SharedLimit limit(before + turn_bytes(8, 132, 16));
  return launch_after_previous(norm_rope_kernel<T, OUT, LAYOUT>, limit, grid, kNT, before + turns, s, P);
}
template <typename T, Output OUT>
cudaError_t launch_layout(Layout layout, dim3 grid, size_t turns, cudaStream_t s, const NormRopeParams &P) {
  return layout == kPaired       ? launch_rows<T, OUT, kPaired>(grid, turns, s, P)
         : layout == kNeighbours ? launch_rows<T, OUT, kNeighbours>(grid, turns, s, P)
                                 : launch_rows<T, OUT, kFar>(grid, turns, s, P);
}

sv_status check_norm(const sv_norm_args &n, const char *who) {
  if (!std::isfinite(n.eps) || n.eps < 0.0f)
    return record_error(SV_ERR_INVALID, "%s: eps must be finite and >= 0", who);
  if (!std::isfinite(n.weight_offset))
    return record_error(SV_ERR_INVALID, "%s: weight_offset must be finite", who);
  for (const float *w : {n.q_weight, n.k_weight})
    if (reinterpret_cast<uintptr_t>(w) % 4)
      return record_error(SV_ERR_INVALID, "%s: weights must be 4-byte aligned", who);
  return SV_OK;
}

// Every sequence has max_q_rows slots, as in a step, unless most would stay empty
// (prompts of different lengths): then a row searches its sequence.
template <typename Params>
void set_slots(Params &P) {
  P.slots = P.positions ? P.num_rows : static_cast<int64_t>(P.batch) * P.max_q_rows;
  P.by_row = !P.positions && P.max_q_rows > 16 && P.slots > P.num_rows + P.num_rows / 4;
  if (P.by_row) P.slots = P.num_rows;
}

sv_status run_rows(const sv_rope_args &a, const sv_norm_args &n, const sv_kv4_cache *cache,
                   const char *who, void *stream) {
  NormRopeParams P{};
  P.batch = a.batch;
  P.max_q_rows = a.max_q_rows;
  P.Hq = a.num_q_heads;
  P.Hkv = a.num_kv_heads;
  P.D = a.head_dim;
  P.half = a.turns ? a.rot_dim / 2 : 0;
  P.num_rows = a.num_rows;
  P.cu_q = a.cu_q;
  P.kv_len = a.kv_len;
  P.positions = a.positions;
  set_slots(P);
  P.q_stride = a.q_stride ? a.q_stride : static_cast<int64_t>(P.Hq) * P.D;
  P.k_stride = a.k_stride ? a.k_stride : static_cast<int64_t>(P.Hkv) * P.D;
  P.v_stride = a.v_stride ? a.v_stride : static_cast<int64_t>(P.Hkv) * P.D;
  P.mscale = a.mscale == 0.0f ? 1.0f : a.mscale;
  P.k_scale = a.k_scale == 0.0f ? 1.0f : a.k_scale;
  P.v_scale = a.v_scale == 0.0f ? 1.0f : a.v_scale;
  P.eps = n.eps;
  P.weight_offset = n.weight_offset;
  P.inverse_D = 1.0f / static_cast<float>(P.D);
  P.q_weight = n.q_weight;
  P.k_weight = n.k_weight;
  P.turns = a.turns;
  P.q = a.q;
  P.k = a.k;
  P.v = a.v;
  P.q_out = a.q_out;
  P.k_out = a.k_out;
  P.v_out = a.v_out;
  P.dev_status = a.dev_status;
  P.nq = P.Hq;
  P.nk = a.k ? P.Hkv : 0;
  P.heads = P.nq + P.nk + (a.v && a.v != a.v_out ? P.Hkv : 0);
  if (cache) {
    P.cache = view_of(*cache);
    P.k_scale = P.cache.k_scale;
    P.v_scale = P.cache.v_scale;
    P.heads = P.nq + 2 * P.Hkv;
  }
  P.k_inverse = exact_inverse(P.k_scale);
  P.v_inverse = exact_inverse(P.v_scale);
  P.k_sixth = sixth_of(P.k_scale);
  P.v_sixth = sixth_of(P.v_scale);
  if (P.num_rows == 0 || P.slots == 0 || P.heads == 0) return SV_OK;
  const int sms = device_sms();
  if (sms <= 0) return record_error(SV_ERR_CUDA, "%s: no current CUDA device", who);

  while ((16 << P.lane_shift) < P.D) ++P.lane_shift;
  const Layout layout = !P.half ? kPaired : a.layout == SV_ROPE_INTERLEAVED ? kNeighbours
                        : P.half % (cache ? 16 : 8) == 0 ? kPaired : kFar;
  // Threads of a row: 128 where rows are few (both ways 4.6 us for 288 slots; 576 rows with pages 7.6
  // by this rule, 6.7 by the next), else as many as leave a lane up to 12 heads (32768 rows of 48
  // heads 123 us; with up to 6, two warps a row, 137).  A few rows' heads are shared by CTAs until
  // each SM has 512 threads of them (288 slots 4.6 us; with 256 5.5, 1024 4.7), more rows' as long as
  // all CTAs run at once (864 and 1440 rows of 48 heads 6.9 and 10.1 us, by the other rule 7.7 and
  // 11.8; 720 rows into pages 7.7, by the other rule 7.5).
  const bool few = P.slots <= 2 * static_cast<int64_t>(sms);
  P.row_shift = few ? 7 : 5;
  while (P.row_shift < 7 && (12 << P.row_shift) < (P.heads << P.lane_shift)) ++P.row_shift;
  P.pairs = (layout == kNeighbours ? P.D / 2 + 3 : P.half + 7) / 4 * 4;
  const int at_once = 1 << (P.row_shift - P.lane_shift), rows_per_cta = kNT >> P.row_shift;
  const int64_t row_ctas = (P.slots + rows_per_cta - 1) / rows_per_cta;
  const int64_t threads = (P.slots * P.heads) << P.lane_shift, room = 512 * static_cast<int64_t>(sms);
  const int64_t resident = static_cast<int64_t>(sms) * (layout == kFar || a.dtype == SV_F32 ? 2 : cache ? 3 : 4);
  const int64_t shares = std::max<int64_t>(1, resident / row_ctas);
  const int64_t heads = few ? (threads + room - 1) / room * at_once : (P.heads + shares - 1) / shares;
  P.heads_per_cta = static_cast<int>(std::min<int64_t>(P.heads, (heads + at_once - 1) / at_once * at_once));
  const dim3 grid(static_cast<unsigned>(row_ctas),
                  static_cast<unsigned>((P.heads + P.heads_per_cta - 1) / P.heads_per_cta));
  const size_t turns = turn_bytes(rows_per_cta, P.pairs, 1 << P.lane_shift);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.dtype == SV_BF16)
    e = cache                     ? launch_layout<uint16_t, kPages>(layout, grid, turns, s, P)
        : a.kv_dtype == SV_E4M3 ? launch_layout<uint16_t, kCodes8>(layout, grid, turns, s, P)
                                  : launch_layout<uint16_t, kRows>(layout, grid, turns, s, P);
  else
    e = cache                     ? launch_layout<float, kPages>(layout, grid, turns, s, P)
        : a.kv_dtype == SV_E4M3 ? launch_layout<float, kCodes8>(layout, grid, turns, s, P)
                                  : launch_layout<float, kRows>(layout, grid, turns, s, P);
  if (e != cudaSuccess) return record_error(SV_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return SV_OK;
}

// The rotary checks, of which those of turns and rot_dim fall away without a table.
sv_status check_rows(sv_rope_args a, const char *who) {
  alignas(16) static const uint64_t none[2] = {0, 0};
  if (!a.turns) {
    a.turns = none;
    a.rot_dim = 2;
  }
  return check_rope(&a, who);
}

}  // namespace

sv_status check_cache(const sv_kv4_cache *c, const char *who) {
  auto scale = [](float x) { return x == 0.0f || (x >= 0x1p-64f && x <= 0x1p64f); };
  if (c->head_dim != 64 && c->head_dim != 128)
    return record_error(SV_ERR_UNSUPPORTED, "%s: head_dim %d (built: 64, 128)", who, c->head_dim);
  if (c->num_kv_heads < 1 || c->num_kv_heads > 1024)
    return record_error(SV_ERR_INVALID, "%s: num_kv_heads %d outside [1, 1024]", who, c->num_kv_heads);
  if (c->page_size < 16 || c->page_size > 4096 || c->page_size % 16)
    return record_error(SV_ERR_INVALID, "%s: page_size %d (a multiple of 16, 16..4096)", who, c->page_size);
  if (c->max_pages < 0 || (c->table_stride != 0 && c->table_stride < c->max_pages) ||
      c->table_stride > (int64_t{1} << 40))
    return record_error(SV_ERR_INVALID, "%s: max_pages %d, table_stride %lld", who, c->max_pages,
                        static_cast<long long>(c->table_stride));
  if (c->num_pages < 1 || c->num_pages >= (int64_t{1} << 31))
    return record_error(SV_ERR_INVALID, "%s: num_pages %lld", who, static_cast<long long>(c->num_pages));
  if (!scale(c->k_scale) || !scale(c->v_scale))
    return record_error(SV_ERR_INVALID, "%s: k_scale / v_scale outside [2^-64, 2^64]", who);
  if (!c->pages || !is_aligned16(c->pages))
    return record_error(SV_ERR_INVALID, "%s: pages null or not 16-byte aligned", who);
  if (!c->table && c->max_pages > 0) return record_error(SV_ERR_INVALID, "%s: null table", who);
  return SV_OK;
}

Kv4View view_of(const sv_kv4_cache &c) {
  Kv4View v{};
  v.pages = static_cast<uint8_t *>(c.pages);
  v.table = c.table;
  v.table_stride = c.table_stride ? c.table_stride : c.max_pages;
  v.num_pages = c.num_pages;
  v.max_pages = c.max_pages;
  v.page_size = c.page_size;
  v.slabs = c.page_size / kSlab;
  v.heads = c.num_kv_heads;
  v.D = c.head_dim;
  v.k_scale = c.k_scale == 0.0f ? 1.0f : c.k_scale;
  v.v_scale = c.v_scale == 0.0f ? 1.0f : c.v_scale;
  return v;
}

}  // namespace sv

extern "C" {

SV_API sv_status spec_norm_rope_rows(const sv_norm_rope_args *a, void *stream) {
  using namespace sv;
  const char *who = "norm_rope";
  if (!a) return record_error(SV_ERR_INVALID, "%s: null arguments", who);
  sv_status st = check_rows(a->rope, who);
  if (st == SV_OK) st = check_norm(a->norm, who);
  if (st != SV_OK) return st;
  return run_rows(a->rope, a->norm, nullptr, who, stream);
}

SV_API sv_status spec_kv4_append(const sv_kv4_append_args *a, void *stream) {
  using namespace sv;
  const char *who = "kv4_append";
  if (!a) return record_error(SV_ERR_INVALID, "%s: null arguments", who);
  sv_status st = check_cache(&a->cache, who);
  if (st != SV_OK) return st;
  sv_rope_args r = a->rows;
  if (r.positions) return record_error(SV_ERR_INVALID, "%s: positions are kv_len + j", who);
  if (r.num_kv_heads != a->cache.num_kv_heads || r.head_dim != a->cache.head_dim)
    return record_error(SV_ERR_INVALID, "%s: rows of %d heads of %d, a cache of %d of %d", who,
                        r.num_kv_heads, r.head_dim, a->cache.num_kv_heads, a->cache.head_dim);
  if (r.num_rows != 0 && (!r.k || !r.v)) return record_error(SV_ERR_INVALID, "%s: null k or v", who);
  r.kv_dtype = 0;
  r.k_scale = r.v_scale = 0.0f;
  r.k_out = r.v_out = a->cache.pages;                // (unused; the checks want some)
  if (r.num_rows != 0 && (r.k == r.k_out || r.v == r.v_out))
    return record_error(SV_ERR_INVALID, "%s: k or v is the cache", who);
  if ((st = check_rows(r, who)) != SV_OK || (st = check_norm(a->norm, who)) != SV_OK) return st;
  return run_rows(r, a->norm, &a->cache, who, stream);
}

SV_API sv_status spec_kv4_read(const sv_kv4_read_args *a, void *stream) {
  using namespace sv;
  const char *who = "kv4_read";
  if (!a) return record_error(SV_ERR_INVALID, "%s: null arguments", who);
  const sv_status st = check_cache(&a->cache, who);
  if (st != SV_OK) return st;
  auto positive = [](float x) { return x == 0.0f || (std::isfinite(x) && x > 0.0f); };
  if (a->batch < 0 || a->max_q_rows < 1 || static_cast<int64_t>(a->batch) * a->max_q_rows >= (int64_t{1} << 31))
    return record_error(SV_ERR_INVALID, "%s: batch %d, max_q_rows %d", who, a->batch, a->max_q_rows);
  if (a->dtype != SV_BF16 && a->dtype != SV_F32 && a->dtype != SV_E4M3)
    return record_error(SV_ERR_INVALID, "%s: dtype %d", who, a->dtype);
  if (a->reserved != 0) return record_error(SV_ERR_INVALID, "%s: reserved must be 0", who);
  if (a->num_rows < 0 || a->num_rows >= (int64_t{1} << 31))
    return record_error(SV_ERR_INVALID, "%s: num_rows %lld", who, static_cast<long long>(a->num_rows));
  if (!positive(a->k_out_scale) || !positive(a->v_out_scale))
    return record_error(SV_ERR_INVALID, "%s: output scales must be finite and >= 0", who);
  if (a->batch > 0 && (!a->cu_q || !a->kv_len))
    return record_error(SV_ERR_INVALID, "%s: null cu_q or kv_len", who);
  if (!is_aligned16(a->k_out) || !is_aligned16(a->v_out))
    return record_error(SV_ERR_INVALID, "%s: outputs must be 16-byte aligned", who);
  ReadParams P{};
  P.batch = a->batch;
  P.max_q_rows = a->max_q_rows;
  P.D = a->cache.head_dim;
  P.num_rows = a->num_rows;
  P.cu_q = a->cu_q;
  P.kv_len = a->kv_len;
  P.k_scale = a->k_out_scale == 0.0f ? 1.0f : a->k_out_scale;
  P.v_scale = a->v_out_scale == 0.0f ? 1.0f : a->v_out_scale;
  P.k_inverse = exact_inverse(P.k_scale);
  P.v_inverse = exact_inverse(P.v_scale);
  P.k_out = a->k_out;
  P.v_out = a->v_out;
  P.cache = view_of(a->cache);
  // (bf16 and fp32 rows keep what f16 would overflow at: factors above 2^4 are not brief there)
  const bool codes = a->dtype == SV_E4M3;
  const float k_all = codes ? P.cache.k_scale / P.k_scale : P.cache.k_scale;
  const float v_all = codes ? P.cache.v_scale / P.v_scale : P.cache.v_scale;
  P.k_short = codes || k_all <= 16.0f ? short_factor(k_all) : 0;
  P.v_short = codes || v_all <= 16.0f ? short_factor(v_all) : 0;
  P.dev_status = a->dev_status;
  set_slots(P);
  if (P.num_rows == 0 || P.slots == 0 || (!P.k_out && !P.v_out)) return SV_OK;
  // Threads of a row: a warp, which looks the row up once for all heads, where rows are
  // many; else as many as a pass over K and V takes, in slices of a head per thread.
  const int sms = device_sms();
  if (sms <= 0) return record_error(SV_ERR_CUDA, "%s: no current CUDA device", who);
  const int threads = P.cache.heads * (P.D / (codes ? kItem<uint8_t> : kItem<float>));          // an item each
  P.row_shift = 5;
  int slices = 1;
  if (P.slots * threads < int64_t{2048} * sms) {
    while (P.row_shift < 7 && (1 << P.row_shift) < threads) ++P.row_shift;
    slices = (threads + (1 << P.row_shift) - 1) >> P.row_shift;
  }
  const int rows_per_cta = kNT >> P.row_shift;
  const dim3 grid(static_cast<unsigned>((P.slots + rows_per_cta - 1) / rows_per_cta),
                  static_cast<unsigned>(slices));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  static SharedLimit none(0);
  const cudaError_t e =
      a->dtype == SV_BF16  ? launch_after_previous(kv4_read_kernel<uint16_t>, none, grid, kNT, size_t{0}, s, P)
      : a->dtype == SV_F32 ? launch_after_previous(kv4_read_kernel<float>, none, grid, kNT, size_t{0}, s, P)
                           : launch_after_previous(kv4_read_kernel<uint8_t>, none, grid, kNT, size_t{0}, s, P);
  if (e != cudaSuccess) return record_error(SV_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return SV_OK;
}

}  // extern "C"
