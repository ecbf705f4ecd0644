// Penalties, biases and grammar masks on logits rows, and the table of tokens
// that the penalties read (sm_103a).  Contract: spec_adjust_logits and
// spec_count_tokens in include/spec_ops.h.
//
// Adjusting is a copy with exceptions.  The copy (out of place: every row read
// and written once, 2 V elements per row) is what the time goes into; the
// exceptions are few: the tokens of the history, the biased ones and the
// block's drafts, a few thousand of V per sequence, but spread so that most
// 512-byte pieces of a row hold one.  What has to stay small is the number of
// instructions per byte, and the chain of dependent loads before the first row
// can be changed.  A CTA takes a chunk of the vocabulary (4 KB of a row, 1 KB
// where that gives too few CTAs) for one sequence; each of its warps lists the
// exceptions of its share of the chunk (the table's bits say where they are, so
// its counts are read only there) while the first rows are on their way.  From
// then on every warp works alone, a row's chunk at a time: 16-byte cp.async
// copies into shared memory, the listed tokens changed there, a lane per token,
// and the chunk written out.  Many long rows in place are not streamed: masked
// rows are written where a token is barred, and the listed tokens of every row
// are changed in global memory.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "ops_host.inl"
#include "spec_ops.h"

namespace sv {

namespace {

constexpr int kNT = 256;                   // threads of the table's kernels
constexpr float kMinRepetition = 0x1p-64f, kMaxRepetition = 0x1p64f;   // (see penalized())
constexpr int64_t kMaxEntries = int64_t{1} << 30;   // tokens, biases: a strided int index stays one
constexpr int kBatch = 3;                  // (sparse) rows in flight per warp
constexpr int kAhead = 4;                  // listed tokens in flight per lane and row
constexpr int kMaskVecs = 4;               // (sparse) vectors of a masked row in flight per lane

// ---------------------------------------------------------------- adjust
template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {
  static constexpr uint16_t kNegInf = 0xFF80u;
  static __device__ __forceinline__ float get(uint16_t b) { return bf16_bits_to_f32(b); }
  static __device__ __forceinline__ uint16_t put(float x) { return f32_to_bf16_rn(x); }
};
template <>
struct Elem<float> {
  static constexpr float kNegInf = -INFINITY;
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};

// A known token's logit.  The quotient by the repetition penalty r from r's rounded
// reciprocal: two corrections by the exact remainder y - q r.  The first leaves less
// than one unit of the last place, from where the second gives the rounded quotient
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) as long as nothing in it over- or underflows: y in [2^-60, 2^60] and
// r in [2^-64, 2^64].  Farther logits take the first product, within 2^-23.  All of it in
// selects, so that the tokens a lane has in flight overlap (bass_b8 verify rows: 6.3 us
// with the product alone, 6.4 so, 7.0 behind a branch, 8.0 by the division operator).
__device__ __forceinline__ float penalized(float y, float rep, float inverse) {
  const float z = y * (y > 0.0f ? inverse : rep);
  float q = fmaf(fmaf(-z, rep, y), inverse, z);
  q = fmaf(fmaf(-q, rep, y), inverse, q);
  constexpr uint32_t kLeast = (127u - 60u) << 23, kRange = 120u << 23;      // 2^-60; up to 2^60
  return __float_as_uint(y) - kLeast <= kRange ? q : z;
}

struct AdjustParams {
  sv_adjust_args a;
  int lines_per_part;            // rows (target, then draft) that one CTA works on
  int64_t mask_bytes;            // bytes per mask row
  int seen_words;
};

// The kPer bits from bit b of mask bytes on; bytes: how many there are.
template <int kPer>
__device__ __forceinline__ uint32_t mask_bits(const uint8_t *m, int b, int64_t bytes) {
  uint32_t w = m[b >> 3];
  if ((b & 7) + kPer > 8 && (b >> 3) + 1 < bytes) w |= static_cast<uint32_t>(m[(b >> 3) + 1]) << 8;
  return (w >> (b & 7)) & ((1u << kPer) - 1);
}

// One vector of a row; the tokens whose bit is 0 are barred.
template <typename T, int kPer>
union Piece {
  uint4 w;
  T e[kPer];
  __device__ __forceinline__ void bar(uint32_t allow) {
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (!((allow >> k) & 1u)) e[k] = Elem<T>::kNegInf;
  }
};

// How a kernel cuts its work.  A CTA takes a chunk of BYTES of a row.  UNIT > 0:
// its warps stream the rows' chunks in units of UNIT bytes, two units of shared
// memory each, every unit with a list of its own.  UNIT = 0: in place, only what
// changes; one list, and few warps, for all they do is wait.
template <typename T, int BYTES, int UNIT>
struct Chunk {
  static constexpr bool kSparse = UNIT == 0;
  static constexpr int kPer = 16 / static_cast<int>(sizeof(T));       // elements of a vector
  static constexpr int kTokens = BYTES / static_cast<int>(sizeof(T));
  static constexpr int kWarps = kSparse ? 4 : 8, kThreads = kWarps * 32;
  static constexpr int kUnitBytes = kSparse ? BYTES : UNIT;
  static constexpr int kUnits = BYTES / kUnitBytes, kUnitTokens = kTokens / kUnits;
  static constexpr int kWords = kTokens / 32 / kWarps;                // of each warp's share
  static constexpr int kVecs = kUnitBytes / 16 / 32;                  // vectors per lane and unit
  static constexpr int kMaskAt = kUnitBytes + 16;                     // (a misaligned row's last vector)
  static constexpr int kSlot = kMaskAt + kUnitTokens / 8;             // a unit and its mask
  static constexpr int kRing = 2;
  static constexpr int kRingBytes = kSparse ? 0 : kWarps * kRing * kSlot;
  static_assert(kWords >= 1 && kWords <= 32 && kTokens <= 2048, "");
  static_assert(kSparse || (kSlot % 16 == 0 && kUnitTokens % (kWords * 32) == 0), "");
};

// A listed token: its place in the chunk; above kDraft: 1 + the first of the
// block's drafts that it is (its row of s_after), or 0; and one flag, that it is
// counted outside the table until its list is complete, that it has a bias then.
constexpr uint16_t kFlag = 0x800u, kPlace = 0x7FFu;
constexpr int kDraft = 12;

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}

// RAGGED: V is no multiple of a vector's elements, so rows differ in alignment.
template <typename T, int BYTES, int UNIT, bool RAGGED>
__global__ void __launch_bounds__(Chunk<T, BYTES, UNIT>::kThreads, UNIT == 0 ? 8 : 4)
adjust_kernel(const __grid_constant__ AdjustParams P) {
  using E = Elem<T>;
  using C = Chunk<T, BYTES, UNIT>;
  constexpr bool SPARSE = C::kSparse;
  constexpr int kPer = C::kPer, kWarps = C::kWarps, kThreads = C::kThreads;
  constexpr uint32_t kAll = (1u << kPer) - 1;
  const sv_adjust_args &a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, i = blockIdx.x;
  const int V = a.vocab, t0 = blockIdx.y * C::kTokens, width = min(V - t0, C::kTokens);
  const bool head = blockIdx.y == 0 && blockIdx.z == 0;      // this CTA reports the sequence

  extern __shared__ __align__(16) unsigned char s_dyn[];     // the ring; with biases: s_last
  int32_t *s_last = reinterpret_cast<int32_t *>(s_dyn + C::kRingBytes);   // 1 + last bias entry of
                                                             // a token; then its bias, as bits
  __shared__ uint32_t s_extra[C::kTokens / 32];              // bits of ctx, draft and bias tokens
  __shared__ uint32_t s_word[C::kTokens];                    // table words of the lists, with ctx
  __shared__ uint16_t s_tok[C::kTokens];                     // the lists
  __shared__ uint32_t s_after[16];                           // [1 + d]: bit e: draft e + 1 is draft d + 1
  __shared__ int s_n[C::kUnits];

  wait_for_previous();
  const int r0 = a.cu_q[i], r1 = a.cu_q[i + 1];
  const float rep = a.repetitions ? a.repetitions[i] : a.repetition;
  const float pres = a.presences ? a.presences[i] : a.presence;
  const float freq = a.frequencies ? a.frequencies[i] : a.frequency;
  const int slot = a.counts == nullptr ? -1 : a.slots ? a.slots[i] : i;
  int b0 = 0, b1 = 0;
  if (a.bias_start) {
    b0 = a.bias_start[i];
    b1 = a.bias_start[i + 1];
    for (int t = tid; t < C::kTokens / 4; t += kThreads)
      reinterpret_cast<int4 *>(s_last)[t] = make_int4(0, 0, 0, 0);
  }
  for (int w = tid; w < C::kTokens / 32; w += kThreads) s_extra[w] = 0;
  if (tid < C::kUnits) s_n[tid] = 0;
  __syncthreads();

  // (compared before they are subtracted: far apart, the difference wraps)
  if (r0 < i || r1 <= r0 || r1 > a.num_rows || r1 - r0 > a.max_q_rows ||
      r1 - (i + 1) > a.num_rows - a.batch) {                 // (its draft rows, too)
    if (head && tid == 0) set_status(a.dev_status, SV_DEV_BAD_LENGTH);
    return;
  }
  const int Ri = r1 - r0;
  const int all = Ri + (a.draft != nullptr ? Ri - 1 : 0);    // target rows, then draft rows
  const int l0 = blockIdx.z * P.lines_per_part, lines = min(all - l0, P.lines_per_part);
  if (lines <= 0) return;

  // Row `line` of this part, at the chunk's first token.
  auto block_row = [&](int line) { return l0 + line < Ri ? l0 + line : l0 + line - Ri; };
  auto row_index = [&](int line) {
    return static_cast<int64_t>(l0 + line < Ri ? r0 : r0 - i) + block_row(line);
  };
  auto row_in = [&](int line) {
    return static_cast<const T *>(l0 + line < Ri ? a.target : a.draft) + row_index(line) * V + t0;
  };
  auto row_out = [&](int line) {
    return static_cast<T *>(l0 + line < Ri ? a.target_out : a.draft_out) + row_index(line) * V + t0;
  };
  // elements from the 16-byte boundary before the chunk to the chunk
  auto misaligned = [&](int line) {
    return RAGGED ? static_cast<int>((static_cast<uint32_t>(row_index(line)) * static_cast<uint32_t>(V)) & (kPer - 1)) : 0;
  };

  // Unit u (row u / kUnits) into slot s of this warp's ring: 16-byte vectors
  // from the boundary at or before the unit's first token up to its last one.
  unsigned char *ring = s_dyn + warp * (C::kRing * C::kSlot);
  const int units = lines * C::kUnits;
  auto fetch = [&](int u, int s) {
    const int line = u / C::kUnits, from = (u % C::kUnits) * C::kUnitTokens, uw = width - from;
    if (uw <= 0) return;
    const int mis = misaligned(line);
    const uint32_t dst = smem_u32(ring + s * C::kSlot) + lane * 16;
    const T *src = row_in(line) + from - mis + lane * kPer;
    if (uw >= C::kUnitTokens) {
#pragma unroll
      for (int q = 0; q < C::kVecs; ++q) cp_async16(dst + q * 512, src + q * 32 * kPer, 16);
      if (RAGGED && lane == 0 && mis)
        cp_async16(dst + C::kUnitBytes, src + C::kUnitTokens, mis * static_cast<int>(sizeof(T)));
    } else {
      const int left = uw + mis - lane * kPer;               // elements from this lane's first on
#pragma unroll 1
      for (int q = 0; left > q * 32 * kPer; ++q)             // (at most kVecs + 1: the slot holds them)
        cp_async16(dst + q * 512, src + q * 32 * kPer,
                   min(16, (left - q * 32 * kPer) * static_cast<int>(sizeof(T))));
    }
  };
  if constexpr (!SPARSE) {
    if (warp < units) fetch(warp, 0);
    if (warp + kWarps < units) fetch(warp + kWarps, 1);
  }

  const bool penal = rep != 1.0f || pres != 0.0f || freq != 0.0f;
  const int nb = b1 - b0;
  bool bad = !(rep >= kMinRepetition && rep <= kMaxRepetition) || !isfinite(pres) || !isfinite(freq) ||
             slot < -1 || slot >= max(a.num_slots, 0) || b0 < 0 || b1 < b0 || b1 > a.num_bias;
  int my_mask = -1;                                          // lane j: mask row of block row j
  if (a.mask && lane < Ri) my_mask = a.mask_rows ? a.mask_rows[r0 + lane] : r0 + lane;
  const int drafts = penal && a.draft_tokens ? Ri - 1 : 0;
  int my_draft = -1;                                         // lane d: draft d + 1, in the chunk
  if (lane < drafts) {
    const int t = a.draft_tokens[r0 - i + lane];
    my_draft = t >= t0 && t - t0 < width ? t - t0 : -1;
  }
  // the table's bits of this warp's share, a word per lane
  const int w0 = warp * C::kWords;
  uint32_t known = 0;
  if (!bad && penal && slot >= 0 && lane < C::kWords && (w0 + lane) * 32 < width)
    known = a.seen[static_cast<int64_t>(slot) * P.seen_words + (t0 >> 5) + w0 + lane];

  // tokens outside the table, by the whole CTA
  const int ctx = penal ? a.num_ctx : 0;
  const int64_t ctx_stride = a.ctx_stride ? a.ctx_stride : a.batch;
  auto mark = [&](int t) { atomicOr(&s_extra[t >> 5], 1u << (t & 31)); };
  auto in_chunk = [&](int t) { return t >= t0 && t - t0 < width; };
  if (!bad) {
    for (int c = tid; c < ctx; c += kThreads) {
      const int t = a.ctx_tokens[c * ctx_stride + i];
      if (in_chunk(t)) mark(t - t0);
    }
#pragma unroll 4
    for (int e = tid; e < nb; e += kThreads) {
      const int t = a.bias_tokens[b0 + e];
      if (in_chunk(t)) {
        mark(t - t0);
        atomicMax(&s_last[t - t0], e + 1);
      } else if (head && (t < 0 || t >= V)) {
        set_status(a.dev_status, SV_DEV_BAD_TOKEN);
      }
    }
  }
  if (warp == 0) {
    const uint32_t same = __match_any_sync(0xffffffffu, my_draft);
    if (lane < 16) s_after[lane] = 0;
    __syncwarp();
    if (my_draft >= 0) {
      mark(my_draft);
      s_after[1 + lane] = same;
    }
  }
  bad |= my_mask < -1 || (my_mask >= 0 && my_mask >= a.num_masks);
  bad = __syncthreads_or(bad);

  if (bad) {                      // rows the sampler fails the sequence on
    if (head && tid == 0) set_status(a.dev_status, SV_DEV_BAD_PARAM);
    if constexpr (!SPARSE) {
      cp_async_commit();
      cp_async_wait<0>();
    }
    for (int line = warp; line < lines; line += kWarps) {
      T *out = row_out(line);
      for (int t = lane; t < width; t += 32) out[t] = E::put(NAN);
    }
    return;
  }
  const uint32_t masked = __ballot_sync(0xffffffffu, my_mask >= 0);   // bit j: row j has a mask
  auto mask_of = [&](int j) -> const uint8_t * {             // by all lanes
    const int m = __shfl_sync(0xffffffffu, my_mask, j);
    return m < 0 ? nullptr : reinterpret_cast<const uint8_t *>(a.mask) + m * P.mask_bytes + (t0 >> 3);
  };
  auto fetch_mask = [&](int u, int s) {                      // a unit's mask words, by all lanes
    const int j = block_row(u / C::kUnits), from = (u % C::kUnits) * C::kUnitTokens;
    if (!((masked >> j) & 1u)) return;
    const uint8_t *mask = mask_of(j) + (from >> 3);
    const uint32_t dst = smem_u32(ring + s * C::kSlot + C::kMaskAt);
    for (int w = lane; w < C::kUnitTokens / 32 && from + w * 32 < width; w += 32)
      cp_async4(dst + w * 4, mask + w * 4);
  };
  if constexpr (!SPARSE) {
    if (warp < units) fetch_mask(warp, 0);
    if (warp + kWarps < units) fetch_mask(warp + kWarps, 1);
    cp_async_commit();                                       // both first units
    cp_async_commit();
  }

  // the share's list: each lane its word's tokens where they are few, else a
  // word at a time with a lane per bit
  const int my_unit = w0 * 32 / C::kUnitTokens;
  {
    uint32_t extra = 0, any = 0;
    if (lane < C::kWords) {
      extra = s_extra[w0 + lane];
      any = known | extra;
      const int left = width - (w0 + lane) * 32;
      if (left < 32) any &= left > 0 ? (1u << left) - 1 : 0u;
    }
    int count = __popc(any), before = count;                 // of this lane, of the lanes up to it
    const int most = __reduce_max_sync(0xffffffffu, count);
#pragma unroll
    for (int o = 1; o < C::kWords; o <<= 1) {
      const int c = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += c;
    }
    const int total = __shfl_sync(0xffffffffu, before, C::kWords - 1);
    before -= count;
    int base = 0;
    if (lane == 0 && total) base = my_unit * C::kUnitTokens + atomicAdd(&s_n[my_unit], total);
    base = __shfl_sync(0xffffffffu, base, 0);
    auto enter = [&](int e, int q, int b, bool in_table, bool out) {
      s_word[e] = in_table;                                  // read below
      s_tok[e] = static_cast<uint16_t>(((w0 + q) * 32 + b) | (out ? kFlag : 0));
    };
    if (most <= 4) {
      int e = base + before;
      while (any) {
        const int b = __ffs(any) - 1;
        any &= any - 1;
        enter(e++, lane, b, (known >> b) & 1u, (extra >> b) & 1u);
      }
    } else {
#pragma unroll 1
      for (int q = 0; q < C::kWords; ++q) {
        const uint32_t w = __shfl_sync(0xffffffffu, any, q), kw = __shfl_sync(0xffffffffu, known, q),
                       ew = __shfl_sync(0xffffffffu, extra, q);
        const int e = base + __shfl_sync(0xffffffffu, before, q) + __popc(w & ((1u << lane) - 1));
        if ((w >> lane) & 1u) enter(e, q, lane, (kw >> lane) & 1u, (ew >> lane) & 1u);
      }
    }
    __syncwarp();
    const int32_t *counts = a.counts + static_cast<int64_t>(slot) * V + t0;
#pragma unroll 4
    for (int e0 = 0; e0 < total; e0 += 32) {
      const int e = base + e0 + lane;
      const bool on = e0 + lane < total;
      const int tok = on ? s_tok[e] : 0, t = tok & kPlace;
      uint32_t word = on && s_word[e] ? static_cast<uint32_t>(counts[t]) : 0u;
      if (__any_sync(0xffffffffu, tok & kFlag)) {
        int entry = t;
        if ((tok & kFlag) && nb > 0 && s_last[t]) {
          s_last[t] = __float_as_int(a.bias_values[b0 + s_last[t] - 1]);
          entry |= kFlag;
        }
        if (tok & kFlag)
          for (int c = 0; c < ctx; ++c) word += a.ctx_tokens[c * ctx_stride + i] == t0 + t;
        for (int d = drafts - 1; d >= 0; --d)
          if (__shfl_sync(0xffffffffu, my_draft, d) == t) entry = (entry & (kFlag | kPlace)) | ((1 + d) << kDraft);
        if (on) s_tok[e] = static_cast<uint16_t>(entry);
      }
      if (on) s_word[e] = word;
    }
  }
  __syncthreads();

  // One listed token of block row j.
  const float inverse = 1.0f / rep;
  auto changed = [&](T old, int tok, uint32_t word, int j) {
    const uint32_t times = (word & 0x7FFFFFFFu) + __popc(s_after[tok >> kDraft] & ((1u << j) - 1));
    float y = E::get(old);
    const float known = penalized(y, rep, inverse);
    y = (word | times) != 0 ? known : y;
    if (times != 0) y -= fmaf(freq, static_cast<float>(times), pres);
    if (tok & kFlag) y += __int_as_float(s_last[tok & kPlace]);
    return E::put(y);
  };

  if constexpr (!SPARSE) {
    int s = 0;
#pragma unroll 1
    for (int u = warp; u < units; u += kWarps, s ^= 1) {
      cp_async_wait<1>();
      __syncwarp();
      const int line = u / C::kUnits, unit = u % C::kUnits, j = block_row(line);
      const int from = unit * C::kUnitTokens, uw = min(width - from, C::kUnitTokens);
      const int mis = misaligned(line), n = s_n[unit];
      unsigned char *row = ring + s * C::kSlot;
      T *x = reinterpret_cast<T *>(row) + mis;               // the unit's tokens
#pragma unroll 1
      for (int eb = 0; eb < n; eb += 32 * kAhead) {
        int tok[kAhead];
        uint32_t word[kAhead];
        T old[kAhead];
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
          if (eb + h * 32 >= n) break;
          const int e = eb + h * 32 + lane;
          if (e < n) {
            tok[h] = s_tok[from + e];
            word[h] = s_word[from + e];
            old[h] = x[(tok[h] & kPlace) - from];
          }
        }
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
          if (eb + h * 32 >= n) break;
          if (eb + h * 32 + lane < n)
            x[(tok[h] & kPlace) - from] = changed(old[h], tok[h], word[h], j);
        }
      }
      __syncwarp();
      const bool barred = (masked >> j) & 1u;
      const uint8_t *bits = row + C::kMaskAt;
      T *out = row_out(line) + from - mis;                   // vectors as they were read
      if (uw == C::kUnitTokens) {
#pragma unroll
        for (int q = 0; q < C::kVecs; ++q) {
          const int v = (lane + q * 32) * kPer, t = v - mis;
          if (RAGGED && t < 0) continue;                     // (shared with the tokens before)
          Piece<T, kPer> piece;
          piece.w = *reinterpret_cast<const uint4 *>(row + (lane + q * 32) * 16);
          if (barred) piece.bar(mask_bits<kPer>(bits, t, C::kUnitTokens / 8));
          *reinterpret_cast<uint4 *>(out + v) = piece.w;
        }
        if (RAGGED && mis && lane < kPer) {                  // the two ends, an element per lane
          const int t = lane >= mis ? lane - mis : C::kUnitTokens - mis + lane;
          const bool allowed = !barred || ((bits[t >> 3] >> (t & 7)) & 1u);
          out[t + mis] = allowed ? x[t] : E::kNegInf;
        }
      } else {
#pragma unroll 1
        for (int v = lane * kPer; v - mis < uw; v += 32 * kPer) {
          const int t = v - mis;
          Piece<T, kPer> piece;
          piece.w = *reinterpret_cast<const uint4 *>(row + v * static_cast<int>(sizeof(T)));
          if (barred)                                        // (bits outside the unit say nothing)
            piece.bar(t >= 0 ? mask_bits<kPer>(bits, t, C::kUnitTokens / 8)
                             : mask_bits<kPer>(bits, 0, C::kUnitTokens / 8) << -t);
          if (t >= 0 && t + kPer <= uw) {
            *reinterpret_cast<uint4 *>(out + v) = piece.w;
          } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
              if (t + k >= 0 && t + k < uw) out[v + k] = piece.e[k];
          }
        }
      }
      __syncwarp();                                          // the slot is free
      if (u + 2 * kWarps < units) {
        fetch(u + 2 * kWarps, s);
        fetch_mask(u + 2 * kWarps, s);
      }
      cp_async_commit();
    }
  } else {
    // masked rows: barred tokens written, vectors that stay whole not touched
    if (masked)
#pragma unroll 1
      for (int line = warp; line < lines; line += kWarps) {
        const uint8_t *mask = mask_of(block_row(line));
        if (!mask) continue;
        const int mis = misaligned(line), first = RAGGED ? (kPer - mis) & (kPer - 1) : 0;
        T *row = row_out(line);
#pragma unroll 1
        for (int t0v = first + lane * kPer; t0v < width; t0v += kMaskVecs * 32 * kPer) {
          Piece<T, kPer> x[kMaskVecs];
          uint32_t allow[kMaskVecs];
#pragma unroll
          for (int q = 0; q < kMaskVecs; ++q) {
            const int t = t0v + q * 32 * kPer;
            allow[q] = t + kPer <= width ? mask_bits<kPer>(mask, t, (width + 7) >> 3) : kAll;
          }
#pragma unroll
          for (int q = 0; q < kMaskVecs; ++q)
            if (allow[q] != 0 && allow[q] != kAll)
              x[q].w = *reinterpret_cast<const uint4 *>(row + t0v + q * 32 * kPer);
#pragma unroll
          for (int q = 0; q < kMaskVecs; ++q)
            if (allow[q] != kAll) {
              x[q].bar(allow[q]);
              *reinterpret_cast<uint4 *>(row + t0v + q * 32 * kPer) = x[q].w;
            }
        }
        if (RAGGED) {                                        // the ends, one by one
          const int tail = first + (width > first ? (width - first) & ~(kPer - 1) : 0);
          const int t = lane < 16 ? (lane < min(first, width) ? lane : -1)
                                  : (tail + lane - 16 < width ? tail + lane - 16 : -1);
          if (t >= 0 && !((mask[t >> 3] >> (t & 7)) & 1u)) row[t] = E::kNegInf;
        }
      }
    if (masked) __syncthreads();
    // The listed tokens of every row: a row per warp where there are enough
    // rows, else the warps of a row share its tokens.
    const int n = s_n[0];
    const int apart = lines >= kWarps ? kWarps : lines >= 2 ? 2 : 1;   // rows worked on at once
    static_assert(kWarps % 2 == 0, "");
#pragma unroll 1
    for (int lb = warp % apart; lb < lines; lb += kBatch * apart) {
      T *row[kBatch];
      const uint8_t *mask[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (lb + u * apart < lines) {
          row[u] = row_out(lb + u * apart);
          mask[u] = mask_of(block_row(lb + u * apart));
        }
#pragma unroll 1
      for (int eb = warp / apart * (32 * kAhead); eb < n; eb += kWarps / apart * (32 * kAhead)) {
        T x[kAhead][kBatch];
        bool allowed[kAhead][kBatch];
        int tok[kAhead];
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
          const int e = eb + h * 32 + lane;
          tok[h] = e < n ? s_tok[e] : 0;
          const int t = tok[h] & kPlace;
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            allowed[h][u] = e < n && lb + u * apart < lines;
            if (!allowed[h][u]) continue;
            x[h][u] = row[u][t];
            if (mask[u]) allowed[h][u] = (mask[u][t >> 3] >> (t & 7)) & 1u;   // barred: written already
          }
        }
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
          if (eb + h * 32 >= n) break;
          const int e = eb + h * 32 + lane, t = tok[h] & kPlace;
          const uint32_t word = e < n ? s_word[e] : 0u;
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            if (lb + u * apart >= lines) break;
            if (allowed[h][u]) row[u][t] = changed(x[h][u], tok[h], word, block_row(lb + u * apart));
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- count
constexpr int kTokens = 4;                 // of its sequence that a resetting thread has in flight
constexpr int kMaxStart = 4096;            // sequences whose start values are kept in shared memory

struct CountParams {
  sv_count_args a;
  int words;                      // of a slot's bits
};

// One token into the table.  Frequent tokens fall on the same words: a mark that
// is there already is not written again, and additions return nothing.
__device__ __forceinline__ void enter_token(const CountParams &P, int slot, int t) {
  const sv_count_args &a = P.a;
  uint32_t *word = reinterpret_cast<uint32_t *>(a.counts) + static_cast<int64_t>(slot) * a.vocab + t;
  uint32_t *seen = a.seen + static_cast<int64_t>(slot) * P.words + (t >> 5);
  const uint32_t bit = 1u << (t & 31), bits = __ldcg(seen);
  if (a.flags & SV_COUNT_PROMPT) {
    if (!(__ldcg(word) >> 31)) atomicOr(word, 0x80000000u);
  } else {
    atomicAdd(word, 1u);
  }
  if (!(bits & bit)) atomicOr(seen, bit);
}

// One token per thread; its sequence is searched in shared memory.
__global__ void __launch_bounds__(kNT) count_kernel(const __grid_constant__ CountParams P) {
  const sv_count_args &a = P.a;
  extern __shared__ __align__(16) uint32_t s_word[];
  int32_t *s_start = reinterpret_cast<int32_t *>(s_word);     // start, where it fits
  wait_for_previous();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kNT + threadIdx.x;
  const int32_t *start = a.start;
  const int t = at < a.num_tokens ? a.tokens[at] : 0;
  if (a.batch <= kMaxStart) {
    for (int i = threadIdx.x; i <= a.batch; i += kNT) s_start[i] = a.start[i];
    start = s_start;
    __syncthreads();
  }
  if (at < a.batch) {             // one thread per sequence reports
    const int i = static_cast<int>(at);
    const int s0 = start[i], s1 = start[i + 1], slot = a.slots ? a.slots[i] : i;
    if (s0 < 0 || s1 < s0 || s1 > a.num_tokens) set_status(a.dev_status, SV_DEV_BAD_LENGTH);
    if (slot < -1 || slot >= a.num_slots) set_status(a.dev_status, SV_DEV_BAD_PARAM);
  }
  if (at >= a.num_tokens) return;
  // the last sequence that starts at or before this token
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= at) lo = mid; else hi = mid;
  }
  const int i = lo, s0 = start[i], s1 = start[i + 1];
  if (s0 < 0 || at < s0 || at >= s1 || s1 > a.num_tokens) return;
  const int slot = a.slots ? a.slots[i] : i;
  if (a.num_accepted && at - s0 > a.num_accepted[i]) return;
  if (slot < 0 || slot >= a.num_slots) return;
  if (t < 0 || t >= a.vocab) set_status(a.dev_status, SV_DEV_BAD_TOKEN);
  else enter_token(P, slot, t);
}

// Clearing and counting: a CTA owns a slice of one slot's vocabulary and takes
// the sequence's tokens that fall into it (of all sequences that share the
// slot, by the first of them) together in shared memory, as bits for a prompt,
// as counts too otherwise.  Frequent tokens meet there, and what is or was not
// 0 in the table is written once.  Every slice reads all of its sequence's
// tokens, from L2.
template <int NT, bool PROMPT>
__global__ void __launch_bounds__(NT) reset_kernel(const __grid_constant__ CountParams P) {
  const sv_count_args &a = P.a;
  constexpr int kSlice = 32 * NT;                             // a word of bits per thread
  __shared__ uint32_t s_bits[NT];
  __shared__ __align__(16) uint32_t s_word[PROMPT ? 4 : kSlice];
  const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int t0 = blockIdx.y * kSlice, width = min(kSlice, a.vocab - t0);
  const bool head = blockIdx.y == 0;
  wait_for_previous();
  const int slot = a.slots ? a.slots[i] : i;
  auto segment = [&](int j, int &s0, int &n) {                // tokens of sequence j
    s0 = a.start[j];
    const int s1 = a.start[j + 1];
    const bool good = s0 >= 0 && s1 >= s0 && s1 <= a.num_tokens;
    n = good ? s1 - s0 : 0;
    if (good && a.num_accepted && a.num_accepted[j] < n) n = max(a.num_accepted[j] + 1, 0);
    return good;
  };
  int s0, n;
  const bool good = segment(i, s0, n);
  if (head && tid == 0) {
    if (!good) set_status(a.dev_status, SV_DEV_BAD_LENGTH);
    if (slot < -1 || slot >= a.num_slots) set_status(a.dev_status, SV_DEV_BAD_PARAM);
  }
  if (slot < 0 || slot >= a.num_slots) return;
  // loads first: the table's bits, a thread's first tokens, the other slots
  uint32_t *seen = a.seen + static_cast<int64_t>(slot) * P.words + t0 / 32;
  const uint32_t old = tid * 32 < width ? seen[tid] : 0u;
  int t[kTokens];
  auto load = [&](int k0) {
#pragma unroll
    for (int u = 0; u < kTokens; ++u) t[u] = k0 + u * NT < n ? a.tokens[s0 + k0 + u * NT] : t0;
  };
  load(tid);
  bool before = false, after = false;                         // others that share the slot
  if (a.slots)
    for (int j = tid; j < a.batch; j += NT)
      if (j != i && a.slots[j] == slot) (j < i ? before : after) = true;
  s_bits[tid] = 0;
  if constexpr (!PROMPT)
    for (int w = tid; w < kSlice / 4; w += NT) reinterpret_cast<uint4 *>(s_word)[w] = make_uint4(0, 0, 0, 0);
  const int shared = __syncthreads_or(before || after);
  if (shared && __syncthreads_or(before)) return;             // the first of them does it
  for (int j = i;;) {
#pragma unroll 1
    for (int k0 = tid; k0 < n;) {
#pragma unroll
      for (int u = 0; u < kTokens; ++u) {
        if (k0 + u * NT >= n) break;
        if (t[u] >= t0 && t[u] - t0 < width) {
          const int at = t[u] - t0;
          atomicOr(&s_bits[at >> 5], 1u << (at & 31));
          if constexpr (!PROMPT) atomicAdd(&s_word[at], 1u);
        } else if (head && (t[u] < 0 || t[u] >= a.vocab)) {
          set_status(a.dev_status, SV_DEV_BAD_TOKEN);
        }
      }
      k0 += NT * kTokens;
      load(k0);
    }
    if (!shared) break;
    do ++j; while (j < a.batch && a.slots[j] != slot);
    if (j >= a.batch) break;
    segment(j, s0, n);
    load(tid);
  }
  __syncthreads();
  // of each warp's words those with tokens one after the other, a lane per token
  uint32_t *counts = reinterpret_cast<uint32_t *>(a.counts) + static_cast<int64_t>(slot) * a.vocab + t0;
  const uint32_t now = s_bits[tid], any = now | old;
  uint32_t left = __ballot_sync(0xffffffffu, any != 0);
  while (left) {
    const int q = __ffs(left) - 1, at = ((tid & ~31) + q) * 32 + lane;
    left &= left - 1;
    const uint32_t change = __shfl_sync(0xffffffffu, any, q), set = __shfl_sync(0xffffffffu, now, q);
    if (((change >> lane) & 1u) && at < width)
      counts[at] = PROMPT ? ((set >> lane) & 1u) << 31 : s_word[at];
  }
  if (now != old) seen[tid] = now;
}

// ---------------------------------------------------------------- host side
template <typename T, int BYTES, int UNIT, bool RAGGED>
cudaError_t launch_adjust(dim3 grid, const AdjustParams &P, cudaStream_t s) {
  using C = Chunk<T, BYTES, UNIT>;
  constexpr int biases = C::kTokens * 4;                     // s_last
  if constexpr (C::kRingBytes + biases + C::kTokens * 6 > 47 * 1024) {   // past the default
    static std::atomic<uint64_t> ready{0};                   // once per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) & bit)) {
      e = cudaFuncSetAttribute(adjust_kernel<T, BYTES, UNIT, RAGGED>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::kRingBytes + biases);
      if (e != cudaSuccess) return e;
      ready.fetch_or(bit, std::memory_order_release);
    }
  }
  return launch_behind(adjust_kernel<T, BYTES, UNIT, RAGGED>, grid, C::kThreads,
                       C::kRingBytes + (P.a.bias_start ? biases : 0), s, P);
}

template <typename T, int BYTES, int UNIT>
cudaError_t launch_adjust(int parts, AdjustParams &P, cudaStream_t s) {
  const sv_adjust_args &a = P.a;
  const int lines = a.draft ? 2 * a.max_q_rows - 1 : a.max_q_rows;
  P.lines_per_part = (lines + parts - 1) / parts;
  // sequences first: the chunks of the frequent tokens, which have the long
  // lists, start first
  const int tokens = Chunk<T, BYTES, UNIT>::kTokens;
  const dim3 grid(a.batch, (a.vocab + tokens - 1) / tokens, (lines + P.lines_per_part - 1) / P.lines_per_part);
  return a.vocab % Chunk<T, BYTES, UNIT>::kPer ? launch_adjust<T, BYTES, UNIT, true>(grid, P, s)
                                               : launch_adjust<T, BYTES, UNIT, false>(grid, P, s);
}

template <typename T>
cudaError_t launch_adjust(int sms, AdjustParams &P, cudaStream_t s) {
  const sv_adjust_args &a = P.a;
  const int lines = a.draft ? 2 * a.max_q_rows - 1 : a.max_q_rows;
  const int64_t row = static_cast<int64_t>(a.vocab) * sizeof(T);
  // CTAs that a chunk of 4 KB and of 1 KB gives, with all rows of a sequence.
  const int64_t big = (row + 4095) / 4096 * a.batch, small = (row + 1023) / 1024 * a.batch;
  auto split = [&](int64_t ctas, int per_part, int64_t room) {   // the rows over parts (each repeats the list)
    int parts = 1;
    while (parts * per_part < lines && ctas * (parts + 1) <= room * sms) ++parts;
    return parts;
  };
  // In place, changing single tokens in memory pays where a sequence's few
  // thousand listed tokens are thin in the row and there are CTAs enough to
  // hide its longer chain of loads.  This against streaming the rows through, in us
  // (bf16, 9 rows a sequence, 2048 tokens of history, 64 biases, a quarter of the
  // rows masked): V = 128256 at B = 64 45 / 62, B = 32 30 / 35, B = 16 18 / 20, B = 8
  // 12.9 / 10.8; V = 65536 at B = 64 36 / 36, B = 16 13.5 / 11.0; V = 32000, 11 rows, at
  // B = 64 29 / 22, B = 8 13.6 / 6.5.  The rule does not look at how much is listed
  // and barred: V = 128256, B = 64 without masks 18 / 58 (no history), 54 / 67 (8192
  // tokens), 75 / 86 (32768), fp32 45 / 110, 69 / 114 and 98 / 129 at 2048, 8192 and
  // 32768; it loses with every row masked, 67 / 64 (2048) to 108 / 91 (32768; fp32 140 /
  // 135), and with long histories of smaller batches, 55 / 31 at B = 16 with 32768 and
  // every row masked, 43 / 27 at V = 70003, B = 32 with 8192.
  if (a.target == a.target_out && a.vocab >= 65536 && big >= 6 * static_cast<int64_t>(sms))
    return launch_adjust<T, 4096, 0>(split(big, 4, 16), P, s);
  // Streaming: 1 KB chunks until the 4 KB ones (fewer repeated starts) give
  // about two CTAs per SM (bf16, V = 32000, 11 rows a sequence, half of them masked: at
  // B = 8 6.5 against 7.4 us, at B = 16 9.0 and 8.9, at B = 32 20.1 against 16.3, at
  // B = 64 34.8 against 22.3; single rows at B = 8 4.7 against 6.7, at B = 64 20.4
  // against 8.2).
  if (big < 2 * static_cast<int64_t>(sms)) return launch_adjust<T, 1024, 1024>(split(small, 8, 4), P, s);
  return launch_adjust<T, 4096, 2048>(split(big, 4, 8), P, s);
}

sv_status check_adjust(const sv_adjust_args *a) {
  auto bad = [](const char *what) { return record_error(SV_ERR_INVALID, "adjust: %s", what); };
  if (!a) return bad("null arguments");
  if (a->batch < 0 || a->batch > 65535)
    return record_error(SV_ERR_UNSUPPORTED, "adjust: batch %d outside [0, 65535]", a->batch);
  if (a->vocab < 1 || a->vocab > (1 << 23))
    return record_error(SV_ERR_UNSUPPORTED, "adjust: vocab %d outside [1, 2^23]", a->vocab);
  if (a->dtype != SV_F32 && a->dtype != SV_BF16)
    return record_error(SV_ERR_INVALID, "adjust: dtype %d", a->dtype);
  if (a->max_q_rows < 1 || a->max_q_rows > 16)
    return record_error(SV_ERR_INVALID, "adjust: max_q_rows %d outside [1, 16]", a->max_q_rows);
  if (a->num_rows < a->batch || a->num_rows > static_cast<int64_t>(a->batch) * a->max_q_rows)
    return record_error(SV_ERR_INVALID, "adjust: num_rows %lld inconsistent with batch %d and max_q_rows %d",
                        static_cast<long long>(a->num_rows), a->batch, a->max_q_rows);
  if (a->repetition != 0.0f && !(a->repetition >= kMinRepetition && a->repetition <= kMaxRepetition))
    return bad("repetition outside [2^-64, 2^64] (0 = off)");
  if (!std::isfinite(a->presence) || !std::isfinite(a->frequency))
    return bad("presence and frequency must be finite");
  if (a->num_ctx < 0 || a->num_ctx > 1024)
    return record_error(SV_ERR_INVALID, "adjust: num_ctx %d outside [0, 1024]", a->num_ctx);
  if (a->ctx_stride < 0) return bad("negative ctx_stride");
  if (a->num_bias < 0 || a->num_bias > kMaxEntries) return bad("num_bias outside [0, 2^30]");
  if (a->num_slots < 0 || a->num_masks < 0) return bad("negative num_slots or num_masks");
  if (a->mask_stride != 0 && a->mask_stride < (a->vocab + 31) / 32)
    return bad("mask_stride below ceil(vocab / 32)");
  if (a->batch == 0) return SV_OK;
  if (!a->cu_q || !a->target || !a->target_out) return bad("null cu_q, target or target_out");
  if ((a->draft == nullptr) != (a->draft_out == nullptr)) return bad("draft without draft_out, or the reverse");
  if (a->draft && (a->draft == a->draft_out) != (a->target == a->target_out))
    return bad("target and draft must both be in place or neither");
  if (!is_aligned16(a->target) || !is_aligned16(a->target_out) || !is_aligned16(a->draft) ||
      !is_aligned16(a->draft_out))
    return bad("logits must be 16-byte aligned");
  if ((a->counts == nullptr) != (a->seen == nullptr)) return bad("counts and seen go together");
  if (a->counts && a->num_slots < 1) return bad("num_slots of a table");
  if (a->num_ctx > 0 && !a->ctx_tokens) return bad("null ctx_tokens");
  if (a->bias_start && a->num_bias > 0 && (!a->bias_tokens || !a->bias_values))
    return bad("null bias_tokens or bias_values");
  if (a->mask && !a->mask_rows && a->num_masks < a->num_rows)
    return bad("num_masks below num_rows without mask_rows");
  return SV_OK;
}

sv_status check_count(const sv_count_args *a) {
  auto bad = [](const char *what) { return record_error(SV_ERR_INVALID, "count: %s", what); };
  if (!a) return bad("null arguments");
  if (a->batch < 0 || a->batch > 65535)
    return record_error(SV_ERR_UNSUPPORTED, "count: batch %d outside [0, 65535]", a->batch);
  if (a->vocab < 1 || a->vocab > (1 << 23))
    return record_error(SV_ERR_UNSUPPORTED, "count: vocab %d outside [1, 2^23]", a->vocab);
  if (a->num_slots < 1) return record_error(SV_ERR_INVALID, "count: num_slots %d", a->num_slots);
  if (a->flags & ~(SV_COUNT_PROMPT | SV_COUNT_RESET))
    return record_error(SV_ERR_INVALID, "count: flags %d", a->flags);
  if (a->num_tokens < 0 || a->num_tokens > kMaxEntries) return bad("num_tokens outside [0, 2^30]");
  if (a->batch == 0) return SV_OK;
  if (!a->start || !a->counts || !a->seen) return bad("null start, counts or seen");
  if (a->num_tokens > 0 && !a->tokens) return bad("null tokens");
  return SV_OK;
}

}  // namespace

}  // namespace sv

extern "C" {

SV_API sv_status spec_adjust_logits(const sv_adjust_args *a, void *stream) {
  using namespace sv;
  const sv_status st = check_adjust(a);
  if (st != SV_OK) return st;
  if (a->batch == 0) return SV_OK;
  AdjustParams P{};
  P.a = *a;
  if (P.a.repetition == 0.0f) P.a.repetition = 1.0f;
  P.seen_words = (a->vocab + 31) / 32;
  P.mask_bytes = 4 * (a->mask_stride ? a->mask_stride : P.seen_words);
  const int sms = device_sms();
  if (sms <= 0) return record_error(SV_ERR_CUDA, "adjust: no current CUDA device");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == SV_BF16 ? launch_adjust<uint16_t>(sms, P, s)
                                            : launch_adjust<float>(sms, P, s);
  if (e != cudaSuccess) return record_error(SV_ERR_CUDA, "adjust launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

SV_API sv_status spec_count_tokens(const sv_count_args *a, void *stream) {
  using namespace sv;
  const sv_status st = check_count(a);
  if (st != SV_OK) return st;
  if (a->batch == 0) return SV_OK;
  CountParams P{};
  P.a = *a;
  P.words = (a->vocab + 31) / 32;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->flags & SV_COUNT_RESET) {
    // For a prompt the slices are as large as a CTA can be (64 prompts of 1024 to
    // 4096 tokens, V = 128256: 8.6 us with 8192 tokens a slice, 7.4 us so; prompts of
    // 100 k tokens 44 us, one alone 29 us, for every slice reads all of its tokens);
    // counts take shared memory (10.0 us for the same tokens).
    auto slices = [&](int threads) { return static_cast<unsigned>((a->vocab + 32 * threads - 1) / (32 * threads)); };
    if (a->flags & SV_COUNT_PROMPT)
      e = launch_behind(reset_kernel<1024, true>, dim3(a->batch, slices(1024)), 1024, 0, s, P);
    else
      e = launch_behind(reset_kernel<256, false>, dim3(a->batch, slices(256)), 256, 0, s, P);
  } else {
    const int64_t threads = a->num_tokens > a->batch ? a->num_tokens : a->batch;
    e = launch_behind(count_kernel, dim3(static_cast<unsigned>((threads + kNT - 1) / kNT)), kNT,
                      a->batch <= kMaxStart ? (a->batch + 1) * 4 : 0, s, P);
  }
  if (e != cudaSuccess) return record_error(SV_ERR_CUDA, "count launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

SV_API int32_t sv_ops_version(void) { return SV_OPS_VERSION; }

SV_API size_t sv_ops_struct_size(int32_t which) {
  return which == 0 ? sizeof(sv_rope_args) : which == 1 ? sizeof(sv_rope_scaling)
         : which == 2 ? sizeof(sv_count_args) : which == 3 ? sizeof(sv_adjust_args) : 0;
}

}  // extern "C"
