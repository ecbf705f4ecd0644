// Penalties, biases and grammar masks on logits rows, and the table of tokens
// that the penalties read (sm_103a).  Contract: spec_adjust_logits and
// spec_count_tokens in include/spec_ops.h.
//
// Adjusting is a copy with exceptions.  The copy (out of place: every row read
// and written once, 2 V elements per row) is what the time goes into; the
// exceptions are few: the tokens of the history, the biased ones and the
// block's drafts, a few thousand of V per sequence, but spread so that most
// warps of a row would meet one.  So they are kept out of the copy: a CTA
// takes a share of the vocabulary for one sequence, copies its part of the
// rows with the masks alone, lists the share's exceptions once (the table's
// bits say where they are, so its counts are read only there), and then works
// the list off for all rows.  In place the copy falls away and only masked
// rows and listed tokens are touched.
//
// A CTA's share is 8 tiles of 256 tokens (one per warp) that lie gridDim.x
// tiles apart, not one run: tokens of small index are the frequent ones, and a
// run of them would give one CTA a list of thousands.
#include <cmath>

#include "common.cuh"
#include "ops_host.inl"
#include "spec_ops.h"

namespace sv {

namespace {

constexpr int kNT = 256;
constexpr int kWarps = kNT / 32;
constexpr int kTile = 256;                 // tokens of one warp
constexpr int kTileWords = kTile / 32;
constexpr int kShare = kWarps * kTile;     // tokens of one CTA
constexpr int kBatch = 4;                  // rows whose vectors are in flight together

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

struct AdjustParams {
  sv_adjust_args a;
  int lines_per_part;            // rows (target, then draft) that one CTA works on
  int64_t mask_bytes;            // bytes per mask row
  int seen_words;
};

// n rows of a sequence, V elements apart: block rows j0 .. of the target's
// logits or of the draft's.
template <typename T>
struct Rows {
  const T *in;
  T *out;
  int n, j0;
  uint32_t index;                // of the first row in its tensor (its alignment)
};

// The kPer bits of tokens t .. of a mask row (token u at bit u % 8 of byte u / 8).
template <int kPer>
__device__ __forceinline__ uint32_t mask_bits(const uint8_t *m, int t, int64_t mask_bytes) {
  const int64_t b = t >> 3;
  uint32_t w = m[b];
  if ((t & 7) + kPer > 8 && b + 1 < mask_bytes) w |= static_cast<uint32_t>(m[b + 1]) << 8;
  return (w >> (t & 7)) & ((1u << kPer) - 1);
}

// One vector of a row: from its mask's bits to its new value.
template <typename T, int kPer>
struct Piece {
  union { uint4 w; T e[kPer]; };
  uint32_t allow;                // all bits: as it is
  __device__ __forceinline__ void bar() {
    if (allow == (1u << kPer) - 1) return;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (!((allow >> k) & 1u)) e[k] = Elem<T>::kNegInf;
  }
};

// RAGGED: V is no multiple of a 16-byte vector's elements, so rows differ in
// alignment: a tile's vectors start at each row's first aligned token, and the
// up to kPer - 1 tokens at either end go one by one.
template <typename T, bool IN_PLACE, bool RAGGED>
__global__ void __launch_bounds__(kNT, 4) adjust_kernel(const __grid_constant__ AdjustParams P) {
  using E = Elem<T>;
  constexpr int kPer = 16 / static_cast<int>(sizeof(T));     // elements of a vector
  constexpr int kVecs = kTile / kPer / 32;                   // vectors per lane and row
  constexpr uint32_t kAll = (1u << kPer) - 1;
  const sv_adjust_args &a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, i = blockIdx.y;
  const int V = a.vocab, shares = gridDim.x;
  const int t0 = (blockIdx.x + warp * shares) * kTile, t1 = min(V, t0 + kTile);   // t1 <= t0: none
  const bool head = blockIdx.x == 0 && blockIdx.z == 0;      // this CTA reports the sequence

  __shared__ uint32_t s_extra[kShare / 32];                  // ctx, draft and bias tokens
  __shared__ int32_t s_mask[16];                             // mask rows of the block rows
  __shared__ int s_n, s_masked;
  __shared__ uint32_t s_tok[kShare];                         // listed token, and above it bit b:
                                                             // draft b + 1 is this token
  __shared__ uint32_t s_word[kShare];                        // its table word, with ctx
  __shared__ float s_bias[kShare];
  __shared__ __align__(16) int32_t s_last[kShare];           // 1 + last bias entry of a token

  const int r0 = a.cu_q[i], Ri = a.cu_q[i + 1] - r0;
  if (r0 < i || Ri < 1 || Ri > a.max_q_rows || r0 + Ri > a.num_rows ||
      r0 + Ri - (i + 1) > a.num_rows - a.batch) {            // (its draft rows, too)
    if (head && tid == 0) set_status(a.dev_status, SV_DEV_BAD_LENGTH);
    return;
  }
  const int lines = Ri + (a.draft != nullptr ? Ri - 1 : 0);  // target rows, then draft rows
  const int l0 = blockIdx.z * P.lines_per_part, l1 = min(lines, l0 + P.lines_per_part);
  if (l0 >= l1) return;
  auto rows_of = [&](const void *in, void *out, int first, int last, int row0) {
    Rows<T> R;
    R.j0 = first;
    R.n = max(last - first, 0);
    R.index = static_cast<uint32_t>(row0 + first);
    const int64_t off = static_cast<int64_t>(row0 + first) * V;
    R.in = static_cast<const T *>(in) + off;
    R.out = static_cast<T *>(out) + off;
    return R;
  };
  const Rows<T> parts[2] = {rows_of(a.target, a.target_out, min(l0, Ri), min(l1, Ri), r0),
                            rows_of(a.draft, a.draft_out, max(l0 - Ri, 0), max(l1 - Ri, 0), r0 - i)};

  // the sequence's values
  const float rep = a.repetitions ? a.repetitions[i] : a.repetition;
  const float pres = a.presences ? a.presences[i] : a.presence;
  const float freq = a.frequencies ? a.frequencies[i] : a.frequency;
  const int slot = a.counts == nullptr ? -1 : a.slots ? a.slots[i] : i;
  int b0 = 0, b1 = 0;
  if (a.bias_start) {
    b0 = a.bias_start[i];
    b1 = a.bias_start[i + 1];
  }
  int bad = !(rep > 0.0f) || !isfinite(rep) || !isfinite(pres) || !isfinite(freq) || slot < -1 ||
            slot >= max(a.num_slots, 0) || b0 < 0 || b1 < b0 || b1 > a.num_bias;
  if (warp == 0) {
    int m = -1;
    if (a.mask && lane < Ri) {
      m = a.mask_rows ? a.mask_rows[r0 + lane] : r0 + lane;
      bad |= m < -1 || m >= a.num_masks;
    }
    if (lane < 16) s_mask[lane] = m;
    const uint32_t masked = __ballot_sync(0xffffffffu, m >= 0);
    if (lane == 0) {
      s_masked = static_cast<int>(masked);
      s_n = 0;
    }
  }
  if (tid < kShare / 32) s_extra[tid] = 0;
  const int nb = b1 - b0;
  if (nb > 0)
    for (int t = tid; t < kShare / 4; t += kNT)
      reinterpret_cast<int4 *>(s_last)[t] = make_int4(0, 0, 0, 0);
  bad = __syncthreads_or(bad);

  if (bad) {                      // rows the sampler fails the sequence on
    if (head && tid == 0) set_status(a.dev_status, SV_DEV_BAD_PARAM);
    for (const Rows<T> &R : parts)
      for (int r = 0; r < R.n; ++r)
        for (int t = t0 + lane; t < t1; t += 32) R.out[static_cast<int64_t>(r) * V + t] = E::put(NAN);
    return;
  }

  const bool penal = rep != 1.0f || pres != 0.0f || freq != 0.0f;
  const int drafts = penal && a.draft_tokens ? Ri - 1 : 0;
  const int32_t *draft_tokens = a.draft_tokens + (r0 - i);
  const int64_t ctx_stride = a.ctx_stride ? a.ctx_stride : a.batch;

  // the table's bits of this warp's tile: word q in lane q
  uint32_t known = 0;
  if (penal && slot >= 0 && lane < kTileWords && t0 + lane * 32 < t1)
    known = a.seen[static_cast<int64_t>(slot) * P.seen_words + (t0 >> 5) + lane];

  // tokens outside the table: index in the share, or -1
  auto local_of = [&](int t) {
    if (t < 0 || t >= V) return -1;
    const int tile = t / kTile, w = tile / shares;
    return tile - w * shares == static_cast<int>(blockIdx.x) ? w * kTile + t % kTile : -1;
  };
  auto mark = [&](int local) { atomicOr(&s_extra[local >> 5], 1u << (local & 31)); };
  if (tid < drafts) {
    const int local = local_of(draft_tokens[tid]);
    if (local >= 0) mark(local);
  }
  if (penal)
    for (int c = tid; c < a.num_ctx; c += kNT) {
      const int local = local_of(a.ctx_tokens[c * ctx_stride + i]);
      if (local >= 0) mark(local);
    }
  for (int e = tid; e < nb; e += kNT) {
    const int t = a.bias_tokens[b0 + e], local = local_of(t);
    if (local >= 0) {
      mark(local);
      atomicMax(&s_last[local], e + 1);
    } else if (head && (t < 0 || t >= V)) {
      set_status(a.dev_status, SV_DEV_BAD_TOKEN);
    }
  }

  // the copy of up to kBatch rows, loads before stores; row r of R, its mask m
  const uint8_t *masks = reinterpret_cast<const uint8_t *>(a.mask);
  const uint32_t masked = static_cast<uint32_t>(s_masked);
  auto copy = [&](const Rows<T> &R, const int (&row)[kBatch], int n) {
    Piece<T, kPer> x[kBatch][kVecs];
    T edge[kBatch];
    int edge_at[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (u >= n) break;
      const T *in = R.in + static_cast<int64_t>(row[u]) * V;
      const int m = masked ? s_mask[R.j0 + row[u]] : -1;
      const uint8_t *bits = masks + m * P.mask_bytes;
      const int mis = RAGGED ? ((R.index + row[u]) * static_cast<uint32_t>(V)) & (kPer - 1) : 0;
      const int first = RAGGED ? min(t1, t0 + ((kPer - mis) & (kPer - 1))) : t0;
#pragma unroll
      for (int q = 0; q < kVecs; ++q) {
        const int t = first + (lane + q * 32) * kPer;
        x[u][q].allow = kAll;
        if (t + kPer > t1) continue;
        if (m >= 0) x[u][q].allow = mask_bits<kPer>(bits, t, P.mask_bytes);
        if (x[u][q].allow != 0 && !(IN_PLACE && x[u][q].allow == kAll))
          x[u][q].w = *reinterpret_cast<const uint4 *>(in + t);
      }
      if constexpr (RAGGED) {
        const int tail = first + ((t1 - first) & ~(kPer - 1));
        int t = lane < 16 ? (t0 + lane < first ? t0 + lane : -1)
                          : (tail + lane - 16 < t1 ? tail + lane - 16 : -1);
        if (t >= 0) {
          const bool allowed = m < 0 || ((bits[t >> 3] >> (t & 7)) & 1u);
          if (!allowed) edge[u] = E::kNegInf;
          else if (IN_PLACE) t = -1;
          else edge[u] = in[t];
        }
        edge_at[u] = t;
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (u >= n) break;
      T *out = R.out + static_cast<int64_t>(row[u]) * V;
      const int mis = RAGGED ? ((R.index + row[u]) * static_cast<uint32_t>(V)) & (kPer - 1) : 0;
      const int first = RAGGED ? min(t1, t0 + ((kPer - mis) & (kPer - 1))) : t0;
#pragma unroll
      for (int q = 0; q < kVecs; ++q) {
        const int t = first + (lane + q * 32) * kPer;
        if (t + kPer > t1 || (IN_PLACE && x[u][q].allow == kAll)) continue;
        x[u][q].bar();
        *reinterpret_cast<uint4 *>(out + t) = x[u][q].w;
      }
      if constexpr (RAGGED) {
        if (edge_at[u] >= 0) out[edge_at[u]] = edge[u];
      }
    }
  };
  if (t0 < t1 && !(IN_PLACE && masked == 0)) {
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const Rows<T> &R = parts[kind];
      if constexpr (IN_PLACE) {              // the masked rows alone
        uint32_t left = R.n > 0 ? (masked >> R.j0) & ((1u << R.n) - 1) : 0u;
        while (left) {
          int row[kBatch] = {0, 0, 0, 0}, n = 0;
#pragma unroll
          for (int u = 0; u < kBatch; ++u)
            if (left) {
              row[u] = __ffs(left) - 1;
              left &= left - 1;
              n = u + 1;
            }
          copy(R, row, n);
        }
      } else {
        for (int r = 0; r < R.n; r += kBatch) {
          const int row[kBatch] = {r, r + 1, r + 2, r + 3};
          copy(R, row, R.n - r);
        }
      }
    }
  }
  __syncthreads();

  // the list: lane b has bit b of the tile's words
  if (t0 < t1) {
    uint32_t any[kTileWords];
    int count = 0;
#pragma unroll
    for (int q = 0; q < kTileWords; ++q) {
      any[q] = __shfl_sync(0xffffffffu, known, q) | s_extra[warp * kTileWords + q];
      if (t1 - t0 - q * 32 < 32) any[q] &= t1 - t0 > q * 32 ? (1u << (t1 - t0 - q * 32)) - 1 : 0u;
      count += __popc(any[q]);
    }
    if (count) {
      int at = 0;
      if (lane == 0) at = atomicAdd(&s_n, count);
      at = __shfl_sync(0xffffffffu, at, 0);
      const int32_t *counts = a.counts + static_cast<int64_t>(slot) * V + t0;
#pragma unroll
      for (int q = 0; q < kTileWords; ++q) {
        if (any[q] == 0) continue;
        const uint32_t kw = __shfl_sync(0xffffffffu, known, q);
        if ((any[q] >> lane) & 1u) {
          const int in_tile = q * 32 + lane, local = warp * kTile + in_tile, t = t0 + in_tile;
          uint32_t word = 0, after = 0;
          float bias = 0.0f;
          if ((kw >> lane) & 1u) word = static_cast<uint32_t>(counts[in_tile]);
          if ((s_extra[warp * kTileWords + q] >> lane) & 1u) {
            if (penal)
              for (int c = 0; c < a.num_ctx; ++c) word += a.ctx_tokens[c * ctx_stride + i] == t;
            for (int d = 0; d < drafts; ++d)
              if (draft_tokens[d] == t) after |= 1u << d;
            if (nb > 0 && s_last[local]) bias = a.bias_values[b0 + s_last[local] - 1];
          }
          const int e = at + __popc(any[q] & ((1u << lane) - 1));
          s_tok[e] = static_cast<uint32_t>(local) | (after << 16);
          s_word[e] = word;
          s_bias[e] = bias;
        }
        at += __popc(any[q]);
      }
    }
  }
  __syncthreads();

  // the list for every row: threads share the entries, and the rows too where
  // the entries are fewer than threads
  const int n = s_n;
  int span = kNT;                                            // threads that share the entries
  while (span > 32 && n <= span / 2) span >>= 1;
  const int step = kNT / span, group = tid / span;
  for (int e = tid & (span - 1); e < n; e += span) {
    const uint32_t tok = s_tok[e], word = s_word[e], after = tok >> 16;
    const int local = tok & 0xFFFFu;
    const int t = (blockIdx.x + (local / kTile) * shares) * kTile + local % kTile;
    const float bias = s_bias[e];
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const Rows<T> &R = parts[kind];
      for (int rb = group; rb < R.n; rb += step * kBatch) {
        T x[kBatch];
        bool allowed[kBatch];
        const int64_t off = static_cast<int64_t>(rb) * V + t, next = static_cast<int64_t>(step) * V;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (rb + u * step >= R.n) break;
          x[u] = R.in[off + u * next];
          allowed[u] = true;
          if (masked) {
            const int m = s_mask[R.j0 + rb + u * step];
            if (m >= 0) allowed[u] = (masks[m * P.mask_bytes + (t >> 3)] >> (t & 7)) & 1u;
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (rb + u * step >= R.n) break;
          if (!allowed[u]) continue;                         // written already
          const uint32_t times = (word & 0x7FFFFFFFu) +
                                 __popc(after & ((1u << (R.j0 + rb + u * step)) - 1));
          float y = E::get(x[u]);
          if (times > 0 || (word >> 31)) y = y > 0.0f ? y / rep : y * rep;
          if (times > 0) y -= fmaf(freq, static_cast<float>(times), pres);
          if (bias != 0.0f) y += bias;
          R.out[off + u * next] = E::put(y);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- count
struct CountParams {
  sv_count_args a;
  int words;                      // of a slot's bits
};

// Clears the batch's slots: the counts that the bits point at, then the bits.
__global__ void __launch_bounds__(kNT) clear_kernel(const __grid_constant__ CountParams P) {
  const sv_count_args &a = P.a;
  const int i = blockIdx.y;
  const int slot = a.slots ? a.slots[i] : i;
  if (slot < 0 || slot >= a.num_slots) return;                // reported by count_kernel
  const int w = blockIdx.x * kNT + threadIdx.x;
  if (w >= P.words) return;
  uint32_t *seen = a.seen + static_cast<int64_t>(slot) * P.words + w;
  uint32_t bits = *seen;
  if (bits == 0) return;
  int32_t *counts = a.counts + static_cast<int64_t>(slot) * a.vocab + w * 32;
  while (bits) {
    const int b = __ffs(bits) - 1;
    bits &= bits - 1;
    if (w * 32 + b < a.vocab) counts[b] = 0;
  }
  *seen = 0;
}

__global__ void __launch_bounds__(kNT) count_kernel(const __grid_constant__ CountParams P) {
  const sv_count_args &a = P.a;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kNT + threadIdx.x;
  if (at < a.batch) {             // one thread per sequence reports
    const int i = static_cast<int>(at);
    const int s0 = a.start[i], s1 = a.start[i + 1], slot = a.slots ? a.slots[i] : i;
    if (s0 < 0 || s1 < s0 || s1 > a.num_tokens) set_status(a.dev_status, SV_DEV_BAD_LENGTH);
    if (slot < -1 || slot >= a.num_slots) set_status(a.dev_status, SV_DEV_BAD_PARAM);
  }
  if (at >= a.num_tokens) return;
  // the last sequence that starts at or before this token
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.start[mid] <= at) lo = mid; else hi = mid;
  }
  const int i = lo, s0 = a.start[i], s1 = a.start[i + 1];
  if (s0 < 0 || at < s0 || at >= s1 || s1 > a.num_tokens) return;
  if (a.num_accepted && at - s0 > a.num_accepted[i]) return;
  const int slot = a.slots ? a.slots[i] : i;
  if (slot < 0 || slot >= a.num_slots) return;
  const int t = a.tokens[at];
  if (t < 0 || t >= a.vocab) {
    set_status(a.dev_status, SV_DEV_BAD_TOKEN);
    return;
  }
  uint32_t *word = reinterpret_cast<uint32_t *>(a.counts) + static_cast<int64_t>(slot) * a.vocab + t;
  if (a.flags & SV_COUNT_PROMPT) {
    if (!(__ldcg(word) >> 31)) atomicOr(word, 0x80000000u);
  } else {
    atomicAdd(word, 1u);
  }
  uint32_t *seen = a.seen + static_cast<int64_t>(slot) * P.words + (t >> 5);
  const uint32_t bit = 1u << (t & 31);
  if (!(__ldcg(seen) & bit)) atomicOr(seen, bit);
}

// ---------------------------------------------------------------- host side
template <typename T>
void launch_adjust(bool in_place, dim3 grid, const AdjustParams &P, cudaStream_t s) {
  const bool ragged = P.a.vocab % (16 / static_cast<int>(sizeof(T))) != 0;
  if (in_place) {
    if (ragged) adjust_kernel<T, true, true><<<grid, kNT, 0, s>>>(P);
    else adjust_kernel<T, true, false><<<grid, kNT, 0, s>>>(P);
  } else {
    if (ragged) adjust_kernel<T, false, true><<<grid, kNT, 0, s>>>(P);
    else adjust_kernel<T, false, false><<<grid, kNT, 0, s>>>(P);
  }
}

sv_status check_adjust(const sv_adjust_args *a) {
  auto bad = [](const char *what) { return record_error(SV_ERR_INVALID, "adjust: %s", what); };
  if (!a) return bad("null arguments");
  if (a->batch < 0 || a->batch > 65535)
    return record_error(SV_ERR_UNSUPPORTED, "adjust: batch %d outside [0, 65535]", a->batch);
  if (a->vocab < 1 || a->vocab > (1 << 30))
    return record_error(SV_ERR_INVALID, "adjust: vocab %d", a->vocab);
  if (a->dtype != SV_F32 && a->dtype != SV_BF16)
    return record_error(SV_ERR_INVALID, "adjust: dtype %d", a->dtype);
  if (a->max_q_rows < 1 || a->max_q_rows > 16)
    return record_error(SV_ERR_INVALID, "adjust: max_q_rows %d outside [1, 16]", a->max_q_rows);
  if (a->num_rows < a->batch || a->num_rows > static_cast<int64_t>(a->batch) * a->max_q_rows)
    return record_error(SV_ERR_INVALID, "adjust: num_rows %lld inconsistent with batch %d and max_q_rows %d",
                        static_cast<long long>(a->num_rows), a->batch, a->max_q_rows);
  if (!std::isfinite(a->repetition) || a->repetition < 0.0f)
    return bad("repetition must be finite and > 0 (0 = off)");
  if (!std::isfinite(a->presence) || !std::isfinite(a->frequency))
    return bad("presence and frequency must be finite");
  if (a->num_ctx < 0 || a->num_ctx > 1024)
    return record_error(SV_ERR_INVALID, "adjust: num_ctx %d outside [0, 1024]", a->num_ctx);
  if (a->ctx_stride < 0) return bad("negative ctx_stride");
  if (a->num_bias < 0 || a->num_bias >= (int64_t{1} << 31)) return bad("num_bias outside [0, 2^31)");
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
  if (a->vocab < 1 || a->vocab > (1 << 30))
    return record_error(SV_ERR_INVALID, "count: vocab %d", a->vocab);
  if (a->num_slots < 1) return record_error(SV_ERR_INVALID, "count: num_slots %d", a->num_slots);
  if (a->flags & ~(SV_COUNT_PROMPT | SV_COUNT_RESET))
    return record_error(SV_ERR_INVALID, "count: flags %d", a->flags);
  if (a->num_tokens < 0 || a->num_tokens >= (int64_t{1} << 31)) return bad("num_tokens outside [0, 2^31)");
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
  const int tiles = (a->vocab + kTile - 1) / kTile, shares = (tiles + kWarps - 1) / kWarps;
  const int lines = a->draft ? 2 * a->max_q_rows - 1 : a->max_q_rows;
  // Few CTAs: the rows are split as well, down to one batch of rows per CTA
  // (each part repeats the list).
  const int sms = device_sms();
  if (sms <= 0) return record_error(SV_ERR_CUDA, "adjust: no current CUDA device");
  const int64_t ctas = static_cast<int64_t>(shares) * a->batch;
  int parts = 1;
  while (parts * kBatch < lines && ctas * (parts + 1) <= 4 * static_cast<int64_t>(sms)) ++parts;
  P.lines_per_part = (lines + parts - 1) / parts;
  const dim3 grid(shares, a->batch, (lines + P.lines_per_part - 1) / P.lines_per_part);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool in_place = a->target == a->target_out;
  if (a->dtype == SV_BF16) launch_adjust<uint16_t>(in_place, grid, P, s);
  else launch_adjust<float>(in_place, grid, P, s);
  const cudaError_t e = cudaGetLastError();
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
  if (a->flags & SV_COUNT_RESET)
    clear_kernel<<<dim3((P.words + kNT - 1) / kNT, a->batch), kNT, 0, s>>>(P);
  const int64_t threads = a->num_tokens > a->batch ? a->num_tokens : a->batch;
  count_kernel<<<static_cast<unsigned>((threads + kNT - 1) / kNT), kNT, 0, s>>>(P);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return record_error(SV_ERR_CUDA, "count launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

SV_API int32_t sv_ops_version(void) { return SV_OPS_VERSION; }

SV_API size_t sv_ops_struct_size(int32_t which) {
  return which == 0 ? sizeof(sv_rope_args) : which == 1 ? sizeof(sv_rope_scaling)
         : which == 2 ? sizeof(sv_count_args) : which == 3 ? sizeof(sv_adjust_args) : 0;
}

}  // extern "C"
