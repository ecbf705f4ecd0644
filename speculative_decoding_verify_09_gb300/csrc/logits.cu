// Penalties, biases and grammar masks on logits rows, and the table of tokens
// that the penalties read (sm_103a).  Contract: spec_adjust_logits and
// spec_count_tokens in include/spec_ops.h.
//
// Adjusting is a copy with exceptions.  The copy (out of place: every row read
// and written once, 2 V elements per row) is what the time goes into; the
// exceptions are few: the tokens of the history, the biased ones and the
// block's drafts, a few thousand of V per sequence, but spread so that most
// 512-byte pieces of a row hold one.  What has to stay small is the number of
// instructions per byte.  A CTA takes a chunk of the vocabulary (4 KB of a row)
// for one sequence and lists the chunk's exceptions once: the table's bits say
// where they are, so its counts are read only there.  From then on every warp
// works alone, a row's chunk at a time: 16-byte cp.async copies into a ring of
// shared memory (kRing rows deep), the listed tokens changed there, a lane per
// token, and the chunk written out.  In place nothing streams: masked rows are
// written where a token is barred, and the listed tokens of every row are
// changed in global memory.
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "ops_host.inl"
#include "spec_ops.h"

namespace sv {

namespace {

constexpr int kNT = 256;                   // threads of the table's kernels
constexpr int kWarps = 4;                  // of an adjusting CTA
constexpr int kThreads = kWarps * 32;
constexpr int kChunkBytes = 4096;          // of a row, per CTA
constexpr int kRing = 2;                   // row chunks in flight per warp
constexpr int kBatch = 4;                  // (in place) rows in flight per warp

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

// A row that the CTA works on, at the chunk's first token.
template <typename T>
struct alignas(16) Line {
  const T *in;
  T *out;
  const uint8_t *mask;           // the row's mask from the chunk's first token on, or null
  int j, mis;                    // block row; elements from the 16-byte boundary before it
};

template <typename T>
struct Chunk {
  static constexpr int kPer = 16 / static_cast<int>(sizeof(T));       // elements of a vector
  static constexpr int kTokens = kChunkBytes / static_cast<int>(sizeof(T));
  static constexpr int kWords = kTokens / 32;
  static constexpr int kVecs = kChunkBytes / 16 / 32;                 // vectors per lane
  static constexpr int kMaskAt = kChunkBytes + 16;                    // (a misaligned row's last vector)
  static constexpr int kSlot = kMaskAt + kWords * 4;                  // a row in the ring, its mask
  static_assert(kSlot % 16 == 0, "vectors of every slot are 16-byte aligned");
};

constexpr uint16_t kOutside = 0x8000u, kBiased = 0x4000u;   // flags of a listed token: counted
                                                            // outside the table, has a bias

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}

// RAGGED: V is no multiple of a vector's elements, so rows differ in alignment.
template <typename T, bool IN_PLACE, bool RAGGED>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const __grid_constant__ AdjustParams P) {
  using E = Elem<T>;
  using C = Chunk<T>;
  constexpr int kPer = C::kPer;
  constexpr uint32_t kAll = (1u << kPer) - 1;
  const sv_adjust_args &a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, i = blockIdx.y;
  const int V = a.vocab, t0 = blockIdx.x * C::kTokens, width = min(V - t0, C::kTokens);
  const bool head = blockIdx.x == 0 && blockIdx.z == 0;      // this CTA reports the sequence

  extern __shared__ __align__(16) unsigned char s_ring[];    // (out of place) kWarps x kRing slots
  __shared__ Line<T> s_line[32];                             // target rows, then draft rows
  __shared__ uint32_t s_extra[C::kWords];                    // bits of ctx, draft and bias tokens
  __shared__ __align__(16) int32_t s_last[C::kTokens];       // 1 + last bias entry of a token; then
                                                             // its bias, as bits
  __shared__ uint32_t s_word[C::kTokens];                    // table words of the list, with ctx
  __shared__ uint16_t s_tok[C::kTokens];                     // the list: tokens in the chunk, flags
  __shared__ int32_t s_draft[16];                            // the block's drafts in the chunk
  __shared__ int s_n;

  const int r0 = a.cu_q[i], Ri = a.cu_q[i + 1] - r0;
  if (r0 < i || Ri < 1 || Ri > a.max_q_rows || r0 + Ri > a.num_rows ||
      r0 + Ri - (i + 1) > a.num_rows - a.batch) {            // (its draft rows, too)
    if (head && tid == 0) set_status(a.dev_status, SV_DEV_BAD_LENGTH);
    return;
  }
  const int all = Ri + (a.draft != nullptr ? Ri - 1 : 0);
  const int l0 = blockIdx.z * P.lines_per_part, lines = min(all - l0, P.lines_per_part);
  if (lines <= 0) return;

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
  const int nb = b1 - b0;
  if (tid < Ri && a.mask) {                                  // every row's, for one verdict
    const int m = a.mask_rows ? a.mask_rows[r0 + tid] : r0 + tid;
    bad |= m < -1 || m >= a.num_masks;
  }
  if (tid < lines) {
    const int l = l0 + tid;
    Line<T> L;
    L.j = l < Ri ? l : l - Ri;
    const int64_t row = l < Ri ? r0 + l : r0 - i + L.j;
    L.in = static_cast<const T *>(l < Ri ? a.target : a.draft) + row * V + t0;
    L.out = static_cast<T *>(l < Ri ? a.target_out : a.draft_out) + row * V + t0;
    L.mis = RAGGED ? static_cast<int>((static_cast<uint32_t>(row) * static_cast<uint32_t>(V)) & (kPer - 1)) : 0;
    L.mask = nullptr;
    if (a.mask) {
      const int m = a.mask_rows ? a.mask_rows[r0 + L.j] : r0 + L.j;
      if (m >= 0) L.mask = reinterpret_cast<const uint8_t *>(a.mask) + m * P.mask_bytes + (t0 >> 3);
    }
    s_line[tid] = L;
  }
  if (tid < C::kWords) s_extra[tid] = 0;
  if (tid == 0) s_n = 0;
  if (nb > 0)
    for (int t = tid; t < C::kTokens / 4; t += kThreads)
      reinterpret_cast<int4 *>(s_last)[t] = make_int4(0, 0, 0, 0);
  bad = __syncthreads_or(bad);

  if (bad) {                      // rows the sampler fails the sequence on
    if (head && tid == 0) set_status(a.dev_status, SV_DEV_BAD_PARAM);
    for (int l = warp; l < lines; l += kWarps)
      for (int t = lane; t < width; t += 32) s_line[l].out[t] = E::put(NAN);
    return;
  }

  // Row chunk `line` into its slot of this warp's ring: 16-byte vectors from
  // the boundary at or before the chunk's first token up to its last one, and
  // the chunk's mask words.
  unsigned char *my_ring = s_ring + warp * (kRing * C::kSlot);
  auto issue = [&](int line, int s) {
    if (line < lines) {
      const Line<T> L = s_line[line];
      const uint32_t dst = smem_u32(my_ring + s * C::kSlot) + lane * 16;
      const T *src = L.in - L.mis + lane * kPer;
      const int left = width + L.mis - lane * kPer;          // elements from this lane's first on
#pragma unroll
      for (int q = 0; q < C::kVecs; ++q)
        if (left > q * 32 * kPer)
          cp_async16(dst + q * 512, src + q * 32 * kPer,
                     min(16, (left - q * 32 * kPer) * static_cast<int>(sizeof(T))));
      if (RAGGED && lane == 0 && left > C::kTokens)
        cp_async16(dst + kChunkBytes, src + C::kTokens, (left - C::kTokens) * static_cast<int>(sizeof(T)));
      if (L.mask)
        for (int w = lane; w * 32 < width; w += 32)
          cp_async4(smem_u32(my_ring + s * C::kSlot + C::kMaskAt) + w * 4, L.mask + w * 4);
    }
    cp_async_commit();
  };
  if constexpr (!IN_PLACE)
    for (int s = 0; s < kRing; ++s) issue(warp + s * kWarps, s);

  const bool penal = rep != 1.0f || pres != 0.0f || freq != 0.0f;
  const int drafts = penal && a.draft_tokens ? Ri - 1 : 0;
  const int ctx = penal ? a.num_ctx : 0;
  const int64_t ctx_stride = a.ctx_stride ? a.ctx_stride : a.batch;

  // the table's bits of the chunk: a word per thread
  uint32_t known = 0;
  if (penal && slot >= 0 && tid < C::kWords && tid * 32 < width)
    known = a.seen[static_cast<int64_t>(slot) * P.seen_words + (t0 >> 5) + tid];
  static_assert(C::kWords <= kThreads, "a word per thread");

  // tokens outside the table
  auto mark = [&](int t) { atomicOr(&s_extra[t >> 5], 1u << (t & 31)); };
  auto in_chunk = [&](int token) { return token >= t0 && token - t0 < width; };
  if (tid < drafts) {
    const int t = a.draft_tokens[r0 - i + tid];
    s_draft[tid] = in_chunk(t) ? t - t0 : -1;
    if (in_chunk(t)) mark(t - t0);
  }
  for (int c = tid; c < ctx; c += kThreads) {
    const int t = a.ctx_tokens[c * ctx_stride + i];
    if (in_chunk(t)) mark(t - t0);
  }
  for (int e = tid; e < nb; e += kThreads) {
    const int t = a.bias_tokens[b0 + e];
    if (in_chunk(t)) {
      mark(t - t0);
      atomicMax(&s_last[t - t0], e + 1);
    } else if (head && (t < 0 || t >= V)) {
      set_status(a.dev_status, SV_DEV_BAD_TOKEN);
    }
  }
  __syncthreads();

  // the list: every thread its word's tokens
  if (tid < C::kWords && tid * 32 < width) {
    const uint32_t extra = s_extra[tid];
    uint32_t any = known | extra;
    if (width - tid * 32 < 32) any &= (1u << (width - tid * 32)) - 1;
    int e = any ? atomicAdd(&s_n, __popc(any)) : 0;
    while (any) {
      const int b = __ffs(any) - 1;
      any &= any - 1;
      s_word[e] = (known >> b) & 1u;                         // read below
      s_tok[e++] = static_cast<uint16_t>(tid * 32 + b) | (((extra >> b) & 1u) ? kOutside : 0);
    }
  }
  __syncthreads();
  const int n = s_n;
  for (int e = tid; e < n; e += kThreads) {
    const int tok = s_tok[e], t = tok & (C::kTokens - 1);
    uint32_t word = 0;
    if (s_word[e]) word = static_cast<uint32_t>(a.counts[static_cast<int64_t>(slot) * V + t0 + t]);
    if (tok & kOutside) {
      for (int c = 0; c < ctx; ++c) word += a.ctx_tokens[c * ctx_stride + i] == t0 + t;
      if (nb > 0 && s_last[t]) {
        s_last[t] = __float_as_int(a.bias_values[b0 + s_last[t] - 1]);
        s_tok[e] = static_cast<uint16_t>(tok | kBiased);
      }
    }
    s_word[e] = word;
  }
  __syncthreads();

  auto changed = [&](T x, int tok, uint32_t word, int j) {
    uint32_t times = word & 0x7FFFFFFFu;
    if (tok & kOutside)
      for (int d = 0; d < min(j, drafts); ++d) times += s_draft[d] == (tok & (C::kTokens - 1));
    float y = E::get(x);
    if (times > 0 || (word >> 31)) y = y > 0.0f ? y / rep : y * rep;
    if (times > 0) y -= fmaf(freq, static_cast<float>(times), pres);
    if (tok & kBiased) y += __int_as_float(s_last[tok & (C::kTokens - 1)]);
    return E::put(y);
  };

  if constexpr (!IN_PLACE) {
    int s = 0;
    for (int line = warp; line < lines; line += kWarps) {
      cp_async_wait<kRing - 1>();
      __syncwarp();
      const Line<T> L = s_line[line];
      unsigned char *row = my_ring + s * C::kSlot;
      T *x = reinterpret_cast<T *>(row) + L.mis;             // the chunk's tokens
      for (int e = lane; e < n; e += 32) {
        const int tok = s_tok[e], t = tok & (C::kTokens - 1);
        x[t] = changed(x[t], tok, s_word[e], L.j);
      }
      __syncwarp();
      const uint8_t *bits = row + C::kMaskAt;
      T *out = L.out - L.mis;                                // vectors as they were read
      if (width == C::kTokens && L.mis == 0) {
#pragma unroll
        for (int q = 0; q < C::kVecs; ++q) {
          const int v = (lane + q * 32) * kPer;
          Piece<T, kPer> piece;
          piece.w = *reinterpret_cast<const uint4 *>(row + (lane + q * 32) * 16);
          if (L.mask) piece.bar(mask_bits<kPer>(bits, v, C::kWords * 4));
          *reinterpret_cast<uint4 *>(out + v) = piece.w;
        }
      } else {
        for (int v = lane * kPer; v - L.mis < width; v += 32 * kPer) {
          const int t = v - L.mis;
          Piece<T, kPer> piece;
          piece.w = *reinterpret_cast<const uint4 *>(row + v * static_cast<int>(sizeof(T)));
          uint32_t allow = kAll;                             // bits past the chunk say nothing
          if (L.mask) allow = t >= 0 ? mask_bits<kPer>(bits, t, C::kWords * 4)
                                     : mask_bits<kPer>(bits, 0, C::kWords * 4) << -t;
          piece.bar(allow);
          if (t >= 0 && t + kPer <= width) {
            *reinterpret_cast<uint4 *>(out + v) = piece.w;
          } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
              if (t + k >= 0 && t + k < width) out[v + k] = piece.e[k];
          }
        }
      }
      __syncwarp();                                          // the slot is free
      issue(line + kRing * kWarps, s);
      s = s + 1 == kRing ? 0 : s + 1;
    }
  } else {
    // masked rows: barred tokens written, vectors that stay whole not touched
    for (int line = warp; line < lines; line += kWarps) {
      const Line<T> L = s_line[line];
      if (!L.mask) continue;
      const int first = RAGGED ? (kPer - L.mis) & (kPer - 1) : 0;
      Piece<T, kPer> x[C::kVecs];
      uint32_t allow[C::kVecs];
#pragma unroll
      for (int q = 0; q < C::kVecs; ++q) {
        const int t = first + (lane + q * 32) * kPer;
        allow[q] = t + kPer <= width ? mask_bits<kPer>(L.mask, t, (width + 7) >> 3) : kAll;
      }
#pragma unroll
      for (int q = 0; q < C::kVecs; ++q)
        if (allow[q] != 0 && allow[q] != kAll)
          x[q].w = *reinterpret_cast<const uint4 *>(L.in + first + (lane + q * 32) * kPer);
#pragma unroll
      for (int q = 0; q < C::kVecs; ++q)
        if (allow[q] != kAll) {
          x[q].bar(allow[q]);
          *reinterpret_cast<uint4 *>(L.out + first + (lane + q * 32) * kPer) = x[q].w;
        }
      if (RAGGED || width != C::kTokens) {                   // the ends, one by one
        const int tail = first + (width > first ? (width - first) & ~(kPer - 1) : 0);
        const int t = lane < 16 ? (lane < min(first, width) ? lane : -1)
                                : (tail + lane - 16 < width ? tail + lane - 16 : -1);
        if (t >= 0 && !((L.mask[t >> 3] >> (t & 7)) & 1u)) L.out[t] = E::kNegInf;
      }
    }
    __syncwarp();
    // the listed tokens of this warp's rows
    for (int e = lane; e < n; e += 32) {
      const int tok = s_tok[e], t = tok & (C::kTokens - 1);
      const uint32_t word = s_word[e];
      for (int lb = warp; lb < lines; lb += kBatch * kWarps) {
        T x[kBatch];
        bool allowed[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          allowed[u] = false;                                // (barred: written already)
          if (lb + u * kWarps >= lines) continue;
          const Line<T> &L = s_line[lb + u * kWarps];
          x[u] = L.in[t];
          allowed[u] = !L.mask || ((L.mask[t >> 3] >> (t & 7)) & 1u);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (allowed[u]) {
            const Line<T> &L = s_line[lb + u * kWarps];
            L.out[t] = changed(x[u], tok, word, L.j);
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
template <typename T, bool IN_PLACE, bool RAGGED>
cudaError_t launch_adjust(dim3 grid, const AdjustParams &P, cudaStream_t s) {
  constexpr int ring = IN_PLACE ? 0 : kWarps * kRing * Chunk<T>::kSlot;
  if constexpr (!IN_PLACE) {      // once per device: the ring and the lists pass 48 KB
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) & bit)) {
      e = cudaFuncSetAttribute(adjust_kernel<T, IN_PLACE, RAGGED>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
      if (e != cudaSuccess) return e;
      ready.fetch_or(bit, std::memory_order_release);
    }
  }
  adjust_kernel<T, IN_PLACE, RAGGED><<<grid, kThreads, ring, s>>>(P);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_adjust(bool in_place, dim3 grid, const AdjustParams &P, cudaStream_t s) {
  const bool ragged = P.a.vocab % Chunk<T>::kPer != 0;
  if (in_place)
    return ragged ? launch_adjust<T, true, true>(grid, P, s) : launch_adjust<T, true, false>(grid, P, s);
  return ragged ? launch_adjust<T, false, true>(grid, P, s) : launch_adjust<T, false, false>(grid, P, s);
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
  const int chunk = a->dtype == SV_BF16 ? Chunk<uint16_t>::kTokens : Chunk<float>::kTokens;
  const int chunks = (a->vocab + chunk - 1) / chunk;
  const int lines = a->draft ? 2 * a->max_q_rows - 1 : a->max_q_rows;
  // Few CTAs: the rows are split as well, down to a row per warp (each part
  // repeats the list).
  const int sms = device_sms();
  if (sms <= 0) return record_error(SV_ERR_CUDA, "adjust: no current CUDA device");
  const int64_t ctas = static_cast<int64_t>(chunks) * a->batch;
  int parts = 1;
  while (parts * kWarps < lines && ctas * (parts + 1) <= 4 * static_cast<int64_t>(sms)) ++parts;
  P.lines_per_part = (lines + parts - 1) / parts;
  const dim3 grid(chunks, a->batch, (lines + P.lines_per_part - 1) / P.lines_per_part);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool in_place = a->target == a->target_out;
  const cudaError_t e = a->dtype == SV_BF16 ? launch_adjust<uint16_t>(in_place, grid, P, s)
                                            : launch_adjust<float>(in_place, grid, P, s);
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
