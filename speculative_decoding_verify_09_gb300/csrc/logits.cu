// Penalties, biases and grammar masks on logits rows, and the table of tokens
// that the penalties read (sm_103a).  Contract: spec_adjust_logits and
// spec_count_tokens in include/spec_ops.h.
//
// Adjusting is a copy with exceptions.  The copy (out of place: every row read
// and written once, 2 V elements per row) is what the time goes into; the
// exceptions are few: the tokens of the history, the biased ones and the
// block's drafts, a few thousand of V per sequence, but spread so that most
// warps of a row would meet one.  So they are kept out of the copy: a CTA
// takes a chunk of the vocabulary for one sequence, copies its part of the
// rows with the masks alone, lists the chunk's exceptions once (the table's
// bits say where they are, so its counts are read only there), and then works
// the list off for all rows, one (row, token) per thread.  In place the copy
// falls away and only masked rows and listed tokens are touched.
#include <cmath>

#include "common.cuh"
#include "ops_host.inl"
#include "spec_ops.h"

namespace sv {

namespace {

constexpr int kNT = 256;
constexpr int kChunk = 2048;               // tokens of one CTA
constexpr int kWords = kChunk / 32;

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
  bool in_place;
};

// A row of the sequence: target row j (line < R_i) or draft row j.
template <typename T>
struct Line {
  const T *in;
  T *out;
  int j;
};

template <typename T>
__device__ __forceinline__ Line<T> line_of(const sv_adjust_args &a, int i, int r0, int Ri, int line) {
  Line<T> L;
  if (line < Ri) {
    const int64_t off = static_cast<int64_t>(r0 + line) * a.vocab;
    L.in = static_cast<const T *>(a.target) + off;
    L.out = static_cast<T *>(a.target_out) + off;
    L.j = line;
  } else {
    const int64_t off = static_cast<int64_t>(r0 - i + line - Ri) * a.vocab;
    L.in = static_cast<const T *>(a.draft) + off;
    L.out = static_cast<T *>(a.draft_out) + off;
    L.j = line - Ri;
  }
  return L;
}

// Bits of tokens t .. t + 7 of a mask row (bytes: token u at bit u % 8 of byte u / 8).
__device__ __forceinline__ uint32_t mask_bits8(const uint8_t *m, int t, int64_t mask_bytes) {
  const int64_t b = t >> 3;
  const uint32_t lo = m[b];
  if ((t & 7) == 0) return lo;
  const uint32_t hi = b + 1 < mask_bytes ? m[b + 1] : 0u;
  return ((lo | (hi << 8)) >> (t & 7)) & 0xFFu;
}

template <typename T>
__global__ void __launch_bounds__(kNT) adjust_kernel(const __grid_constant__ AdjustParams P) {
  using E = Elem<T>;
  constexpr int kPer = 16 / static_cast<int>(sizeof(T));     // elements of a 16-byte vector
  constexpr int kVecs = kChunk / kPer / kNT;                 // vectors per thread and row
  const sv_adjust_args &a = P.a;
  const int tid = threadIdx.x, i = blockIdx.y;
  const int V = a.vocab, c0 = blockIdx.x * kChunk, c1 = min(V, c0 + kChunk);
  const bool head = blockIdx.x == 0 && blockIdx.z == 0;      // this CTA reports the sequence

  __shared__ uint32_t s_extra[kWords];                       // ctx, draft and bias tokens
  __shared__ int32_t s_mask[16];
  __shared__ int s_n;
  __shared__ uint16_t s_tok[kChunk];
  __shared__ uint16_t s_after[kChunk];                       // bit b: draft b + 1 is this token
  __shared__ uint32_t s_word[kChunk];
  __shared__ float s_bias[kChunk];
  __shared__ int32_t s_last[kChunk];                         // 1 + last bias entry of a token

  const int r0 = a.cu_q[i], Ri = a.cu_q[i + 1] - r0;
  if (r0 < i || Ri < 1 || Ri > a.max_q_rows || r0 + Ri > a.num_rows ||
      r0 + Ri - (i + 1) > a.num_rows - a.batch) {            // (its draft rows, too)
    if (head && tid == 0) set_status(a.dev_status, SV_DEV_BAD_LENGTH);
    return;
  }
  const int lines = Ri + (a.draft != nullptr ? Ri - 1 : 0);
  const int l0 = blockIdx.z * P.lines_per_part, l1 = min(lines, l0 + P.lines_per_part);
  if (l0 >= l1) return;

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
  if (tid < Ri) {
    int m = -1;
    if (a.mask) {
      m = a.mask_rows ? a.mask_rows[r0 + tid] : r0 + tid;
      bad |= m < -1 || m >= a.num_masks;
    }
    s_mask[tid] = m;
  }
  if (tid < kWords) s_extra[tid] = 0;
  if (tid == 0) s_n = 0;
  const int nb = b1 - b0;
  if (nb > 0)
    for (int t = tid; t < kChunk; t += kNT) s_last[t] = 0;
  bad = __syncthreads_or(bad);

  if (bad) {                      // rows the sampler fails the sequence on
    if (head && tid == 0) set_status(a.dev_status, SV_DEV_BAD_PARAM);
    for (int l = l0; l < l1; ++l) {
      const Line<T> L = line_of<T>(a, i, r0, Ri, l);
      for (int t = c0 + tid; t < c1; t += kNT) L.out[t] = E::put(NAN);
    }
    return;
  }

  const bool penal = rep != 1.0f || pres != 0.0f || freq != 0.0f;
  const int drafts = penal && a.draft_tokens ? Ri - 1 : 0;
  const int32_t *draft_tokens = a.draft_tokens + (r0 - i);
  const int64_t ctx_stride = a.ctx_stride ? a.ctx_stride : a.batch;

  // tokens outside the table: bits of the chunk
  auto mark = [&](int t) {
    if (t >= c0 && t < c1) atomicOr(&s_extra[(t - c0) >> 5], 1u << ((t - c0) & 31));
  };
  if (tid < drafts) mark(draft_tokens[tid]);
  if (penal)
    for (int c = tid; c < a.num_ctx; c += kNT) mark(a.ctx_tokens[c * ctx_stride + i]);
  for (int e = tid; e < nb; e += kNT) {
    const int t = a.bias_tokens[b0 + e];
    if (t < 0 || t >= V) {
      if (head) set_status(a.dev_status, SV_DEV_BAD_TOKEN);
    } else if (t >= c0 && t < c1) {
      mark(t);
      atomicMax(&s_last[t - c0], e + 1);
    }
  }

  // the copy: 16-byte vectors from the first aligned token of each row, the
  // ends one by one
  for (int l = l0; l < l1; ++l) {
    const Line<T> L = line_of<T>(a, i, r0, Ri, l);
    const int m = s_mask[L.j];
    if (P.in_place && m < 0) continue;
    const uint8_t *bits =
        m < 0 ? nullptr : reinterpret_cast<const uint8_t *>(a.mask) + m * P.mask_bytes;
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(L.in + c0) / sizeof(T)) % kPer);
    const int first = min(c1, c0 + (mis ? kPer - mis : 0));
    const int nvec = (c1 - first) / kPer;
#pragma unroll
    for (int q = 0; q < kVecs; ++q) {
      const int v = tid + q * kNT;
      if (v < nvec) {
        const int t = first + v * kPer;
        uint32_t allow = 0xFFu;
        if (bits) allow = mask_bits8(bits, t, P.mask_bytes);
        if constexpr (kPer == 4) allow &= 0xFu;
        constexpr uint32_t kAll = (1u << kPer) - 1;
        union { uint4 w; T e[kPer]; } x;
        if (allow != 0 && !(P.in_place && allow == kAll)) x.w = *reinterpret_cast<const uint4 *>(L.in + t);
        if (allow != kAll) {
#pragma unroll
          for (int u = 0; u < kPer; ++u)
            if (!((allow >> u) & 1u)) x.e[u] = E::kNegInf;
        }
        if (!(P.in_place && allow == kAll)) *reinterpret_cast<uint4 *>(L.out + t) = x.w;
      }
    }
    const int edge = first - c0, tail = first + nvec * kPer;
    int t = -1;
    if (tid < edge) t = c0 + tid;
    else if (tid >= 32 && tail + tid - 32 < c1) t = tail + tid - 32;
    if (t >= 0) {
      const bool allowed = !bits || ((bits[t >> 3] >> (t & 7)) & 1u);
      if (!allowed) L.out[t] = E::kNegInf;
      else if (!P.in_place) L.out[t] = L.in[t];
    }
  }
  __syncthreads();

  // the list: a thread per word of bits
  if (tid < kWords && c0 + tid * 32 < c1) {
    const uint32_t extra = s_extra[tid];
    uint32_t known = 0;
    if (penal && slot >= 0) known = a.seen[static_cast<int64_t>(slot) * P.seen_words + (c0 >> 5) + tid];
    uint32_t any = known | extra;
    if (c1 - c0 - tid * 32 < 32) any &= (1u << (c1 - c0 - tid * 32)) - 1;
    int at = any ? atomicAdd(&s_n, __popc(any)) : 0;
    while (any) {
      const int b = __ffs(any) - 1;
      any &= any - 1;
      const int local = tid * 32 + b, t = c0 + local;
      uint32_t word = 0, after = 0;
      float bias = 0.0f;
      if ((known >> b) & 1u)
        word = static_cast<uint32_t>(a.counts[static_cast<int64_t>(slot) * V + t]);
      if ((extra >> b) & 1u) {
        if (penal)
          for (int c = 0; c < a.num_ctx; ++c) word += a.ctx_tokens[c * ctx_stride + i] == t;
        for (int d = 0; d < drafts; ++d)
          if (draft_tokens[d] == t) after |= 1u << d;
        if (nb > 0 && s_last[local]) bias = a.bias_values[b0 + s_last[local] - 1];
      }
      s_tok[at] = static_cast<uint16_t>(local);
      s_after[at] = static_cast<uint16_t>(after);
      s_word[at] = word;
      s_bias[at] = bias;
      ++at;
    }
  }
  __syncthreads();

  // the list for every row: one (row, token) per thread
  const int n = s_n, total = n * (l1 - l0);
  for (int it = tid; it < total; it += kNT) {
    const int lr = it / n, e = it - lr * n;
    const Line<T> L = line_of<T>(a, i, r0, Ri, l0 + lr);
    const int t = c0 + s_tok[e], m = s_mask[L.j];
    if (m >= 0) {
      const uint8_t *bits = reinterpret_cast<const uint8_t *>(a.mask) + m * P.mask_bytes;
      if (!((bits[t >> 3] >> (t & 7)) & 1u)) continue;        // barred: written already
    }
    const uint32_t word = s_word[e];
    const uint32_t times =
        (word & 0x7FFFFFFFu) + __popc(s_after[e] & ((1u << L.j) - 1));
    float x = E::get(L.in[t]);
    if (times > 0 || (word >> 31)) x = x > 0.0f ? x / rep : x * rep;
    if (times > 0) x -= fmaf(freq, static_cast<float>(times), pres);
    const float bias = s_bias[e];
    if (bias != 0.0f) x += bias;
    L.out[t] = E::put(x);
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

// ---------------------------------------------------------------- host checks
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
  P.in_place = a->target == a->target_out;
  const int chunks = (a->vocab + kChunk - 1) / kChunk;
  const int lines = a->draft ? 2 * a->max_q_rows - 1 : a->max_q_rows;
  P.lines_per_part = lines;
  const dim3 grid(chunks, a->batch, 1);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->dtype == SV_BF16) adjust_kernel<uint16_t><<<grid, kNT, 0, s>>>(P);
  else adjust_kernel<float><<<grid, kNT, 0, s>>>(P);
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
