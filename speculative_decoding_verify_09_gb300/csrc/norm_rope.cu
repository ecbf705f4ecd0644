// RMS norms of q and k heads and rotary positions in one pass over ragged rows
// (sm_103a), to contiguous rows or, K and V as 4-bit codes, into a paged cache;
// and rows read back out of the pages.  Contracts: spec_norm_rope_rows,
// spec_kv4_append and spec_kv4_read in include/spec_kv4.h.
//
// A head's D elements lie with D / 16 neighbouring lanes (rounded up to a power of
// two), 16 each, so that its sum of squares and the largest magnitude of 16
// elements are a few shuffles away and nothing is read twice.  Where the two
// halves of a pair are a multiple of 8 apart a lane holds 8 elements and the 8
// partners of these; neighbouring pairs lie with one lane anyway; for other
// distances the partner is fetched through shared memory.  Angles as in rope.cu:
// the position times the turn fraction modulo 2^64, a quarter turn taken off,
// the rest rounded once.
#include <algorithm>
#include <cmath>

#include "kv4.inl"
#include "ops_host.inl"
#include "rows.inl"

namespace sv {

namespace {

constexpr int kNT = 256;
constexpr int kPad = 20;                             // floats between lanes in the exchange

enum Output { kRows, kCodes8, kPages };              // k and v: as they came, E4M3, E2M1 in pages

struct NormRopeParams {
  int batch, max_q_rows, Hq, Hkv, D, half;           // half: pairs that are turned
  int nq, nk, heads;                                 // q heads, k heads, all heads of a row
  int lane_shift, row_shift, pairs;                  // log2 lanes of a head, threads of a row
  int heads_per_cta;
  int by_row, interleaved;
  int64_t num_rows, slots;
  int64_t q_stride, k_stride, v_stride;
  float mscale, k_scale, v_scale, k_inverse, v_inverse;
  float eps, weight_offset;
  const float *q_weight, *k_weight;
  const uint64_t *turns;
  const int32_t *cu_q, *kv_len;
  const int64_t *positions;
  const void *q, *k, *v;
  void *q_out, *k_out, *v_out;
  Kv4View cache;
  uint32_t *dev_status;
};

// Codes and scale of 16 elements whose largest magnitude is m, of which this lane
// holds N (eight, or all): unit = scale * factor is what a code of 1 stands for.
__device__ __forceinline__ uint32_t scale_code(float m, float factor, float &unit) {
  const uint32_t s = e4m3x2_of(__fdiv_rn(m, __fmul_rn(6.0f, factor)), 0.0f) & 0xFFu;
  unit = __fmul_rn(e4m3_to_f32(s), factor);
  return s;
}
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float unit) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = unit == 0.0f ? 0.0f : __fdiv_rn(x[i], unit);
  return e2m1x8_of(y);
}
__device__ __forceinline__ float largest(const float (&x)[8]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(x[i]));
  return m;
}

// PAIRED: the half layout with half a multiple of 8 (16 for pages), or no pairs;
// else 16 elements in a row lie with a lane.
template <typename T, Output OUT, bool PAIRED>
__global__ void __launch_bounds__(kNT, 3) norm_rope_kernel(const NormRopeParams P) {
  extern __shared__ __align__(16) float s_turn[];    // [rows][cos, sin][pairs]
  __shared__ float s_swap[PAIRED ? 1 : kNT * kPad];
  const int row_threads = 1 << P.row_shift, lanes = 1 << P.lane_shift;
  const int rl = threadIdx.x >> P.row_shift, t = threadIdx.x & (row_threads - 1);
  const int hl = t >> P.lane_shift, c = t & (lanes - 1), hstep = row_threads >> P.lane_shift;
  const int h_begin = blockIdx.y * P.heads_per_cta;
  const int h_end = min(P.heads, h_begin + P.heads_per_cta);
  wait_for_previous();

  int64_t row = 0, pos = 0;
  int seq = 0;
  bool bad;
  const bool live = find_row(P, static_cast<int64_t>(blockIdx.x) * (kNT >> P.row_shift) + rl, row, pos,
                             bad, &seq);
  if (bad && t == 0 && blockIdx.y == 0) set_status(P.dev_status, SV_DEV_BAD_LENGTH);
  if (P.by_row && blockIdx.y == 0)                   // (a bad sequence need not be found by a row)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNT + threadIdx.x; i < P.batch;
         i += static_cast<int64_t>(gridDim.x) * kNT)
      if (!good_sequence(P, static_cast<int>(i))) set_status(P.dev_status, SV_DEV_BAD_LENGTH);

  // this lane's column: two vectors of 8 elements of a head
  const bool turn = PAIRED && 8 * c < P.half;
  const int o0 = !PAIRED ? 16 * c : turn ? 8 * c : 2 * P.half + 16 * (c - P.half / 8);
  const int o1 = turn ? o0 + P.half : o0 + 8;
  const bool column = live && o0 < P.D, both = column && o1 < P.D;

  Vec<T, 8> cur[2], nxt[2];
  const int k0 = P.nq * P.D, v0 = (P.nq + P.nk) * P.D;
  const T *in_q = static_cast<const T *>(P.q) + row * P.q_stride;
  const T *in_k = static_cast<const T *>(P.k) + row * P.k_stride - k0;
  const T *in_v = static_cast<const T *>(P.v) + row * P.v_stride - v0;
  auto fetch = [&](Vec<T, 8> (&v)[2], int h) {
    if (!column || h >= h_end) return;
    const T *p = (h < P.nq ? in_q : h < P.nq + P.nk ? in_k : in_v) + h * P.D;
    v[0].load(p + o0);
    if (both) v[1].load(p + o1);
  };
  fetch(cur, h_begin + hl);

  // cos and sin of the row's pairs, by the threads that share the row
  float *s_cos = s_turn + rl * 2 * P.pairs, *s_sin = s_cos + P.pairs;
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
  uint8_t *slab = nullptr;                           // of the row's token, KV head 0
  if (OUT == kPages && live) {
    uint32_t why = 0;
    slab = find_slab(P.cache, seq, pos, &why);
    if (why && t == 0 && blockIdx.y == 0) set_status(P.dev_status, why);
  }
  __syncthreads();
  if (!live) return;                                 // (all threads of a warp share a row)

  // the pairs of this column, and its weights, fetched again where q's end and k's begin
  float cs[8], sn[8], w0[8], w1[8];
  if (any_turn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = 8 * c + i;
      const bool on = (PAIRED || P.interleaved) && p < P.half;
      cs[i] = on ? s_cos[p] : 1.0f;
      sn[i] = on ? s_sin[p] : 0.0f;
    }
  }
  const bool norms = P.q_weight != nullptr || P.k_weight != nullptr;
  const float *have = nullptr;                       // whose weights w0 and w1 hold
  const int64_t kv_row = row * P.Hkv * P.D;
  const int token = static_cast<int>(pos) & (kSlab - 1);

  for (int hb = h_begin; hb < h_end; hb += hstep) {
    const int h = hb + hl;
    const bool on = column && h < h_end;
    const bool is_q = h < P.nq, is_k = !is_q && h < P.nq + P.nk;
    fetch(nxt, h + hstep);
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.0f;
    if (on) cur[0].get(x);
    if (on && both) cur[1].get(y);
    if (norms) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
      for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float *w = is_q ? P.q_weight : is_k ? P.k_weight : nullptr;
      if (on && w != nullptr) {
        if (w != have) {
          have = w;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            w0[i] = w[o0 + i] + P.weight_offset;
            w1[i] = both ? w[o1 + i] + P.weight_offset : 0.0f;
          }
        }
        const float r = 1.0f / sqrtf(ss / static_cast<float>(P.D) + P.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = x[i] * r * w0[i];
          y[i] = y[i] * r * w1[i];
        }
      }
    }
    if constexpr (PAIRED) {
      if (turn && any_turn && (is_q || is_k)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = x[i], b = y[i];
          x[i] = a * cs[i] - b * sn[i];
          y[i] = b * cs[i] + a * sn[i];
        }
      }
    } else if (any_turn) {
      if (P.interleaved) {
        if (is_q || is_k) {
          auto turn4 = [&](float (&z)[8], int first) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = z[2 * i], b = z[2 * i + 1];
              if (8 * c + first + i < P.half) {
                z[2 * i] = a * cs[first + i] - b * sn[first + i];
                z[2 * i + 1] = b * cs[first + i] + a * sn[first + i];
              }
            }
          };
          turn4(x, 0);
          turn4(y, 4);
        }
      } else {                                       // partners through shared memory
        float *mine = s_swap + threadIdx.x * kPad, *head = s_swap + (threadIdx.x - c) * kPad;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          mine[i] = x[i];
          mine[8 + i] = y[i];
        }
        __syncwarp();
        if (is_q || is_k) {
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
        }
      }
    }
    if (OUT == kPages) {                             // (all lanes: shuffles)
      float m0 = largest(x), m1 = largest(y);
      const float n0 = __shfl_xor_sync(0xffffffffu, m0, 1), n1 = __shfl_xor_sync(0xffffffffu, m1, 1);
      const float all = max_nan(m0, m1);
      m0 = turn ? max_nan(m0, n0) : all;
      m1 = turn ? max_nan(m1, n1) : all;
      if (on && !is_q && slab != nullptr) {
        const int hk = is_k ? h - P.nq : h - P.nq - P.nk;
        uint8_t *at = slab + hk * head_bytes(P.cache) + (is_k ? 0 : slab_v(P.D));
        const float factor = is_k ? P.k_scale : P.v_scale;
        float u0, u1;
        const uint32_t s0 = scale_code(m0, factor, u0), s1 = scale_code(m1, factor, u1);
        uint8_t *codes = at + token * (P.D / 2), *scales = at + slab_k_scales(P.D) + token * (P.D / 16);
        *reinterpret_cast<uint32_t *>(codes + o0 / 2) = codes_of(x, u0);
        *reinterpret_cast<uint32_t *>(codes + o1 / 2) = codes_of(y, u1);
        if (!turn || c % 2 == 0) {                   // one lane of those that share 16 elements
          scales[o0 / 16] = static_cast<uint8_t>(s0);
          if (turn) scales[o1 / 16] = static_cast<uint8_t>(s1);
        }
      }
    }
    if (on && (OUT != kPages || is_q)) {
      if (OUT == kCodes8 && !is_q) {
        uint8_t *o = static_cast<uint8_t *>(is_k ? P.k_out : P.v_out) + kv_row + (h * P.D - (is_k ? k0 : v0));
        const float scale = is_k ? P.k_scale : P.v_scale, inverse = is_k ? P.k_inverse : P.v_inverse;
        store_codes(o + o0, x, scale, inverse);
        if (both) store_codes(o + o1, y, scale, inverse);
      } else {
        T *o = is_q ? static_cast<T *>(P.q_out) + row * P.Hq * P.D + h * P.D
                    : static_cast<T *>(is_k ? P.k_out : P.v_out) + kv_row + (h * P.D - (is_k ? k0 : v0));
        if (is_q || is_k) {                          // (v keeps its bits)
          cur[0].set(x);
          cur[1].set(y);
        }
        cur[0].store(o + o0);
        if (both) cur[1].store(o + o1);
      }
    }
    cur[0] = nxt[0];
    cur[1] = nxt[1];
  }
}

// ---------------------------------------------------------------- read
struct ReadParams {
  int batch, max_q_rows, D, row_shift;
  int by_row;
  int64_t num_rows, slots;
  float k_scale, v_scale, k_inverse, v_inverse;      // E4M3 outputs
  const int32_t *cu_q, *kv_len;
  const int64_t *positions;                          // nullptr
  void *k_out, *v_out;
  Kv4View cache;
  uint32_t *dev_status;
};

// The threads of a row take 16 elements (8 bytes of codes, one scale) at a time
// from its K and V heads in turn.
template <typename T>
__global__ void __launch_bounds__(kNT) kv4_read_kernel(const ReadParams P) {
  const int row_threads = 1 << P.row_shift;
  const int rl = threadIdx.x >> P.row_shift, t = threadIdx.x & (row_threads - 1);
  wait_for_previous();
  int64_t row = 0, pos = 0;
  int seq = 0;
  bool bad;
  const bool live = find_row(P, static_cast<int64_t>(blockIdx.x) * (kNT >> P.row_shift) + rl, row, pos,
                             bad, &seq);
  if (bad && t == 0 && blockIdx.y == 0) set_status(P.dev_status, SV_DEV_BAD_LENGTH);
  if (P.by_row && blockIdx.y == 0)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNT + threadIdx.x; i < P.batch;
         i += static_cast<int64_t>(gridDim.x) * kNT)
      if (!good_sequence(P, static_cast<int>(i))) set_status(P.dev_status, SV_DEV_BAD_LENGTH);
  if (!live) return;
  uint32_t why = 0;
  const uint8_t *slab = find_slab(P.cache, seq, pos, &why);
  if (why && t == 0 && blockIdx.y == 0) set_status(P.dev_status, why);
  if (slab == nullptr) return;
  const int token = static_cast<int>(pos) & (kSlab - 1);
  const int groups = P.D / 16, items = 2 * P.cache.heads * groups;
  for (int it = blockIdx.y * row_threads + t; it < items; it += gridDim.y * row_threads) {
    const int part = it / groups, g = it - part * groups;
    const bool is_v = part >= P.cache.heads;
    void *out = is_v ? P.v_out : P.k_out;
    if (out == nullptr) continue;
    const int h = is_v ? part - P.cache.heads : part;
    const uint8_t *at = slab + h * head_bytes(P.cache) + (is_v ? slab_v(P.D) : 0);
    const uint2 codes = *reinterpret_cast<const uint2 *>(at + token * (P.D / 2) + 8 * g);
    const float s = e4m3_to_f32(at[slab_k_scales(P.D) + token * groups + g]);
    const float factor = is_v ? P.cache.v_scale : P.cache.k_scale;
    T *o = static_cast<T *>(out) + (row * P.cache.heads + h) * P.D + 16 * g;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t pair[4];
      e2m1x8_to_f16x2(half ? codes.y : codes.x, pair);
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = f16_bits_to_f32(i % 2 ? pair[i / 2] >> 16 : pair[i / 2] & 0xFFFFu);
        x[i] = __fmul_rn(__fmul_rn(c, s), factor);   // the first product is exact
      }
      if constexpr (sizeof(T) == 1) {
        store_codes(o + 8 * half, x, is_v ? P.v_scale : P.k_scale, is_v ? P.v_inverse : P.k_inverse);
      } else {
        Vec<T, 8> v;
        v.set(x);
        v.store(o + 8 * half);
      }
    }
  }
}

float exact_inverse(float x) {                       // 1 / x where x is a power of two, else 0
  int e;
  const float inv = 1.0f / x;
  return std::frexp(x, &e) == 0.5f && std::isnormal(inv) ? inv : 0.0f;
}

template <typename T, Output OUT>
cudaError_t launch_layout(bool paired, dim3 grid, size_t smem, cudaStream_t s, const NormRopeParams &P) {
  return paired ? launch_after_previous(norm_rope_kernel<T, OUT, true>, grid, kNT, smem, s, P)
                : launch_after_previous(norm_rope_kernel<T, OUT, false>, grid, kNT, smem, s, P);
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
  P.interleaved = a.layout == SV_ROPE_INTERLEAVED;
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
  if (P.num_rows == 0 || P.slots == 0 || P.heads == 0) return SV_OK;
  const int sms = device_sms();
  if (sms <= 0) return record_error(SV_ERR_CUDA, "%s: no current CUDA device", who);

  while ((16 << P.lane_shift) < P.D) ++P.lane_shift;
  const bool paired = !P.half || (!P.interleaved && P.half % (cache ? 16 : 8) == 0);
  const int64_t threads = (P.slots * P.heads) << P.lane_shift, room = 512 * static_cast<int64_t>(sms);
  P.row_shift = 7;
  if (P.slots > 6 * static_cast<int64_t>(sms))
    for (P.row_shift = 5; P.row_shift < 7 && (6 << P.row_shift) < (P.heads << P.lane_shift);) ++P.row_shift;
  P.pairs = (P.half + 7) / 4 * 4;
  const int at_once = 1 << (P.row_shift - P.lane_shift);
  P.heads_per_cta = static_cast<int>(
      std::min<int64_t>(P.heads, std::max<int64_t>(1, (threads + room - 1) / room) * at_once));
  const int rows_per_cta = kNT >> P.row_shift;
  const dim3 grid(static_cast<unsigned>((P.slots + rows_per_cta - 1) / rows_per_cta),
                  static_cast<unsigned>((P.heads + P.heads_per_cta - 1) / P.heads_per_cta));
  const size_t smem = static_cast<size_t>(rows_per_cta) * 2 * P.pairs * sizeof(float);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.dtype == SV_BF16)
    e = cache                     ? launch_layout<uint16_t, kPages>(paired, grid, smem, s, P)
        : a.kv_dtype == SV_E4M3 ? launch_layout<uint16_t, kCodes8>(paired, grid, smem, s, P)
                                  : launch_layout<uint16_t, kRows>(paired, grid, smem, s, P);
  else
    e = cache                     ? launch_layout<float, kPages>(paired, grid, smem, s, P)
        : a.kv_dtype == SV_E4M3 ? launch_layout<float, kCodes8>(paired, grid, smem, s, P)
                                  : launch_layout<float, kRows>(paired, grid, smem, s, P);
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
  P.dev_status = a->dev_status;
  set_slots(P);
  if (P.num_rows == 0 || P.slots == 0 || (!P.k_out && !P.v_out)) return SV_OK;
  const int items = 2 * P.cache.heads * (P.D / 16);
  for (P.row_shift = 5; P.row_shift < 8 && (1 << P.row_shift) < items;) ++P.row_shift;
  const int rows_per_cta = kNT >> P.row_shift;
  const dim3 grid(static_cast<unsigned>((P.slots + rows_per_cta - 1) / rows_per_cta));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      a->dtype == SV_BF16  ? launch_after_previous(kv4_read_kernel<uint16_t>, grid, kNT, size_t{0}, s, P)
      : a->dtype == SV_F32 ? launch_after_previous(kv4_read_kernel<float>, grid, kNT, size_t{0}, s, P)
                           : launch_after_previous(kv4_read_kernel<uint8_t>, grid, kNT, size_t{0}, s, P);
  if (e != cudaSuccess) return record_error(SV_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return SV_OK;
}

}  // extern "C"
