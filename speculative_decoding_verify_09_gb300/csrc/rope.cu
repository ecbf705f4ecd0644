// Rotary positions of ragged rows, fused with the E4M3 quantization of K and V
// (sm_103a).  Contract: spec_rope_rows in include/spec_ops.h.
//
// Pair (a, b) of a row at position t becomes m (a cos x - b sin x, b cos x + a
// sin x), x = t f_p.  What has to be exact is x modulo a turn: at t = 2^20 an
// fp32 product is off by 2^-4 radians.  f_p / (2 pi) is kept as a 64-bit
// fraction of a turn, so t times it modulo 2^64 -- one integer multiplication
// -- is the exact fraction of a turn (up to t * 2^-65 from rounding f_p).  The
// nearest quarter turn is taken off as an integer too, so that the one rounding
// of the angle to fp32 (for sincospif) is of an eighth of a turn at most.
//
// The kernel is one pass over the rows: bytes bound for prompts, launch bound
// for a step's rows.  A row's cos and sin are computed once per CTA into shared
// memory (rot_dim / 2 pairs, one per thread), while the first 16-byte vectors
// of the row are in flight, and each thread keeps the pairs of its vector
// column in registers over all heads of the row.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "ops_host.inl"
#include "spec_ops.h"

namespace sv {

namespace {

constexpr int kNT = 256;
constexpr int kMaxDim = 256;
constexpr int kMaxHeads = 16384;                     // of q, and of k and v
constexpr int kPasses = 6;                           // heads that one thread works on, about

// How a thread's elements of a head meet their partners.  G = 8, 4, 2, 1 (the
// half layout): G elements and the G that are rot_dim / 2 further on, i.e. G
// whole pairs, where G is the largest that divides rot_dim / 2 and so keeps the
// accesses aligned.  kNeighbor (the interleaved layout, rot_dim a multiple of 16): two
// vectors of 8 elements, 4 whole pairs each.  kMixed (any other rot_dim): the same, but
// one column holds the last pairs and copied elements; those keep their bits, so its
// pairs are turned in place, one by one.  In one kernel the selects cost the other
// columns registers (176 rows of 48 heads, half of each turned: 2.9 us so, 3.1 to 3.7 us
// by where they stand in a common one; 32768 rows of 48 heads of 128, bf16: 126 us,
// with rot_dim 40 130 us).
constexpr int kNeighbor = 0, kMixed = -1;

struct RopeParams {
  int batch, max_q_rows, Hq, Hkv, D, rot;
  int nq, nk, heads;            // q heads, k heads, all heads of a row (q, k, then v)
  int columns, per_column;      // threads that share a head, and 2^16 / columns rounded up: (x *
                                // per_column) >> 16 is x / columns for x up to 256
  int row_shift, pairs;         // log2 threads that share a row; its room for cos and for sin
  int heads_per_cta;
  int64_t num_rows, slots;      // slots: rows, or max_q_rows for every sequence
  int by_row;                   // slots are rows, whose sequences are searched
  int64_t q_stride, k_stride, v_stride;
  float mscale, k_scale, v_scale;
  float k_inverse, v_inverse;   // reciprocals of scales that are powers of two, else 0
  const uint64_t *turns;
  const int32_t *cu_q, *kv_len;
  const int64_t *positions;
  const void *q, *k, *v;
  void *q_out, *k_out, *v_out;
  uint32_t *dev_status;
};

// N elements as they lie in memory.
template <int BYTES> struct Raw;
template <> struct Raw<32> { uint4 a, b; };
template <> struct Raw<16> { uint4 a; };
template <> struct Raw<8> { uint2 a; };
template <> struct Raw<4> { uint32_t a; };
template <> struct Raw<2> { uint16_t a; };

template <typename T, int N>
struct Vec {
  union {
    Raw<N * static_cast<int>(sizeof(T))> raw;
    T e[N];
  };
  __device__ __forceinline__ void load(const T *p) { raw = *reinterpret_cast<const decltype(raw) *>(p); }
  __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<decltype(raw) *>(p) = raw; }
  __device__ __forceinline__ void get(float (&x)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 2) x[i] = bf16_bits_to_f32(e[i]);
      else x[i] = e[i];
    }
  }
  __device__ __forceinline__ void set(const float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 4) {
        e[i] = x[i];
      } else if (N % 2) {
        e[i] = f32_to_bf16_rn(x[i]);
      } else if (i % 2 == 0) {
        const uint32_t two = pack_bf16x2(x[i], x[i + 1]);
        e[i] = static_cast<uint16_t>(two);
        e[i + 1] = static_cast<uint16_t>(two >> 16);
      }
    }
  }
  // The pair of elements i (even) and i + 1 turned in place, or left as it is.
  __device__ __forceinline__ void turn_pair(int i, float cs, float sn, bool on) {
    if constexpr (sizeof(T) == 2) {
      const float a = bf16_bits_to_f32(e[i]), b = bf16_bits_to_f32(e[i + 1]);
      const uint32_t two = pack_bf16x2(a * cs - b * sn, b * cs + a * sn);
      e[i] = on ? static_cast<uint16_t>(two) : e[i];
      e[i + 1] = on ? static_cast<uint16_t>(two >> 16) : e[i + 1];
    } else {
      const float a = e[i], b = e[i + 1];
      e[i] = on ? a * cs - b * sn : a;
      e[i + 1] = on ? b * cs + a * sn : b;
    }
  }
};

// Two floats -> two E4M3 codes (lo in the lower byte), nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Codes of x / scale; inverse: 1 / scale where that is exact (scale a power of two), else 0.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t *p, const float (&x)[N], float scale, float inverse) {
  float y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = inverse != 0.0f ? x[i] * inverse : x[i] / scale;
  if constexpr (N == 1) {
    *p = static_cast<uint8_t>(e4m3x2_of(y[0], 0.0f));
  } else {
    Vec<uint16_t, N / 2> v;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v.e[i] = static_cast<uint16_t>(e4m3x2_of(y[2 * i], y[2 * i + 1]));
    v.store(reinterpret_cast<uint16_t *>(p));
  }
}

// Whether sequence i's rows agree with the host's bounds.
__device__ __forceinline__ bool good_sequence(const RopeParams &P, int i) {
  const int r0 = P.cu_q[i], r1 = P.cu_q[i + 1];
  return r0 >= 0 && r1 >= r0 && r1 <= P.num_rows && r1 - r0 <= P.max_q_rows && P.kv_len[i] >= 0;
}

// Row and position of slot `slot`; false if there is no such row (or a bad one).
__device__ __forceinline__ bool find_row(const RopeParams &P, int64_t slot, int64_t &row,
                                         int64_t &pos, bool &bad) {
  bad = false;
  if (slot >= P.slots) return false;
  if (P.positions != nullptr) {
    row = slot;
    pos = P.positions[slot];
    bad = pos <= -(int64_t{1} << 31) || pos >= (int64_t{1} << 31);
    return !bad;
  }
  int i, j;
  if (P.by_row) {                 // the last sequence that starts at or before the row
    int lo = 0, hi = P.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (P.cu_q[mid] <= slot) lo = mid; else hi = mid;
    }
    i = lo;
    j = static_cast<int>(slot) - P.cu_q[i];
  } else {
    i = static_cast<int>(static_cast<uint32_t>(slot) / static_cast<uint32_t>(P.max_q_rows));
    j = static_cast<int>(slot) - i * P.max_q_rows;
  }
  const int r0 = P.cu_q[i], r1 = P.cu_q[i + 1], L = P.kv_len[i];
  if (!good_sequence(P, i)) {
    bad = true;
    return false;
  }
  if (j < 0 || j >= r1 - r0) return false;
  row = r0 + j;
  pos = static_cast<int64_t>(L) + j;
  return true;
}

// Heads that a thread has in flight (and as many that it works on): narrow
// columns load little at a time.  CTAs per SM that the registers are capped for.
// As measured (32768 rows of 48 heads of 128): bf16 G = 8 122 us at 4 CTAs, 134 at
// 3, 131 at 5; fp32 237 us at 3, 253 at 4; with codes 131 us at 3, 165 at 5; one,
// two, four heads at G = 1 304, 266, 232 us, at G = 2 180, 168, 150 us, one and two
// at G = 4 162 and 134 us.  The caps cost some kernels a little local memory, which stays
// in L1: 16 and 20 bytes a thread in bf16 with codes, interleaved and at G = 8, 28 and 32
// in fp32 with codes, 12 to 40 at G = 4 with codes or in fp32.  A CTA per SM less needs
// none, but takes 167 against 135 us (bf16, codes, G = 8), 169 against 140 (interleaved),
// 243 against 218 (fp32, codes, G = 8); only at G = 4 with codes it would pay (162 against
// 187 us in bf16, 225 against 258 in fp32).
template <int G, bool KV8>
struct InFlight {
  static constexpr int kHeads = G == 1 || G == 2 ? (KV8 ? 2 : 4) : G == 4 ? 2 : 1;
};
template <typename T, int G, bool KV8>
constexpr int min_ctas() {
  return (G == 8 || G <= kNeighbor) && (KV8 || sizeof(T) == 4) ? 3 : 4;
}

template <typename T, int G, bool KV8>
__global__ void __launch_bounds__(kNT, min_ctas<T, G, KV8>()) rope_kernel(const RopeParams P) {
  extern __shared__ __align__(16) float s_turn[];        // [rows][cos, sin][pairs]
  const int row_threads = 1 << P.row_shift;
  const int rl = threadIdx.x >> P.row_shift, t = threadIdx.x & (row_threads - 1);
  const int hl = (t * P.per_column) >> 16, c = t - hl * P.columns;
  const int hstep = (row_threads * P.per_column) >> 16;
  const int h_begin = blockIdx.y * P.heads_per_cta;
  const int h_end = min(P.heads, h_begin + P.heads_per_cta);
  const int half = P.rot >> 1;
  wait_for_previous();

  int64_t row = 0, pos = 0;
  bool bad;
  const bool live = find_row(P, static_cast<int64_t>(blockIdx.x) * (kNT >> P.row_shift) + rl, row,
                             pos, bad);
  if (bad && t == 0 && blockIdx.y == 0) set_status(P.dev_status, SV_DEV_BAD_LENGTH);
  if (P.by_row && blockIdx.y == 0)                       // (a bad sequence need not be found by a row)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNT + threadIdx.x; i < P.batch;
         i += static_cast<int64_t>(gridDim.x) * kNT)
      if (!good_sequence(P, static_cast<int>(i))) set_status(P.dev_status, SV_DEV_BAD_LENGTH);

  // this thread's column: element offsets inside a head
  constexpr bool kBeside = G <= kNeighbor;               // a pair's elements stand side by side
  constexpr int N = kBeside ? 8 : G;
  const bool turn = kBeside ? 2 * N * c < P.rot : c < half / N;   // the column holds pairs
  const int o0 = kBeside ? 2 * N * c : turn ? N * c : P.rot + 2 * N * (c - half / N);
  const int o1 = !kBeside && turn ? o0 + half : o0 + N;
  const bool column = live && hl < hstep;
  const bool both = o1 < P.D;                            // (the last column may be single)

  constexpr int U = InFlight<G, KV8>::kHeads;
  Vec<T, N> cur[U][2], nxt[U][2];
  // the row's heads, numbered through q, k, v: element h D of these
  const int k0 = P.nq * P.D, v0 = (P.nq + P.nk) * P.D;
  const T *in_q = static_cast<const T *>(P.q) + row * P.q_stride;
  const T *in_k = static_cast<const T *>(P.k) + row * P.k_stride - k0;
  const T *in_v = static_cast<const T *>(P.v) + row * P.v_stride - v0;
  auto source = [&](int h) { return (h < P.nq ? in_q : h < P.nq + P.nk ? in_k : in_v) + h * P.D; };
  auto fetch = [&](Vec<T, N> (&v)[2], int h) {
    if (!column || h >= h_end) return;
    const T *p = source(h);
    v[0].load(p + o0);
    if (both) v[1].load(p + o1);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) fetch(cur[u], h_begin + hl + u * hstep);

  // cos and sin of the row's pairs, by the threads that share the row
  float *s_cos = s_turn + rl * 2 * P.pairs, *s_sin = s_cos + P.pairs;
  const bool any_turn = h_begin < P.nq + P.nk;
  if (live && any_turn) {
    for (int p = t; p < half; p += row_threads) {
      const uint64_t part = static_cast<uint64_t>(pos) * P.turns[p];
      const uint64_t quarter = (part + (uint64_t{1} << 61)) >> 62;      // the nearest, 0..3
      const int64_t rest = static_cast<int64_t>(part - (quarter << 62));
      float s0, c0;                                                   // of the rest, then of the angle
      sincospif(__ll2float_rn(rest) * 0x1p-63f, &s0, &c0);
      const float sn = quarter & 1 ? c0 : s0, cs = quarter & 1 ? s0 : c0;
      s_cos[p] = ((quarter + 1) & 2 ? -cs : cs) * P.mscale;
      s_sin[p] = (quarter & 2 ? -sn : sn) * P.mscale;
    }
  }
  __syncthreads();
  if (!column) return;

  // the pairs of this column
  float cs[N], sn[N];
  if (any_turn && turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = N * c + i;
      cs[i] = p < half ? s_cos[p] : 1.0f;
      sn[i] = p < half ? s_sin[p] : 0.0f;
    }
  }

  const int64_t kv_row = row * P.Hkv * P.D;
  T *out_q = static_cast<T *>(P.q_out) + row * P.Hq * P.D;
  T *out_k = static_cast<T *>(P.k_out) + kv_row - k0, *out_v = static_cast<T *>(P.v_out) + kv_row - v0;
  uint8_t *codes_k = static_cast<uint8_t *>(P.k_out) + kv_row - k0;
  uint8_t *codes_v = static_cast<uint8_t *>(P.v_out) + kv_row - v0;
  auto finish = [&](Vec<T, N> (&v)[2], int h) {
    const bool is_q = h < P.nq, is_k = !is_q && h < P.nq + P.nk, codes = KV8 && !is_q;
    float x[N], y[N];
    bool done = false;
    if constexpr (G == kMixed) {                         // pair by pair, the copied elements not touched
      done = !codes;
      if (done && turn && (is_q || is_k)) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i / 4].turn_pair(i % 4 * 2, cs[i], sn[i], N * c + i < half);
      }
    }
    if (!done && ((turn && (is_q || is_k)) || codes)) {
      v[0].get(x);
      v[1].get(y);
    }
    if (!done && turn && (is_q || is_k)) {
      if constexpr (!kBeside) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float a = x[i], b = y[i];
          x[i] = a * cs[i] - b * sn[i];
          y[i] = b * cs[i] + a * sn[i];
        }
      } else {
        auto turn4 = [&](float (&z)[N], int first) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = z[2 * i], b = z[2 * i + 1];
            if (G == kNeighbor || N * c + first + i < half) {
              z[2 * i] = a * cs[first + i] - b * sn[first + i];
              z[2 * i + 1] = b * cs[first + i] + a * sn[first + i];
            }
          }
        };
        turn4(x, 0);
        turn4(y, 4);
      }
      if (!codes) {
        v[0].set(x);
        v[1].set(y);
      }
    }
    if (codes) {
      uint8_t *o = (is_k ? codes_k : codes_v) + h * P.D;
      const float scale = is_k ? P.k_scale : P.v_scale, inverse = is_k ? P.k_inverse : P.v_inverse;
      store_codes(o + o0, x, scale, inverse);
      if (both) store_codes(o + o1, y, scale, inverse);
    } else {
      T *o = (is_q ? out_q : is_k ? out_k : out_v) + h * P.D;
      v[0].store(o + o0);
      if (both) v[1].store(o + o1);
    }
  };
  for (int h = h_begin + hl; h < h_end; h += U * hstep) {
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(nxt[u], h + (U + u) * hstep);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * hstep < h_end) finish(cur[u], h + u * hstep);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int n = 0; n < 2; ++n) cur[u][n] = nxt[u][n];
  }
}

template <typename T, bool KV8>
cudaError_t launch_shape(int g, dim3 grid, const RopeParams &P, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(kNT >> P.row_shift) * 2 * P.pairs * sizeof(float);
  if (g == kNeighbor) return launch_behind(rope_kernel<T, kNeighbor, KV8>, grid, kNT, smem, s, P);
  if (g == kMixed) return launch_behind(rope_kernel<T, kMixed, KV8>, grid, kNT, smem, s, P);
  if (g == 8) return launch_behind(rope_kernel<T, 8, KV8>, grid, kNT, smem, s, P);
  if (g == 4) return launch_behind(rope_kernel<T, 4, KV8>, grid, kNT, smem, s, P);
  if (g == 2) return launch_behind(rope_kernel<T, 2, KV8>, grid, kNT, smem, s, P);
  return launch_behind(rope_kernel<T, 1, KV8>, grid, kNT, smem, s, P);
}

bool positive(float x) { return std::isfinite(x) && x > 0.0f; }

sv_status check_rope(const sv_rope_args *a) {
  auto bad = [](const char *what) { return record_error(SV_ERR_INVALID, "rope: %s", what); };
  if (!a) return bad("null arguments");
  if (a->dtype != SV_F32 && a->dtype != SV_BF16)
    return record_error(SV_ERR_INVALID, "rope: dtype %d", a->dtype);
  if (a->kv_dtype != 0 && a->kv_dtype != SV_E4M3)
    return record_error(SV_ERR_INVALID, "rope: kv_dtype %d (0 or SV_E4M3)", a->kv_dtype);
  if (a->num_q_heads < 0 || a->num_q_heads > kMaxHeads || a->num_kv_heads < 0 || a->num_kv_heads > kMaxHeads)
    return record_error(SV_ERR_INVALID, "rope: heads Hq=%d Hkv=%d outside [0, %d]", a->num_q_heads,
                        a->num_kv_heads, kMaxHeads);
  if (a->head_dim < 8 || a->head_dim > kMaxDim || a->head_dim % 8)
    return record_error(SV_ERR_UNSUPPORTED, "rope: head_dim %d (built: multiples of 8 up to %d)",
                        a->head_dim, kMaxDim);
  if (a->rot_dim < 2 || a->rot_dim > a->head_dim || a->rot_dim % 2)
    return record_error(SV_ERR_INVALID, "rope: rot_dim %d (even, 2..head_dim %d)", a->rot_dim,
                        a->head_dim);
  if (a->layout != SV_ROPE_HALF && a->layout != SV_ROPE_INTERLEAVED)
    return record_error(SV_ERR_INVALID, "rope: layout %d", a->layout);
  if (a->num_rows < 0 || a->num_rows >= (int64_t{1} << 31))
    return record_error(SV_ERR_INVALID, "rope: num_rows %lld", static_cast<long long>(a->num_rows));
  if (!(a->mscale == 0.0f || positive(a->mscale))) return bad("mscale must be finite and >= 0");
  if (!(a->k_scale == 0.0f || positive(a->k_scale)) || !(a->v_scale == 0.0f || positive(a->v_scale)))
    return bad("k_scale / v_scale must be finite and >= 0");
  if (!a->positions) {
    if (a->batch < 0) return record_error(SV_ERR_INVALID, "rope: batch %d", a->batch);
    if (a->max_q_rows < 1) return record_error(SV_ERR_INVALID, "rope: max_q_rows %d", a->max_q_rows);
    const int64_t slots = static_cast<int64_t>(a->batch) * a->max_q_rows;
    if (slots >= (int64_t{1} << 31)) return bad("batch * max_q_rows passes 2^31");
    if (a->batch > 0 && (!a->cu_q || !a->kv_len)) return bad("null cu_q / kv_len without positions");
  }
  if (a->num_rows == 0) return SV_OK;
  if (!a->turns) return bad("null turns");
  const int64_t esz = a->dtype == SV_F32 ? 4 : 2;
  struct { const void *in; void *out; int heads; int64_t stride; bool kv; const char *name; } const
      tensors[3] = {{a->q, a->q_out, a->num_q_heads, a->q_stride, false, "q"},
                    {a->k, a->k_out, a->num_kv_heads, a->k_stride, true, "k"},
                    {a->v, a->v_out, a->num_kv_heads, a->v_stride, true, "v"}};
  for (const auto &x : tensors) {
    if (x.heads == 0 || (!x.in && x.kv)) continue;
    if (!x.in || !x.out) return record_error(SV_ERR_INVALID, "rope: null %s or %s_out", x.name, x.name);
    if (!is_aligned16(x.in) || !is_aligned16(x.out))
      return record_error(SV_ERR_INVALID, "rope: %s and %s_out must be 16-byte aligned", x.name, x.name);
    const int64_t width = static_cast<int64_t>(x.heads) * a->head_dim;
    const int64_t stride = x.stride ? x.stride : width;
    if (stride < width || stride * esz % 16 || stride > (int64_t{1} << 40))
      return record_error(SV_ERR_INVALID, "rope: %s row stride %lld (a multiple of 16 bytes, at least %lld)",
                          x.name, static_cast<long long>(stride), static_cast<long long>(width));
    if (x.in == x.out && (stride != width || (x.kv && a->kv_dtype == SV_E4M3)))
      return record_error(SV_ERR_INVALID, "rope: %s in place needs contiguous rows of one dtype", x.name);
  }
  return SV_OK;
}

}  // namespace

}  // namespace sv

extern "C" {

SV_API sv_status spec_rope_rows(const sv_rope_args *a, void *stream) {
  using namespace sv;
  const sv_status st = check_rope(a);
  if (st != SV_OK) return st;
  RopeParams P{};
  P.batch = a->batch;
  P.max_q_rows = a->max_q_rows;
  P.Hq = a->num_q_heads;
  P.Hkv = a->num_kv_heads;
  P.D = a->head_dim;
  P.rot = a->rot_dim;
  P.num_rows = a->num_rows;
  // Every sequence has max_q_rows slots, as in a step, unless most would stay
  // empty (prompts of different lengths): then a row searches its sequence.
  P.slots = a->positions ? a->num_rows : static_cast<int64_t>(a->batch) * a->max_q_rows;
  P.by_row = !a->positions && a->max_q_rows > 16 && P.slots > a->num_rows + a->num_rows / 4;
  if (P.by_row) P.slots = a->num_rows;
  const int64_t D = a->head_dim;
  P.q_stride = a->q_stride ? a->q_stride : P.Hq * D;
  P.k_stride = a->k_stride ? a->k_stride : P.Hkv * D;
  P.v_stride = a->v_stride ? a->v_stride : P.Hkv * D;
  P.mscale = a->mscale == 0.0f ? 1.0f : a->mscale;
  P.k_scale = a->k_scale == 0.0f ? 1.0f : a->k_scale;
  P.v_scale = a->v_scale == 0.0f ? 1.0f : a->v_scale;
  auto inverse = [](float x) {
    int e;
    const float inv = 1.0f / x;
    return std::frexp(x, &e) == 0.5f && std::isnormal(inv) ? inv : 0.0f;
  };
  P.k_inverse = inverse(P.k_scale);
  P.v_inverse = inverse(P.v_scale);
  P.turns = a->turns;
  P.cu_q = a->cu_q;
  P.kv_len = a->kv_len;
  P.positions = a->positions;
  P.q = a->q;
  P.k = a->k;
  P.v = a->v;
  P.q_out = a->q_out;
  P.k_out = a->k_out;
  P.v_out = a->v_out;
  P.dev_status = a->dev_status;
  P.nq = P.Hq;
  P.nk = a->k ? P.Hkv : 0;
  P.heads = P.nq + P.nk + (a->v && a->v != a->v_out ? P.Hkv : 0);   // v onto itself: nothing to do
  if (a->num_rows == 0 || P.slots == 0 || P.heads == 0) return SV_OK;

  const int half = P.rot / 2;
  int g = P.rot % 16 ? kMixed : kNeighbor;
  P.columns = (P.D + 15) / 16;
  if (a->layout == SV_ROPE_HALF) {
    g = half % 8 == 0 ? 8 : half % 4 == 0 ? 4 : half % 2 == 0 ? 2 : 1;
    P.columns = half / g + (P.D - P.rot + 2 * g - 1) / (2 * g);
  }
  const int sms = device_sms();
  if (sms <= 0) return record_error(SV_ERR_CUDA, "rope: no current CUDA device");
  // A pass is one head per P.columns threads; a CTA makes as many as leave about
  // two CTAs per SM (576 rows of 48 heads, E4M3: one pass 6.9 us, all heads 3.8
  // us; 8 rows of 96 heads: 2.3 against 2.7 us).  Its rows lie side by side: two,
  // or, once pairs of rows fill the SMs, as many as about kPasses heads per
  // thread give (1152 rows of 48 heads, E4M3: 7.5 against 6.7 us; 2210 fp32 rows of
  // 12 heads of 64: 5.6 against 4.0 us).
  const int64_t threads = P.slots * P.heads * P.columns, room = 512 * static_cast<int64_t>(sms);
  P.row_shift = 7;
  const int resident = a->kv_dtype == SV_E4M3 || a->dtype == SV_F32 ? 3 : 4;   // CTAs per SM (min_ctas)
  if (P.slots > 2 * resident * static_cast<int64_t>(sms))
    for (P.row_shift = 4; P.row_shift < 7 && ((1 << P.row_shift) < P.columns || (kPasses << P.row_shift) < P.heads * P.columns);)
      ++P.row_shift;
  P.per_column = 65536 / P.columns + 1;
  P.pairs = (half + 7) / 4 * 4;
  const int at_once = (1 << P.row_shift) / P.columns;
  P.heads_per_cta = static_cast<int>(std::min<int64_t>(P.heads, std::max<int64_t>(1, (threads + room - 1) / room) * at_once));
  const int rows_per_cta = kNT >> P.row_shift;
  const dim3 grid(static_cast<unsigned>((P.slots + rows_per_cta - 1) / rows_per_cta),
                  static_cast<unsigned>((P.heads + P.heads_per_cta - 1) / P.heads_per_cta));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool kv8 = a->kv_dtype == SV_E4M3;
  const cudaError_t e =
      a->dtype == SV_BF16
          ? (kv8 ? launch_shape<uint16_t, true>(g, grid, P, s) : launch_shape<uint16_t, false>(g, grid, P, s))
          : (kv8 ? launch_shape<float, true>(g, grid, P, s) : launch_shape<float, false>(g, grid, P, s));
  if (e != cudaSuccess) return record_error(SV_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

SV_API sv_status sv_rope_turns(const sv_rope_scaling *sc, int32_t rot_dim, uint64_t *turns,
                               float *mscale) {
  using sv::record_error;
  if (!sc || !turns) return record_error(SV_ERR_INVALID, "rope turns: null argument");
  if (rot_dim < 2 || rot_dim > sv::kMaxDim || rot_dim % 2)
    return record_error(SV_ERR_INVALID, "rope turns: rot_dim %d (even, 2..%d)", rot_dim, sv::kMaxDim);
  if (sc->kind < SV_ROPE_PLAIN || sc->kind > SV_ROPE_BANDED)
    return record_error(SV_ERR_INVALID, "rope turns: kind %d", sc->kind);
  if (!std::isfinite(sc->base) || !(sc->base > 1.0))
    return record_error(SV_ERR_INVALID, "rope turns: base must be finite and > 1");
  const double factor = sc->kind == SV_ROPE_PLAIN ? 1.0 : sc->factor;
  if (!std::isfinite(factor) || !(factor >= 1.0))
    return record_error(SV_ERR_INVALID, "rope turns: factor must be finite and >= 1");
  const double two_pi = 2.0 * 3.14159265358979323846;
  const double rot = rot_dim, L = sc->trained_len;
  double base = sc->base, m = 1.0, lo = 0.0, hi = 0.0, low = 0.0, high = 0.0;
  if ((sc->kind == SV_ROPE_YARN || sc->kind == SV_ROPE_BANDED) && sc->trained_len < 1)
    return record_error(SV_ERR_INVALID, "rope turns: trained_len %d", sc->trained_len);
  if (sc->kind == SV_ROPE_NTK && rot_dim > 2) base *= std::pow(factor, rot / (rot - 2.0));
  if (!std::isfinite(base)) return record_error(SV_ERR_INVALID, "rope turns: scaled base overflows");
  if (sc->kind == SV_ROPE_YARN) {
    const double fast = sc->beta_fast == 0.0 ? 32.0 : sc->beta_fast;
    const double slow = sc->beta_slow == 0.0 ? 1.0 : sc->beta_slow;
    if (!std::isfinite(fast) || !(slow > 0.0) || !(fast >= slow))
      return record_error(SV_ERR_INVALID, "rope turns: beta_fast >= beta_slow > 0 wanted");
    // the pair that makes n turns over L positions: base^(-2 p / rot) L = 2 pi n
    lo = std::fmax(std::floor(rot * std::log(L / (fast * two_pi)) / (2.0 * std::log(base))), 0.0);
    hi = std::fmin(std::ceil(rot * std::log(L / (slow * two_pi)) / (2.0 * std::log(base))), rot - 1.0);
    m = 0.1 * std::log(factor) + 1.0;
  }
  if (sc->kind == SV_ROPE_BANDED) {
    low = sc->low_freq == 0.0 ? 1.0 : sc->low_freq;
    high = sc->high_freq == 0.0 ? 4.0 : sc->high_freq;
    if (!std::isfinite(high) || !(low > 0.0) || !(high > low))
      return record_error(SV_ERR_INVALID, "rope turns: high_freq > low_freq > 0 wanted");
  }
  for (int p = 0; p < rot_dim / 2; ++p) {
    double f = std::pow(base, -2.0 * p / rot);
    if (sc->kind == SV_ROPE_LINEAR) f /= factor;
    if (sc->kind == SV_ROPE_YARN) {
      const double ramp = std::fmin(std::fmax((p - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    if (sc->kind == SV_ROPE_BANDED) {
      const double keep = std::fmin(std::fmax((L * f / two_pi - low) / (high - low), 0.0), 1.0);
      f = f / factor * (1.0 - keep) + f * keep;
    }
    turns[p] = static_cast<uint64_t>(std::nearbyint(std::ldexp(f / two_pi, 64)));   // < 2^62: f <= 1
  }
  if (mscale) *mscale = static_cast<float>(m);
  return SV_OK;
}

}  // extern "C"
