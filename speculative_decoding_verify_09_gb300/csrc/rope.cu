// Rotary positions of ragged rows, fused with the E4M3 quantization of K and V
// (sm_103a).  Contract: spec_rope_rows in include/spec_ops.h.
//
// Pair (a, b) of a row at position t becomes m (a cos x - b sin x, b cos x + a
// sin x), x = t f_p.  What has to be exact is x modulo a turn: at t = 2^20 an
// fp32 product is off by 2^-4 radians.  f_p / (2 pi) is kept as a 64-bit
// fraction of a turn, so t times it modulo 2^64 -- one integer multiplication
// -- is the exact fraction of a turn (up to t * 2^-65 from rounding f_p), whose
// signed value feeds sincospif.
//
// The kernel is one pass over the rows: bytes bound for prompts, launch bound
// for a step's rows.  A row's cos and sin are computed once per CTA into shared
// memory (rot_dim / 2 pairs, one per thread), while the first 16-byte vectors
// of the row are in flight, and each thread keeps the pairs of its vector
// column in registers over all heads of the row.
#include <cmath>

#include "common.cuh"
#include "ops_host.inl"
#include "spec_ops.h"

namespace sv {

namespace {

constexpr int kNT = 256;
constexpr int kMaxDim = 256;
constexpr int kMinRowThreads = 64;                   // threads that share one row, at least
constexpr int kMaxRows = kNT / kMinRowThreads;       // rows per CTA, at most

// How a thread's 8 elements (or two times 8) of a head meet their partners.
enum Shape {
  kHalf = 0,      // half layout, rot_dim % 16 == 0 and D % 16 == 0: a thread holds the vectors
                  // at 8 c and 8 c + rot_dim / 2, i.e. 8 whole pairs
  kNeighbor = 1,  // interleaved: a vector holds 4 whole pairs
  kRagged = 2     // half layout otherwise: a vector's partners are read one by one (L1 hits)
};

struct RopeParams {
  int batch, max_q_rows, Hq, Hkv, D, rot;
  int nq, nk, heads;            // q heads, k heads, all heads of a row (q, k, then v)
  int gshift, row_shift;        // log2 threads per head, per row
  int heads_per_cta;
  int64_t num_rows, slots;
  int64_t q_stride, k_stride, v_stride;
  float mscale, k_scale, v_scale;
  const uint64_t *turns;
  const int32_t *cu_q, *kv_len;
  const int64_t *positions;
  const void *q, *k, *v;
  void *q_out, *k_out, *v_out;
  uint32_t *dev_status;
};

template <typename T>
struct Vec8;                    // 8 elements as they lie in memory
template <>
struct Vec8<uint16_t> {         // bf16
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t *p) { w = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<uint4 *>(p) = w; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    w = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
  }
  static __device__ __forceinline__ float one(const uint16_t *p) { return bf16_bits_to_f32(*p); }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void store(float *p) const {
    reinterpret_cast<float4 *>(p)[0] = a;
    reinterpret_cast<float4 *>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
  static __device__ __forceinline__ float one(const float *p) { return *p; }
};

// Two floats -> two E4M3 codes (lo in the lower byte), nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void store_codes(uint8_t *p, const float (&x)[8], float scale) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = e4m3x2_of(x[2 * i] / scale, x[2 * i + 1] / scale);
  *reinterpret_cast<uint2 *>(p) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
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
  const int i = static_cast<int>(static_cast<uint32_t>(slot) / static_cast<uint32_t>(P.max_q_rows));
  const int j = static_cast<int>(slot) - i * P.max_q_rows;
  const int r0 = P.cu_q[i], r1 = P.cu_q[i + 1], L = P.kv_len[i];
  if (r0 < 0 || r1 < r0 || r1 > P.num_rows || r1 - r0 > P.max_q_rows || L < 0) {
    bad = true;
    return false;
  }
  if (j >= r1 - r0) return false;
  row = r0 + j;
  pos = static_cast<int64_t>(L) + j;
  return true;
}

template <typename T, int SHAPE, bool KV8>
__global__ void __launch_bounds__(kNT) rope_kernel(const RopeParams P) {
  __shared__ __align__(16) float s_cos[kMaxRows][kMaxDim / 2 + 4];
  __shared__ __align__(16) float s_sin[kMaxRows][kMaxDim / 2 + 4];
  const int row_threads = 1 << P.row_shift;
  const int rl = threadIdx.x >> P.row_shift, t = threadIdx.x & (row_threads - 1);
  const int c = t & ((1 << P.gshift) - 1), hl = t >> P.gshift;
  const int hstep = row_threads >> P.gshift;
  const int h_begin = blockIdx.y * P.heads_per_cta;
  const int h_end = min(P.heads, h_begin + P.heads_per_cta);
  const int iters = (h_end - h_begin + hstep - 1) / hstep;
  const int half = P.rot >> 1;

  int64_t row = 0, pos = 0;
  bool bad;
  const bool live = find_row(P, static_cast<int64_t>(blockIdx.x) * (kNT >> P.row_shift) + rl, row,
                             pos, bad);
  if (bad && t == 0 && blockIdx.y == 0) set_status(P.dev_status, SV_DEV_BAD_LENGTH);

  // this thread's vector column: element offsets inside a head
  constexpr int NV = SHAPE == kHalf ? 2 : 1;
  const bool column = live && c < P.D / (8 * NV);
  const bool turn = SHAPE != kHalf || c < P.rot / 16;    // (kHalf) the column holds pairs
  const int o0 = SHAPE == kHalf ? (turn ? 8 * c : P.rot + 16 * (c - P.rot / 16)) : 8 * c;
  const int o1 = SHAPE == kHalf ? (turn ? o0 + half : o0 + 8) : 0;

  Vec8<T> cur[NV], nxt[NV];
  float pcur[8], pnxt[8];                                // (kRagged) the partners
  auto source = [&](int h) -> const T * {
    if (h < P.nq) return static_cast<const T *>(P.q) + row * P.q_stride + static_cast<int64_t>(h) * P.D;
    h -= P.nq;
    if (h < P.nk) return static_cast<const T *>(P.k) + row * P.k_stride + static_cast<int64_t>(h) * P.D;
    return static_cast<const T *>(P.v) + row * P.v_stride + static_cast<int64_t>(h - P.nk) * P.D;
  };
  auto fetch = [&](Vec8<T> (&v)[NV], float (&pv)[8], int h) {
    if (!column || h >= h_end) return;
    const T *p = source(h);
    v[0].load(p + o0);
    if constexpr (NV == 2) v[1].load(p + o1);
    if constexpr (SHAPE == kRagged) {
      if (h < P.nq + P.nk) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = o0 + i;
          pv[i] = e < P.rot ? Vec8<T>::one(p + (e < half ? e + half : e - half)) : 0.0f;
        }
      }
    }
  };
  fetch(cur, pcur, h_begin + hl);

  // cos and sin of the row's pairs, by the threads that share the row
  if (live && h_begin < P.nq + P.nk) {
    for (int p = t; p < half; p += row_threads) {
      const uint64_t part = static_cast<uint64_t>(pos) * __ldg(P.turns + p);
      float sn, cs;
      sincospif(__ll2float_rn(static_cast<int64_t>(part)) * 0x1p-63f, &sn, &cs);
      s_cos[rl][p] = cs * P.mscale;
      s_sin[rl][p] = sn * P.mscale;
    }
  }
  __syncthreads();

  // the pairs of this column
  constexpr int NP = SHAPE == kNeighbor ? 4 : 8;
  float cs[NP], sn[NP];
  if (column && h_begin < P.nq + P.nk) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      int p;                                             // pair, or >= half: none
      if constexpr (SHAPE == kHalf) p = turn ? 8 * c + i : half;
      if constexpr (SHAPE == kNeighbor) p = 4 * c + i;
      if constexpr (SHAPE == kRagged) {
        const int e = 8 * c + i;
        p = e < half ? e : e < P.rot ? e - half : half;
      }
      cs[i] = p < half ? s_cos[rl][p] : 1.0f;
      sn[i] = p < half ? s_sin[rl][p] : 0.0f;
    }
  }

  for (int it = 0; it < iters; ++it) {
    const int h = h_begin + hl + it * hstep;
    fetch(nxt, pnxt, h + hstep);
    // kRagged in place: every lane of a head has read before one of them writes
    if constexpr (SHAPE == kRagged) __syncwarp();
    if (column && h < h_end) {
      const bool rotated = h < P.nq + P.nk, is_q = h < P.nq;
      float x[8], y[8];
      if (rotated) {
        cur[0].get(x);
        if constexpr (SHAPE == kHalf) {
          if (turn) {
            float b[8];
            cur[1].get(b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              y[i] = b[i] * cs[i] + x[i] * sn[i];
              x[i] = x[i] * cs[i] - b[i] * sn[i];
            }
            if (!KV8 || is_q) {
              cur[0].set(x);
              cur[1].set(y);
            }
          } else if (KV8 && !is_q) {
            cur[1].get(y);
          }
        }
        if constexpr (SHAPE == kNeighbor) {
          if (8 * c < P.rot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[2 * i], b = x[2 * i + 1];
              if (4 * c + i < half) {
                x[2 * i] = a * cs[i] - b * sn[i];
                x[2 * i + 1] = b * cs[i] + a * sn[i];
              }
            }
            if (!KV8 || is_q) cur[0].set(x);
          }
        }
        if constexpr (SHAPE == kRagged) {
          if (8 * c < P.rot) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int e = 8 * c + i;
              if (e < half) x[i] = x[i] * cs[i] - pcur[i] * sn[i];
              else if (e < P.rot) x[i] = x[i] * cs[i] + pcur[i] * sn[i];
            }
            if (!KV8 || is_q) cur[0].set(x);
          }
        }
      } else if (KV8) {
        cur[0].get(x);
        if constexpr (NV == 2) cur[1].get(y);
      }
      if (KV8 && !is_q) {
        const bool is_k = h < P.nq + P.nk;
        const int hk = h - P.nq - (is_k ? 0 : P.nk);
        uint8_t *o = static_cast<uint8_t *>(is_k ? P.k_out : P.v_out) +
                     (row * P.Hkv + hk) * static_cast<int64_t>(P.D);
        const float scale = is_k ? P.k_scale : P.v_scale;
        store_codes(o + o0, x, scale);
        if constexpr (NV == 2) store_codes(o + o1, y, scale);
      } else {
        T *o;
        if (is_q) {
          o = static_cast<T *>(P.q_out) + (row * P.Hq + h) * static_cast<int64_t>(P.D);
        } else {
          const bool is_k = h < P.nq + P.nk;
          const int hk = h - P.nq - (is_k ? 0 : P.nk);
          o = static_cast<T *>(is_k ? P.k_out : P.v_out) + (row * P.Hkv + hk) * static_cast<int64_t>(P.D);
        }
        cur[0].store(o + o0);
        if constexpr (NV == 2) cur[1].store(o + o1);
      }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) cur[n] = nxt[n];
    if constexpr (SHAPE == kRagged) {
#pragma unroll
      for (int i = 0; i < 8; ++i) pcur[i] = pnxt[i];
    }
  }
}

template <typename T, bool KV8>
void launch_shape(int shape, dim3 grid, const RopeParams &P, cudaStream_t s) {
  if (shape == kHalf) rope_kernel<T, kHalf, KV8><<<grid, kNT, 0, s>>>(P);
  else if (shape == kNeighbor) rope_kernel<T, kNeighbor, KV8><<<grid, kNT, 0, s>>>(P);
  else rope_kernel<T, kRagged, KV8><<<grid, kNT, 0, s>>>(P);
}

bool positive(float x) { return std::isfinite(x) && x > 0.0f; }

sv_status check_rope(const sv_rope_args *a) {
  auto bad = [](const char *what) { return record_error(SV_ERR_INVALID, "rope: %s", what); };
  if (!a) return bad("null arguments");
  if (a->dtype != SV_F32 && a->dtype != SV_BF16)
    return record_error(SV_ERR_INVALID, "rope: dtype %d", a->dtype);
  if (a->kv_dtype != 0 && a->kv_dtype != SV_E4M3)
    return record_error(SV_ERR_INVALID, "rope: kv_dtype %d (0 or SV_E4M3)", a->kv_dtype);
  if (a->num_q_heads < 0 || a->num_q_heads > 65535 || a->num_kv_heads < 0 || a->num_kv_heads > 65535)
    return record_error(SV_ERR_INVALID, "rope: heads Hq=%d Hkv=%d outside [0, 65535]",
                        a->num_q_heads, a->num_kv_heads);
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
  P.slots = a->positions ? a->num_rows : static_cast<int64_t>(a->batch) * a->max_q_rows;
  const int64_t D = a->head_dim;
  P.q_stride = a->q_stride ? a->q_stride : P.Hq * D;
  P.k_stride = a->k_stride ? a->k_stride : P.Hkv * D;
  P.v_stride = a->v_stride ? a->v_stride : P.Hkv * D;
  P.mscale = a->mscale == 0.0f ? 1.0f : a->mscale;
  P.k_scale = a->k_scale == 0.0f ? 1.0f : a->k_scale;
  P.v_scale = a->v_scale == 0.0f ? 1.0f : a->v_scale;
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

  const int shape = a->layout == SV_ROPE_INTERLEAVED ? kNeighbor
                    : (P.rot % 16 == 0 && P.D % 16 == 0) ? kHalf : kRagged;
  const int columns = shape == kHalf ? P.D / 16 : P.D / 8;
  while ((1 << P.gshift) < columns) ++P.gshift;
  // Many rows: kMinRowThreads threads per row, so that a thread keeps its pairs'
  // cos and sin over many heads.  Few rows: a CTA per row and share of the heads.
  const int sms = device_sms();
  if (sms <= 0) return record_error(SV_ERR_CUDA, "rope: no current CUDA device");
  const bool few = P.slots < 4 * static_cast<int64_t>(sms);
  P.row_shift = few ? 8 : 6;
  const int at_once = (1 << P.row_shift) >> P.gshift;
  P.heads_per_cta = few ? at_once : P.heads;
  const int rows_per_cta = kNT >> P.row_shift;
  const dim3 grid(static_cast<unsigned>((P.slots + rows_per_cta - 1) / rows_per_cta),
                  static_cast<unsigned>((P.heads + P.heads_per_cta - 1) / P.heads_per_cta));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool kv8 = a->kv_dtype == SV_E4M3;
  if (a->dtype == SV_BF16) {
    if (kv8) launch_shape<uint16_t, true>(shape, grid, P, s);
    else launch_shape<uint16_t, false>(shape, grid, P, s);
  } else {
    if (kv8) launch_shape<float, true>(shape, grid, P, s);
    else launch_shape<float, false>(shape, grid, P, s);
  }
  const cudaError_t e = cudaGetLastError();
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
