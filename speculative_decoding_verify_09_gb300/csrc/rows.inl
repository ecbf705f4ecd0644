// What the kernels over ragged rows of heads share: vectors of elements, E4M3
// codes, and how a slot of a launch finds its row and position.
//
// Params of find_row and good_sequence: batch, max_q_rows, num_rows, slots,
// by_row, cu_q, kv_len, positions (nullptr: by cu_q and kv_len).
#pragma once

#include "common.cuh"

namespace sv {

namespace {

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
template <typename Params>
__device__ __forceinline__ bool good_sequence(const Params &P, int i) {
  const int r0 = P.cu_q[i], r1 = P.cu_q[i + 1];
  return r0 >= 0 && r1 >= r0 && r1 <= P.num_rows && r1 - r0 <= P.max_q_rows && P.kv_len[i] >= 0;
}

// Row and position of slot `slot`; false if there is no such row (or a bad one).
template <typename Params>
__device__ __forceinline__ bool find_row(const Params &P, int64_t slot, int64_t &row, int64_t &pos,
                                         bool &bad, int *sequence = nullptr) {
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
  if (sequence != nullptr) *sequence = i;
  row = r0 + j;
  pos = static_cast<int64_t>(L) + j;
  return true;
}

}  // namespace

}  // namespace sv
