// The 4-bit cache format on the device: E2M1 codes, their scales, and where a
// token's rows are (spec_kv4.h has the layout).
#pragma once

#include "common.cuh"
#include "spec_kv4.h"

namespace sv {

constexpr int kSlab = 16;                            // tokens of a slab

// Bytes of a slab of one KV head, and where its parts begin.
__host__ __device__ constexpr int slab_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int slab_k_scales(int D) { return 8 * D; }
__host__ __device__ constexpr int slab_v(int D) { return 9 * D; }

// What a kernel needs of sv_kv4_cache.
struct Kv4View {
  uint8_t *pages;
  const int32_t *table;
  int64_t table_stride, num_pages;
  int32_t max_pages, page_size, slabs, heads, D;     // slabs of a page; KV heads
  float k_scale, v_scale;
};

// Bytes from one KV head's slabs of a page to the next head's.
__device__ __forceinline__ int64_t head_bytes(const Kv4View &c) {
  return static_cast<int64_t>(c.slabs) * slab_bytes(c.D);
}

// Where token `pos` (0 .. 2^32 - 1) of sequence i is, in two steps: its page is asked for,
// then its slab (of KV head 0) found: nullptr with the problem's bit in *why.
struct Kv4Spot {
  uint32_t slab;                                     // of the page
  int32_t page;
  bool in_table;
};
__device__ __forceinline__ Kv4Spot find_page(const Kv4View &c, int i, int64_t pos) {
  const uint32_t slab = static_cast<uint32_t>(pos) / kSlab, at = slab / static_cast<uint32_t>(c.slabs);
  Kv4Spot s;
  s.slab = slab - at * c.slabs;
  s.in_table = at < static_cast<uint32_t>(c.max_pages);
  s.page = s.in_table ? c.table[i * c.table_stride + at] : 0;
  return s;
}
__device__ __forceinline__ uint8_t *find_slab(const Kv4View &c, const Kv4Spot &s, uint32_t *why) {
  if (!s.in_table) {
    *why = SV_DEV_CAPACITY;
    return nullptr;
  }
  if (s.page < 0 || s.page >= c.num_pages) {
    *why = SV_DEV_BAD_PARAM;
    return nullptr;
  }
  return c.pages + s.page * (c.heads * head_bytes(c)) + static_cast<int64_t>(s.slab) * slab_bytes(c.D);
}

// Four bytes of code pairs -> four f16x2 (a byte's lower code in the lower half).
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t codes, uint32_t (&h)[4]) {
  asm("{.reg .b8 b0, b1, b2, b3;\n"
      "mov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
      "cvt.rn.f16x2.e2m1x2 %3, b3;}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

// Eight floats -> their codes, nearest even, saturating; element n in bits 4 n.
__device__ __forceinline__ uint32_t e2m1x8_of(const float (&x)[8]) {
  uint32_t r;
  asm("{.reg .b8 b0, b1, b2, b3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      "mov.b32 %0, {b0, b1, b2, b3};}\n"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

__device__ __forceinline__ float f16_bits_to_f32(uint32_t h) {
  float r;
  asm("cvt.f32.f16 %0, %1;\n" : "=f"(r) : "h"(static_cast<uint16_t>(h)));
  return r;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t code) {
  return f16_bits_to_f32(e4m3x2_to_f16x2(code));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// D = A * B + D, m16n8k16, f16 inputs, fp32 accumulators; may be moved by the compiler.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two f16 -> two E4M3 codes (in order), nearest even, saturating.
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(h));
  return r;
}

// The largest of three; NaN if any is.
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Host: checks of sv_kv4_cache in the name of entry point `who`, and its view.
sv_status check_cache(const sv_kv4_cache *c, const char *who);
Kv4View view_of(const sv_kv4_cache &c);

}  // namespace sv
