/*
 * spec_kv4.h -- C ABI of the per-head norms and of the paged 4-bit KV cache
 * (sm_103a).
 *
 * The unpaged pool of spec_verify.h holds K and V in fp32, bf16 or E4M3.  The
 * cache here holds them in 4 bits, in pages that a block table gives to
 * sequences: a token's K and V rows of 128 elements take 144 bytes per KV head
 * against 512 in bf16, and attention, which reads them all for every step, is
 * bound by those bytes.
 *
 *   spec_norm_rope_rows   RMS norms of the q and k heads and rotary positions in
 *                         one pass, to contiguous rows (for the unpaged pool)
 *   spec_kv4_append       the same (norms optional), k and v into the pages
 *   spec_kv4_attn         attention of the block's rows over the pages
 *   spec_kv4_read         rows of the pages as contiguous rows
 *
 * One step of a batch over the pages is, in order on one stream:
 *   spec_kv4_append, spec_kv4_attn, spec_adjust_logits, spec_reject_sample,
 * and kv_len[i] += num_accepted[i] + 1 (which is + 0 for a failed sequence).
 * The whole block enters the pages before attention reads them; rows of
 * rejected drafts stay behind the new length and the next step writes over
 * them, so nothing is copied after the decision.
 *
 * Conventions are those of spec_verify.h and spec_ops.h: [dev] pointers,
 * caller-owned buffers, calls asynchronous on `stream`, host-checkable errors
 * returned as a status with sv_last_error() and nothing launched, data-dependent
 * problems as bits OR-ed into *dev_status (may be NULL).  All calls can be
 * captured into a graph.  Nothing may overlap except where an argument says so.
 */
#ifndef SPEC_KV4_H
#define SPEC_KV4_H

#include "spec_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SV_KV4_VERSION 1

/* ------------------------------------------------------------------- cache
 * An element x of K (V) is an E2M1 code c times the E4M3 scale s of its 16
 * elements times k_scale (v_scale): x = (c * s) * k_scale.  E2M1 values are 0,
 * .5, 1, 1.5, 2, 3, 4, 6 for the codes' lower three bits 0..7, negative with
 * bit 3.  c * s has six significant bits: exact in bf16 and f16.
 *
 * A page holds page_size tokens of all KV heads as page_size / 16 slabs per
 * head.  A slab is 18 * D bytes, for 16 tokens in order:
 *   K codes   [16, D / 2]   element 2 n in the lower, 2 n + 1 in the upper 4 bits
 *   K scales  [16, D / 16]
 *   V codes   [16, D / 2]
 *   V scales  [16, D / 16]
 * Token t of sequence i is in page table[i, t / page_size].  Pages may be shared
 * by sequences that only read them (prefixes). */
typedef struct sv_kv4_cache {
  int32_t num_kv_heads;     /* Hkv, 1..1024 */
  int32_t head_dim;         /* D: 64 or 128 */
  int32_t page_size;        /* tokens: a multiple of 16, 16..4096 */
  int32_t max_pages;        /* columns of the table, >= 0 */
  int64_t num_pages;        /* pages in the pool, 1..2^31-1 */
  int64_t table_stride;     /* elements between table rows; 0 -> max_pages */
  float k_scale;            /* in [2^-64, 2^64]; 0 -> 1 */
  float v_scale;            /* in [2^-64, 2^64]; 0 -> 1 */
  void *pages;              /* [dev] [num_pages, Hkv, page_size / 16, 18 * D] bytes,
                               16-byte aligned */
  const int32_t *table;     /* [dev] [B, max_pages] page of each page_size tokens;
                               entries that no token needs may hold anything */
} sv_kv4_cache;

/* ------------------------------------------------------------------- norms
 * y = x / sqrt(mean(x^2) + eps) * (weight + weight_offset) over the D elements
 * of a head, before the rotation. */
typedef struct sv_norm_args {
  const float *q_weight;    /* [dev] [D]; NULL: q is not normed */
  const float *k_weight;    /* [dev] [D]; NULL: k is not normed */
  float eps;                /* >= 0, finite */
  float weight_offset;      /* finite; 1 for weights kept as differences from 1 */
} sv_norm_args;

/* spec_rope_rows (whose contract holds for all else) with norms in front of the
 * rotation.  rope.turns may be NULL: norms only (rot_dim is then ignored, cu_q
 * and kv_len, or positions, still say which rows there are).  All arithmetic in
 * fp32, rounded once to the output type; sums of squares in fp32 (a head whose sum
 * passes fp32's range comes out as zeros).  A row of zeros with eps 0 is NaN.  Weights 4-byte aligned. */
typedef struct sv_norm_rope_args {
  sv_rope_args rope;
  sv_norm_args norm;
} sv_norm_rope_args;

SV_API sv_status spec_norm_rope_rows(const sv_norm_rope_args *args, void *stream);

/* ------------------------------------------------------------------ append
 * Row j of sequence i becomes token kv_len[i] + j of its pages: k normed (where
 * k_weight is given) and rotated (where rows.turns is), v as it is, both then
 * quantized: with f the tensor's scale and m the largest magnitude of 16
 * elements,
 *   s = e4m3(m / (6 f)),   c = e2m1(x / (s f)),
 * both rounded to nearest even and saturating, of fp32 quotients; where s is 0 the
 * codes are 0.  16 elements with a NaN among them get a scale of NaN.  q goes to q_out as in
 * spec_norm_rope_rows (num_q_heads 0: none). */
typedef struct sv_kv4_append_args {
  sv_rope_args rows;        /* q, k, v, q_out, positions by cu_q and kv_len (positions
                               NULL), rotation; k_out, v_out, kv_dtype, k_scale and
                               v_scale are ignored; num_kv_heads and head_dim are
                               the cache's, k and v both given */
  sv_norm_args norm;
  sv_kv4_cache cache;
} sv_kv4_append_args;

/* A sequence whose cu_q / kv_len disagree with the host bounds is left unwritten
 * with SV_DEV_BAD_LENGTH, rows behind the table's last page with
 * SV_DEV_CAPACITY and rows whose page is outside [0, num_pages) with
 * SV_DEV_BAD_PARAM are not stored (their q_out is written).  Where cu_q does not
 * ascend, rows of other sequences may be left unwritten too.  Two sequences may not
 * append to the same page's same tokens. */
SV_API sv_status spec_kv4_append(const sv_kv4_append_args *args, void *stream);

/* -------------------------------------------------------------------- read
 * Row j of sequence i of the outputs is token kv_len[i] + j of its pages. */
typedef struct sv_kv4_read_args {
  sv_kv4_cache cache;
  int32_t batch;            /* B >= 0 */
  int32_t max_q_rows;       /* host bound on the rows of one sequence, >= 1;
                               B * max_q_rows < 2^31 */
  int32_t dtype;            /* SV_BF16, SV_F32 or SV_E4M3: k_out and v_out */
  int32_t reserved;         /* 0 */
  int64_t num_rows;         /* R, 0..2^31-1 */
  float k_out_scale;        /* SV_E4M3: code = round(k / k_out_scale); 0 -> 1 */
  float v_out_scale;        /* 0 -> 1 */
  const int32_t *cu_q;      /* [dev] [B+1] */
  const int32_t *kv_len;    /* [dev] [B] */
  void *k_out;              /* [dev] [R, Hkv, D], 16-byte aligned; NULL: V only */
  void *v_out;              /* [dev] [R, Hkv, D], 16-byte aligned; NULL: K only */
  uint32_t *dev_status;     /* [dev] one word or NULL */
} sv_kv4_read_args;

/* fp32 rows are the values' products rounded to fp32, bf16 rows and E4M3 codes (as
 * in spec_rope_rows) are those rounded; with factors that are powers of two the
 * first are exact, and in bf16 too.  Rows that spec_kv4_append would
 * not store (bad lengths, behind the table, bad pages) are left unwritten with the
 * same bits. */
SV_API sv_status spec_kv4_read(const sv_kv4_read_args *args, void *stream);

/* --------------------------------------------------------------- attention
 * out[row j of sequence i, head h] = softmax(scale * q . K^T) V over tokens
 * 0 .. kv_len[i] + j of the pages, KV head h / (Hq / Hkv): the block's own rows
 * have to be in the pages already.  A draft position or plain decoding is the
 * case of one row per sequence. */
typedef struct sv_kv4_attn_args {
  sv_kv4_cache cache;
  int32_t batch;            /* B, 0..768 */
  int32_t num_q_heads;      /* Hq, a multiple of Hkv; Hq / Hkv <= 256 */
  int32_t max_q_rows;       /* host bound on R_i, 1..1024; times Hq / Hkv <= 16384 */
  int32_t dtype;            /* SV_BF16: q and out */
  int64_t num_rows;         /* R */
  int64_t q_stride;         /* elements from one q row to the next; 0 -> Hq * D */
  float scale;              /* 0 -> 1 / sqrt(D) */
  int32_t reserved;         /* 0 */
  const int32_t *cu_q;      /* [dev] [B+1] rows of sequence i (may be none) */
  const int32_t *kv_len;    /* [dev] [B] tokens before the block */
  const void *q;            /* [dev] [R, Hq, D] rows q_stride apart, 16-byte aligned */
  void *out;                /* [dev] [R, Hq, D], 16-byte aligned */
  uint32_t *dev_status;     /* [dev] one word or NULL */
} sv_kv4_attn_args;

/* Bytes of workspace that spec_kv4_attn needs for these shapes (cu_q, kv_len and
 * tensors are not read); 0 with sv_last_error() where they are refused.  A
 * workspace is 256-byte aligned, zeroed once (sv_workspace_init) and kept to
 * spec_kv4_attn; any shapes that fit may take turns on it, in stream order, also
 * from graphs.  Every completed call leaves its counters zero; after
 * SV_DEV_TIMEOUT it is zeroed again. */
SV_API size_t sv_kv4_workspace_bytes(const sv_kv4_attn_args *args);

/* q is rounded to f16, exact for bf16 values from 2^-17 to 65504.  Smaller ones are
 * off by up to 2^-25; where scale * k_scale * head_dim passes 16, so that this could
 * show, rows and heads below 2^15 are multiplied by a power of two first, and elements
 * are off by up to 2^-40 of the largest.  Beyond +-65504 q becomes infinite and its own
 * row and head non-finite.  Scores and sums are fp32; weights are
 * rounded to f16: by 2^-11, or by 2^-32 of the row's largest where that is
 * more (smaller ones are lost).  What tokens that a row does not see hold, be it
 * NaN, does not reach it.  Sequences whose cu_q / kv_len disagree with the host
 * bounds (SV_DEV_BAD_LENGTH) or whose tokens pass the table (SV_DEV_CAPACITY) are
 * left unwritten; one with a page outside [0, num_pages) gets NaN in the rows of
 * the parts it was needed for, with SV_DEV_BAD_PARAM.  A score that passes fp32's
 * range makes its row and head non-finite.  The max_q_rows * Hq / Hkv rows that a
 * block has per KV head go in parts of 16 (up to 24: one part), each with its own
 * pass over the tokens; B * Hkv times the parts may not pass 65536. */
SV_API sv_status spec_kv4_attn(const sv_kv4_attn_args *args, void *ws, size_t ws_bytes, void *stream);

/* SV_KV4_VERSION of the loaded library. */
SV_API int32_t sv_kv4_version(void);

/* sizeof(sv_kv4_cache), sv_norm_args, sv_norm_rope_args, sv_kv4_append_args,
 * sv_kv4_read_args, sv_kv4_attn_args for which = 0..5 (lets a binding check its
 * mirrors). */
SV_API size_t sv_kv4_struct_size(int32_t which);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_KV4_H */
