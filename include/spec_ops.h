/*
 * spec_ops.h -- C ABI of the operators around a verify step (sm_103a).
 *
 * A verify step (spec_verify.h) takes two things from the target's forward
 * pass, and these operators make them ready for it:
 *   - the block rows' q, k and v enter the attention and the KV cache:
 *     spec_rope_rows rotates q and k at their sequences' own positions and
 *     turns k and v into the codes of an 8-bit cache;
 *   - the block's logits rows enter the rejection sampler: spec_adjust_logits
 *     applies penalties for repeated tokens, biases and grammar masks to the
 *     target and draft rows, each row seeing the drafts before it, and
 *     spec_count_tokens keeps the table of prompt and output tokens that the
 *     penalties read.
 * The speculative-sampling paper (section "Modified rejection sampling") has
 * such changes of the probabilities precede the scheme on both sides, so the
 * target row and the draft row of one position take the same adjustment.
 *
 * One step of a batch is, in order on one stream:
 *   spec_rope_rows, spec_adjust_logits, spec_verify_step, spec_count_tokens
 * (the last with the step's out_tokens and num_accepted).
 *
 * Conventions are those of spec_verify.h: [dev] pointers, caller-owned
 * buffers, calls asynchronous on `stream`, host-checkable errors returned as
 * a status with sv_last_error() and nothing launched, data-dependent problems
 * as bits OR-ed into *dev_status (may be NULL).  These calls need no
 * workspace, keep no state of their own, and can be captured into a graph.
 * Nothing may overlap except where an argument says so.
 */
#ifndef SPEC_OPS_H
#define SPEC_OPS_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SV_OPS_VERSION 1

/* ------------------------------------------------------------------ rotary
 * The first rot_dim elements of every q and k head are rot_dim / 2 pairs;
 * pair p of a row at position t is turned by the angle t * f_p:
 *   a' = m (a cos - b sin),  b' = m (b cos + a sin).
 * SV_ROPE_HALF: a = x[p], b = x[p + rot_dim / 2]; SV_ROPE_INTERLEAVED:
 * a = x[2 p], b = x[2 p + 1].  Elements from rot_dim on are copied.  v rows
 * are copied (or quantized).  Arithmetic in fp32, rounded once to the output
 * type; angles are formed exactly in 64-bit fixed point (below), so far
 * positions lose nothing. */
enum { SV_ROPE_HALF = 0, SV_ROPE_INTERLEAVED = 1 };

typedef struct sv_rope_args {
  int32_t batch;            /* B >= 0 (ignored with positions) */
  int32_t num_q_heads;      /* Hq, 0..16384; 0: no q */
  int32_t num_kv_heads;     /* Hkv, 0..16384; 0: no k and v */
  int32_t head_dim;         /* D: a multiple of 8, 8..256 */
  int32_t rot_dim;          /* even, 2..D */
  int32_t layout;           /* SV_ROPE_HALF or SV_ROPE_INTERLEAVED */
  int32_t dtype;            /* SV_F32 or SV_BF16: q, k, v and q_out */
  int32_t kv_dtype;         /* 0 (k_out, v_out in dtype) or SV_E4M3 codes */
  int64_t num_rows;         /* R rows of q, k and v */
  int32_t max_q_rows;       /* host bound on the rows of one sequence, >= 1;
                               B * max_q_rows < 2^31 (ignored with positions) */
  float mscale;             /* m, the factor on cos and sin; 0 -> 1 */
  float k_scale;            /* E4M3: code = round(k / k_scale); 0 -> 1 */
  float v_scale;            /* E4M3: code = round(v / v_scale); 0 -> 1 */
  int64_t q_stride;         /* elements from one q row to the next; 0 -> Hq * D */
  int64_t k_stride;         /* 0 -> Hkv * D */
  int64_t v_stride;         /* 0 -> Hkv * D */
  const uint64_t *turns;    /* [dev] [rot_dim / 2] f_p / (2 pi) as a fraction of
                               2^64 (sv_rope_turns fills it) */
  const int32_t *cu_q;      /* [dev] [B+1] rows of sequence i: cu_q[i] ..
                               cu_q[i+1]-1 (may be none) */
  const int32_t *kv_len;    /* [dev] [B] row j of sequence i is at kv_len[i] + j */
  const int64_t *positions; /* [dev] [R] or NULL: the rows' positions themselves,
                               instead of cu_q and kv_len; |position| < 2^31.
                               A rotation by -t undoes one by t (but for m^2) and is
                               its transpose: gradients of q_out and k_out go back
                               through the same call with negated positions */
  const void *q;            /* [dev] [R, Hq, D] rows q_stride apart */
  const void *k;            /* [dev] [R, Hkv, D]; NULL: v only */
  const void *v;            /* [dev] [R, Hkv, D]; NULL: none */
  void *q_out;              /* [dev] [R, Hq, D]; may be q itself (contiguous) */
  void *k_out;              /* [dev] [R, Hkv, D]; may be k itself (contiguous, in dtype) */
  void *v_out;              /* [dev] [R, Hkv, D]; may be v itself (contiguous, in dtype) */
  uint32_t *dev_status;     /* [dev] one word or NULL */
} sv_rope_args;

/* Rotates q and k (and quantizes k and v) of every row.  Tensors 16-byte
 * aligned, row strides multiples of 16 bytes and at least a row.  E4M3 codes
 * are rounded to nearest even and saturate at +-448 code values; NaN stays
 * NaN.  A sequence whose cu_q / kv_len are inconsistent with the host bounds,
 * or a row whose position is out of range, is left unwritten with
 * SV_DEV_BAD_LENGTH (with max_q_rows > 16, a cu_q that does not ascend may leave
 * other sequences' rows unwritten too).  Rows behind cu_q[B] stay as they are. */
SV_API sv_status spec_rope_rows(const sv_rope_args *rope, void *stream);

/* Frequencies of the pairs, with the usual changes for contexts longer than
 * the trained one:
 *   SV_ROPE_PLAIN   f_p = base^(-2 p / rot_dim)
 *   SV_ROPE_LINEAR  f_p / factor (positions interpolated)
 *   SV_ROPE_NTK     base * factor^(rot_dim / (rot_dim - 2)) as the base
 *                   (factor unused at rot_dim 2, whose one pair has f = 1)
 *   SV_ROPE_YARN    pairs that make more than beta_fast turns over the trained
 *                   length keep f_p, those below beta_slow take f_p / factor,
 *                   linear in p between the two pairs; m = 0.1 ln(factor) + 1
 *   SV_ROPE_BANDED  by turns over the trained length: above high_freq keep
 *                   f_p, below low_freq f_p / factor, linear between */
enum { SV_ROPE_PLAIN = 0, SV_ROPE_LINEAR = 1, SV_ROPE_NTK = 2, SV_ROPE_YARN = 3, SV_ROPE_BANDED = 4 };

typedef struct sv_rope_scaling {
  int32_t kind;             /* SV_ROPE_PLAIN .. SV_ROPE_BANDED */
  int32_t trained_len;      /* trained context length, >= 1 (YARN, BANDED) */
  double base;              /* > 1 */
  double factor;            /* >= 1; the context is extended by it */
  double beta_fast, beta_slow;   /* YARN: 0 -> 32, 1 */
  double low_freq, high_freq;    /* BANDED: 0 -> 1, 4 */
} sv_rope_scaling;

/* Host only: fills turns[rot_dim / 2] [host] for sv_rope_args.turns (copy it to
 * the device once) and *mscale (may be NULL). */
SV_API sv_status sv_rope_turns(const sv_rope_scaling *scaling, int32_t rot_dim, uint64_t *turns,
                               float *mscale);

/* ----------------------------------------------------------- token counts
 * The table of tokens a sequence has had: counts int32 [num_slots, V] (sign
 * bit: the token is in the prompt; low 31 bits: times it was emitted) and
 * seen uint32 [num_slots, ceil(V / 32)] (bit t % 32 of word t / 32 set where
 * counts[t] is not 0; it lets the readers skip the rest).  Zero both once; only
 * this call changes them from then on. */
enum { SV_COUNT_PROMPT = 1,  /* the tokens are a prompt's: marked, not counted */
       SV_COUNT_RESET = 2 }; /* clear the batch's slots first (new requests) */

typedef struct sv_count_args {
  int32_t batch;            /* B, 0..65535 */
  int32_t vocab;            /* V, 1..2^23 */
  int32_t num_slots;        /* rows of the table, >= 1 */
  int32_t flags;            /* SV_COUNT_* */
  int64_t num_tokens;       /* T, the tokens in `tokens`; 0..2^30 */
  const int32_t *start;     /* [dev] [B+1] tokens of sequence i: start[i] ..
                               start[i+1]-1 (a step's cu_q; may be none) */
  const int32_t *tokens;    /* [dev] [T] (a step's out_tokens) */
  const int32_t *num_accepted; /* [dev] [B] or NULL: only the sequence's first
                               num_accepted[i] + 1 tokens (none if negative),
                               as a step emits them */
  const int32_t *slots;     /* [dev] [B] the sequences' rows of the table, NULL -> i;
                               two sequences may share one; -1: not counted.
                               (With SV_COUNT_RESET sharers are found by a scan of
                               the batch and taken by one CTA each: 0.5 ms for 1024
                               of 64 tokens, 7.6 ms for 16384 of 4) */
  int32_t *counts;          /* [dev] [num_slots, V] */
  uint32_t *seen;           /* [dev] [num_slots, ceil(V / 32)] */
  uint32_t *dev_status;     /* [dev] one word or NULL */
} sv_count_args;

/* Adds the batch's tokens to the table.  A token outside [0, V) is skipped
 * with SV_DEV_BAD_TOKEN, a sequence with a slot outside [-1, num_slots) with
 * SV_DEV_BAD_PARAM.  start values that do not ascend within [0, num_tokens] set
 * SV_DEV_BAD_LENGTH and may leave any of the batch's tokens uncounted (slots are
 * cleared all the same).  Counts are exact up to 2^31 - 1. */
SV_API sv_status spec_count_tokens(const sv_count_args *count, void *stream);

/* ---------------------------------------------------------------- logits
 * Row j of sequence i (block rows as in spec_verify.h) follows the tokens of
 * the table, the ctx tokens and drafts 1..j of its block; n is how often a
 * token was emitted among them, and a token is known if n > 0 or the prompt
 * holds it.  For every token:
 *   known:   l = l > 0 ? l / repetition : l * repetition
 *   n > 0:   l = l - (frequency * n + presence)
 *   biased:  l = l + bias
 *   barred:  l = -inf                (the mask's bit is 0; whatever l was)
 * Each line's result is rounded to nearest in fp32 (the bracket before it, too: one
 * rounding), the last one to the logits' type.  Quotients of l outside [2^-60, 2^60] are
 * within 2^-23 of the exact value instead of 2^-24.
 * Tokens that nothing of this touches keep their bits (a NaN where a later
 * draft's token stands remains some NaN).  Draft row j takes what target row j
 * takes.  A row whose mask bars everything is all -inf (the
 * sampler then fails its sequence with SV_DEV_NONFINITE). */
typedef struct sv_adjust_args {
  int32_t batch;            /* B, 0..65535 */
  int32_t vocab;            /* V, 1..2^23 */
  int32_t dtype;            /* SV_F32 or SV_BF16: all logits */
  int32_t max_q_rows;       /* host bound on R_i, 1..16 */
  int64_t num_rows;         /* R = cu_q[B] (host copy) */
  const int32_t *cu_q;      /* [dev] [B+1] (0..B: single rows, as at a draft position) */
  const void *target;       /* [dev] [R, V] */
  void *target_out;         /* [dev] [R, V]; may be target itself (in place) */
  const void *draft;        /* [dev] [R - B, V] or NULL */
  void *draft_out;          /* [dev] [R - B, V] or NULL; draft itself if and only if
                               target_out is target */
  const int32_t *draft_tokens; /* [dev] [R - B] or NULL: no drafts counted.  Tokens
                               outside [0, V) are not counted (the sampler
                               reports them) */
  /* history */
  const int32_t *counts;    /* [dev] [num_slots, V] or NULL: no table */
  const uint32_t *seen;     /* [dev] [num_slots, ceil(V / 32)] (with counts) */
  int32_t num_slots;        /* rows of the table (0 without one) */
  int32_t num_ctx;          /* ctx tokens per sequence, 0..1024 */
  const int32_t *slots;     /* [dev] [B] rows of the table, NULL -> i; -1: none */
  const int32_t *ctx_tokens;/* [dev] token c of sequence i at [c * ctx_stride + i]: emitted
                               tokens not yet in the table (the drafts so far, at
                               a draft position); outside [0, V): not counted.
                               Meant for some ten: every listed token that is not the
                               table's alone looks at all of them (8 rows of V = 32000:
                               4.6 us with 3, 5.1 with 64, 44 with 1024) */
  int64_t ctx_stride;       /* elements between ctx positions; 0 -> B */
  /* penalties */
  float repetition;         /* in [2^-64, 2^64]; 0 -> 1 (off) */
  float presence;           /* finite */
  float frequency;          /* finite */
  int32_t num_masks;        /* rows of mask (0 without one) */
  const float *repetitions; /* [dev] [B] per-sequence values (not 0) or NULL */
  const float *presences;   /* [dev] [B] or NULL */
  const float *frequencies; /* [dev] [B] or NULL */
  /* biases */
  const int32_t *bias_start;/* [dev] [B+1] entries of sequence i; NULL: none */
  const int32_t *bias_tokens;  /* [dev] [num_bias]; of a token named twice by one
                               sequence the last entry holds */
  const float *bias_values; /* [dev] [num_bias] */
  int64_t num_bias;         /* 0..2^30 */
  /* grammar masks */
  const uint32_t *mask;     /* [dev] [num_masks, mask_stride] bit t % 32 of word t / 32 is 1
                               where token t is allowed; NULL: none */
  int64_t mask_stride;      /* words per row; 0 -> ceil(V / 32) */
  const int32_t *mask_rows; /* [dev] [R] mask row of each block row, -1: none;
                               NULL: row r has mask row r (num_masks >= R) */
  uint32_t *dev_status;     /* [dev] one word or NULL */
} sv_adjust_args;

/* Adjusts the target (and draft) rows.  Logits tensors 16-byte aligned.  A
 * sequence with a bad cu_q is skipped with SV_DEV_BAD_LENGTH (rows unwritten).
 * A sequence with a bad per-sequence value (repetition out of range,
 * presence or frequency not finite), slot, bias range or mask row gets rows of
 * NaN with SV_DEV_BAD_PARAM, so that the sampler fails it too; a bias token
 * outside [0, V) is ignored with SV_DEV_BAD_TOKEN. */
SV_API sv_status spec_adjust_logits(const sv_adjust_args *adjust, void *stream);

/* SV_OPS_VERSION of the loaded library. */
SV_API int32_t sv_ops_version(void);

/* sizeof(sv_rope_args), sv_rope_scaling, sv_count_args, sv_adjust_args for
 * which = 0..3 (lets a binding check its mirrors). */
SV_API size_t sv_ops_struct_size(int32_t which);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_OPS_H */
