/*
 * sparse_step.h - C ABI of the operators around the selection of a
 * sparse-attention step (GB300, sm_103a), in the same library as
 * topk_indexer.h, with its status codes, stream type and conventions:
 *
 *   sparse_rotary          rotary positions on queries and keys, optionally
 *                          written straight into a paged cache
 *   sparse_indexer_scores  the indexer's FP32 scores over a paged key cache
 *                          (the input of topk_ragged / topk_paged)
 *   sparse_attention       attention over the selected entries of a paged
 *                          cache (the consumer of their output)
 *
 * All pointers are DEVICE pointers owned by the caller, all strides are in
 * elements; the stride of a dimension of one element is not used. A call
 * enqueues one kernel on `stream`, allocates nothing, keeps nothing and never
 * synchronises. Invalid arguments, and sizes that would need more than 2^31 - 1
 * work units, return TOPK_EINVAL before anything is enqueued, a device other
 * than sm_103 TOPK_EDEVICE, a failing CUDA call TOPK_ECUDA. Waits inside a kernel
 * end after a second; results that such a wait left unfinished are NaN.
 *
 * A paged cache is read and written through page ids: entry i of a sequence
 * lies at page page_table[i / page_size], place i % page_size. An id or a
 * slot outside the cache is never dereferenced: what it stands for counts as
 * absent, as each call states.
 */
#ifndef SPARSE_STEP_H_
#define SPARSE_STEP_H_

#include <stdint.h>

#include "topk_indexer.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum sparse_type {
  SPARSE_BF16 = 0,
  SPARSE_FP16 = 1,
  SPARSE_FP32 = 2, /* sparse_rotary only */
  SPARSE_E4M3 = 3  /* sparse_indexer_scores only */
} sparse_type;

typedef enum sparse_rotary_layout {
  SPARSE_ROTARY_HALF = 0,       /* pair i is (x[i], x[i + rotated / 2]) */
  SPARSE_ROTARY_INTERLEAVED = 1 /* pair i is (x[2 i], x[2 i + 1]) */
} sparse_rotary_layout;

#define SPARSE_ROTARY_MAX_D 1024
#define SPARSE_ROTARY_MAX_H (1 << 30)
#define SPARSE_SCORES_MAX_D 128
#define SPARSE_SCORES_MAX_H 128
#define SPARSE_ATTENTION_MAX_D 256

/*
 * sparse_rotary - for every token t and head h, with a_i = positions[t] *
 * frequencies[i] (radians) and pairs (u, v) of x[t, h, offset .. offset +
 * rotated):
 *     u' = scale * (u cos a_i - v sin a_i),  v' = scale * (v cos a_i + u sin a_i)
 * and the rest of the head copied. `inverse` turns by -a_i, which with the
 * same scale is the gradient of the call. The angle is exact modulo whole
 * turns up to the rounding of frequencies[i] / 2 pi to 2^-63 turns, times the
 * position (2^-32 turns at the end of the 32-bit range), and 2^-32 turns of its
 * own: positions of that whole range are as accurate as small ones. Sine and
 * cosine are good to 2 ulp in SPARSE_FP32, to 2^-20 in the 16-bit types.
 *
 * out may be x itself with the same strides (in place; only the rotated part
 * is then touched); it must not overlap x in any other way. With `slots`, out
 * is a paged cache: token t goes to page slots[t] / page_size, place
 * slots[t] % page_size; a token whose slot is negative or past the cache is
 * not written. Two tokens of one call must not share a slot.
 */
typedef struct sparse_rotary_args {
  const void* x;             /* [T, H, D], unit stride in D */
  int64_t x_token_stride, x_head_stride;
  void* out;                 /* as x, or the cache when slots != NULL */
  int64_t out_page_stride;   /* used with slots */
  int64_t out_token_stride, out_head_stride;
  const void* positions;     /* [T] int32, or int64 when positions_64 */
  const double* frequencies; /* [rotated / 2], |f| < 2^40 */
  const int32_t* slots;      /* [T] or NULL */
  int64_t num_pages;         /* with slots */
  int32_t page_size;         /* with slots */
  int32_t T, H, D;
  int32_t rotated, offset;   /* rotated even, 2 <= rotated, offset + rotated <= D */
  int32_t layout, type, positions_64, inverse;
  float scale;
} sparse_rotary_args;
topk_status sparse_rotary(const sparse_rotary_args* args, topk_stream_t stream);

/*
 * sparse_indexer_scores - for every sequence b, query token t and position
 * s < n = clamp(lengths[b, t], 0, width):
 *     out[b, t, s] = key_scales[e] * sum_h weights[b, t, h] * max(0, q[b, t, h] . keys[e])
 * with e the cache entry of position s of sequence b. Positions from n on are
 * not written. Products and sums are FP32; infinities and NaN follow the
 * formula, whatever the number of heads. A position whose
 * page id lies outside the cache gets -inf, which no present key ranks below.
 */
typedef struct sparse_scores_args {
  const void* q;             /* [B, T, H, D], unit stride in D, any alignment of its elements */
  int64_t q_seq_stride, q_token_stride, q_head_stride;
  const float* weights;      /* [B, T, H] contiguous */
  const void* keys;          /* [num_pages, page_size, D]: 16-byte aligned, strides multiples of 16 bytes */
  int64_t key_page_stride, key_token_stride;
  const float* key_scales;   /* [num_pages, page_size] contiguous, or NULL for 1 */
  const int32_t* lengths;    /* [B, T] contiguous */
  const int32_t* page_table; /* [B, table_width], rows table_stride apart (0: shared by all sequences) */
  int64_t table_stride, table_width;
  float* out;                /* [B, T, width], unit stride in width */
  int64_t out_seq_stride, out_token_stride;
  int64_t num_pages;
  int64_t width;             /* <= table_width * page_size, < 2^31 */
  int32_t page_size;
  int32_t B, T, H, D;        /* H <= 128; D <= 128, whole 16-byte units */
  int32_t type;              /* of q and keys: SPARSE_BF16, SPARSE_FP16 or SPARSE_E4M3 */
} sparse_scores_args;
topk_status sparse_indexer_scores(const sparse_scores_args* args, topk_stream_t stream);

/*
 * sparse_attention - for every row (b, t) and query head h, over the
 * positions p_j = indices[b, t, j] that are seen:
 *     z_j = scale * q[b, t, h] . k[p_j, g],  g = h / (Hq / Hkv)
 *     z_j = softcap * tanh(z_j / softcap)                  (softcap > 0: any, its error is relative to z_j)
 *     z_j = z_j + slopes[h] * (p_j - query_positions[b, t]) (slopes given)
 *     lse = log sum_j exp(z_j),  out = sum_j exp(z_j - lse) * v[p_j, g]
 * Position p_j is seen when it is not negative, its page id lies in the
 * table and the cache, p_j <= query_positions[b, t] and p_j >= first[b, t]
 * (each only where given). The rest of the cache is never read, whatever it
 * holds. A row that sees nothing gets out = 0 and lse = -inf. A position that
 * is listed twice counts twice. With page_table NULL the indices are slots
 * (page * page_size + place, the output of topk_paged), which have no
 * position: query_positions, first and slopes must be NULL.
 * v may be a prefix of the entries of k (same pointer and strides): the entry
 * is then fetched once.
 * A NaN that is seen makes NaN of every result it enters, and so does a
 * logit of +infinity without a cap; with one an infinite logit is +-softcap. A
 * logit of -infinity has weight 0; a row of nothing else sees nothing. An
 * infinity of v that is seen makes its column infinite or NaN.
 * Sums, statistics and the accumulation of out are FP32; the weights
 * exp(z_j - m) are rounded to the type of v for the second product, once.
 */
typedef struct sparse_attention_args {
  const void* q;             /* [B, T, Hq, D], unit stride in D */
  int64_t q_seq_stride, q_token_stride, q_head_stride;
  const void* k;             /* [num_pages, page_size, Hkv, D]: 16-byte aligned, strides multiples of 16 bytes */
  int64_t k_page_stride, k_token_stride, k_head_stride;
  const void* v;             /* [num_pages, page_size, Hkv, Dv], as k */
  int64_t v_page_stride, v_token_stride, v_head_stride;
  const int32_t* indices;    /* [B, T, K] contiguous */
  const int32_t* page_table; /* [B, table_width] or NULL */
  int64_t table_stride, table_width;
  const int32_t* query_positions; /* [B, T] contiguous or NULL */
  const int32_t* first;      /* [B, T] contiguous or NULL */
  const float* slopes;       /* [Hq] or NULL; needs query_positions */
  void* out;                 /* [B, T, Hq, Dv] contiguous, 16-byte aligned */
  float* lse;                /* [B, T, Hq] contiguous or NULL */
  int64_t num_pages;
  int32_t page_size;
  int32_t B, T, Hq, Hkv, D, Dv, K; /* Hq a multiple of Hkv; D, Dv <= 256, multiples of 8 */
  int32_t type;              /* of q, k, v, out: SPARSE_BF16 or SPARSE_FP16 */
  float scale, softcap;      /* finite; softcap >= 0, 0 for none */
} sparse_attention_args;
topk_status sparse_attention(const sparse_attention_args* args, topk_stream_t stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* SPARSE_STEP_H_ */
