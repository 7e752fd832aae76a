/*
 * sparse_cache.h - C ABI of the operators of a paged cache held in 8 bits
 * (GB300, sm_103a), in the same library as topk_indexer.h and sparse_step.h,
 * with their status codes, stream type and conventions:
 *
 *   sparse_append          keys and values appended to a paged cache of their
 *                          own type or in 8 bits, the keys rotated on the way
 *   sparse_attention_e4m3  sparse_attention over a cache in 8 bits
 *
 * A cache in 8 bits holds its entries as E4M3 numbers in units of a scale that
 * the entries of a block share, one for each head: with `blocks` blocks a page,
 * entry `place` of a page belongs to block place / (page_size / blocks), and
 * scales are FP32 [num_pages, blocks, H], contiguous. One block a page shares a
 * scale over the page, page_size blocks give each entry its own (and with one
 * head the key_scales that sparse_indexer_scores reads).
 */
#ifndef SPARSE_CACHE_H_
#define SPARSE_CACHE_H_

#include <stdint.h>

#include "sparse_step.h"
#include "topk_indexer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPARSE_APPEND_MAX_D 1024
#define SPARSE_APPEND_MAX_H 65535

/*
 * sparse_append - token t's keys, rotated as by sparse_rotary, and its values
 * as they are, for every head, go to page slots[t] / page_size, place slots[t] %
 * page_size of their caches; a token whose slot is negative or past the cache is
 * not written, and neither is anything else of the caches. Two tokens of one
 * call must not share a slot.
 *
 * A cache of the inputs' type takes the results rounded to it. A cache in
 * SPARSE_E4M3 takes them in units of their block's scale s:
 *   - `first` is the least place in a block of the call's tokens, which may come in
 *     any order (fastest with those of a block one behind the other).
 *   - size = scale (|u| + |v|) for the pairs (u, v) that turn, |x| for the rest and
 *     for values, bounds the stored numbers at any position. need = the smallest
 *     power of two, 2^-126 at least, with size <= 448 need for all of the block's
 *     tokens in this call, numbers that are not finite aside.
 *   - With first = 0 the block begins: s = need. Otherwise the places before
 *     `first` hold entries: s = max(s, need), and where that is more than
 *     before they are rounded again in the new unit (between powers of two only
 *     numbers below 2^-6 of the new unit lose digits). A scale of 0 marks a block
 *     that holds nothing yet; any other is positive and normal. What lies behind
 *     `first` counts as nothing.
 *   - Numbers are rounded to nearest, once; results that are not finite become NaN.
 * The angle is as exact as sparse_rotary's, sine and cosine good to 2^-20 where
 * the cache has less than 32 bits, to 2 ulp in SPARSE_FP32.
 */
typedef struct sparse_append_args {
  const void* k;             /* [T, H, D], unit stride in D */
  int64_t k_token_stride, k_head_stride;
  const void* v;             /* [T, H, Dv], unit stride in Dv, or NULL: keys only */
  int64_t v_token_stride, v_head_stride;
  void* k_cache;             /* [num_pages, page_size, H, D], unit stride in D */
  int64_t k_cache_page_stride, k_cache_token_stride, k_cache_head_stride;
  void* v_cache;             /* [num_pages, page_size, H, Dv]; used with v */
  int64_t v_cache_page_stride, v_cache_token_stride, v_cache_head_stride;
  float* k_scales;           /* [num_pages, blocks, H] contiguous; caches in SPARSE_E4M3 only */
  float* v_scales;           /* the same */
  const void* positions;     /* [T] int32, or int64 when positions_64; used with frequencies */
  const double* frequencies; /* [rotated / 2], |f| < 2^40 */
  const int32_t* slots;      /* [T] */
  int64_t num_pages;
  int32_t page_size, blocks; /* blocks divides page_size; 0 with a cache of the inputs' type */
  int32_t T, H, D, Dv;       /* H <= 65535; D, Dv <= 1024 */
  int32_t rotated, offset;   /* of the keys; rotated even, 0 for none, offset + rotated <= D */
  int32_t layout, type;      /* of k and v: SPARSE_BF16, SPARSE_FP16 or SPARSE_FP32 */
  int32_t cache_type;        /* `type`, or SPARSE_E4M3 */
  int32_t positions_64;
  float scale;
} sparse_append_args;
topk_status sparse_append(const sparse_append_args* args, topk_stream_t stream);

/*
 * sparse_attention_e4m3 - sparse_attention (its masks, cap, biases, empty rows
 * and slots, word for word) over a cache whose entries stand for k = k_scales[b,
 * g] * the numbers of attention.k, v = v_scales[b, g] * those of attention.v, with b
 * the entry's block and g the key head. attention.type is the type of q and out.
 * Scales are finite, and so is a key's scale times attention.scale times a 2^7th part of a query
 * head's largest element, in FP32; values' scales of 2^-60 to 2^60 lose nothing, below that the
 * values fade out. A NaN in an entry that is seen makes NaN of every result it
 * enters, and so does a query that is not finite.
 * Products are exact: a bf16 or fp16 query is split into two or three E4M3 terms
 * (elements below 2^-13 of their head's largest one keep steps of 2^-20, or 2^-24, of
 * that); sums and statistics are FP32. A weight, times its value's scale, is rounded to
 * 9 bits (SPARSE_BF16) or to fp16's 11 (SPARSE_FP16) for the second product, once;
 * weights below 2^-10 of a head's largest keep steps of 2^-19, or 2^-23, of it, where a
 * list has more than 2048 entries those of each of up to eight parts of it by themselves.
 */
typedef struct sparse_attention_e4m3_args {
  sparse_attention_args attention; /* k, v: SPARSE_E4M3, 16-byte aligned, strides multiples of 16; D, Dv <= 256, multiples of 16 */
  const float* k_scales;           /* [num_pages, blocks, Hkv] contiguous */
  const float* v_scales;           /* the same, or the same ones */
  int32_t blocks;                  /* divides page_size */
} sparse_attention_e4m3_args;
topk_status sparse_attention_e4m3(const sparse_attention_e4m3_args* args, topk_stream_t stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* SPARSE_CACHE_H_ */
