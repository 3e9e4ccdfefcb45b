/*
 * dq4_attn — the attention around the 4-bit projections of dq4.h, for NVIDIA GB300
 * (compute capability 10.3): the norm of queries and keys with the position rotation
 * (forward and backward), the append to a paged key/value cache held in 8 bits, and the
 * attention that reads it.
 *
 * Conventions are those of dq4.h: DEVICE pointers owned by the caller, no allocation and
 * no synchronization inside, work enqueued on `stream`, a status code returned (nothing is
 * enqueued on an error other than DQ4_ERR_LAUNCH), host threads may call concurrently, but
 * calls that share a workspace one at a time: dq4_kv8_attention may take two launches, which
 * have to follow each other in the stream.
 * Element types are DQ4_OUT_F16 / DQ4_OUT_BF16 / DQ4_OUT_F32 (`dtype`).  Strides count
 * elements.  Sums, softmax statistics and norms are FP32.
 *
 * The rotation R(pos) turns the first `rotary` values of a head (rotary even, <= head_dim)
 * by the angles whose cosines and sines stand in row pos of the FP32 tables cos and sin
 * (table_rows x rotary / 2, row-major):
 *   interleaved == 0: values i and i + rotary / 2 are a pair;
 *   interleaved != 0: values 2 i and 2 i + 1 are a pair;
 *   (a, b) -> (a c - b s, b c + a s) in FP32, every product and sum rounded on its own, but
 *   for dq4_qk_norm_rope with weights, which may multiply a value's factors in another order.
 * The other values pass.  cos == sin == NULL: no rotation (tables of no rows are tables).
 *
 * `bad` is an optional device int (NULL to skip) that counts what a call could not do,
 * as each entry point says; it stays 0 for valid inputs.
 */
#ifndef DQ4_ATTN_H
#define DQ4_ATTN_H

#include <stdint.h>

#include "dq4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Norm and rotation of every head of q and of k in one launch:
 *   y = R(positions[t]) (w * x * rstd),  rstd = 1 / sqrt(mean(x^2) + eps)
 *   q, k            tokens x q_heads x head_dim and tokens x k_heads x head_dim of `dtype`,
 *                   values of a head contiguous, tokens and heads at the given strides
 *                   (views of a fused projection's rows); k_heads may be 0 (k NULL)
 *   q_weight, k_weight  `dtype`[head_dim]; both NULL: no norm, the rotation alone
 *   positions       int64[tokens], rows of cos and sin (NULL without them).  A position
 *                   outside [0, table_rows) yields zeros for the token's heads, each
 *                   counted into bad.
 *   q_out, k_out    contiguous tokens x heads x head_dim of `dtype`, not overlapping x
 * head_dim: even, 2 .. 1024.  Fastest for head_dim 64, 128 or 256 with rotary % 8 == 0,
 * 4-value groups aligned to their size (strides % 4 == 0), which one pass of registers
 * covers; other shapes take a second kernel with the same results up to FP32 rounding.
 */
int dq4_qk_norm_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                     int64_t k_token_stride, int64_t k_head_stride, int32_t dtype,
                     int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                     const void* q_weight, const void* k_weight, float eps, const float* cos,
                     const float* sin, int64_t table_rows, int32_t rotary, int32_t interleaved,
                     const int64_t* positions, void* q_out, void* k_out, int* bad,
                     void* stream);

/*
 * The gradients of dq4_qk_norm_rope: from dq_out, dk_out (contiguous, `dtype`) and its
 * inputs, with g = R(-pos) dy and xh = x * rstd,
 *   dx = rstd * (g w - xh * mean(g w xh)),    dw = sum over tokens and heads of g xh
 *   dq, dk          contiguous, `dtype`, as q_out and k_out
 *   dq_weight, dk_weight  FP32[head_dim] (both NULL without weights, when dx = g)
 *   workspace       dq4_qk_norm_rope_backward_workspace_bytes(head_dim) bytes, 256-byte
 *                   aligned, the first 256 zero before its first use; a completed call leaves
 *                   it ready for the next in the same stream (not for concurrent calls or
 *                   replays of captured ones).
 *                   Not used without weights.
 * The sums over tokens are taken in a fixed order: the same call gives the same bits.
 */
int dq4_qk_norm_rope_backward(const void* dq_out, const void* dk_out, const void* q,
                              int64_t q_token_stride, int64_t q_head_stride, const void* k,
                              int64_t k_token_stride, int64_t k_head_stride, int32_t dtype,
                              int64_t tokens, int32_t q_heads, int32_t k_heads,
                              int32_t head_dim, const void* q_weight, const void* k_weight,
                              float eps, const float* cos, const float* sin,
                              int64_t table_rows, int32_t rotary, int32_t interleaved,
                              const int64_t* positions, void* dq, void* dk, float* dq_weight,
                              float* dk_weight, void* workspace, int64_t workspace_bytes,
                              int* bad, void* stream);
int64_t dq4_qk_norm_rope_backward_workspace_bytes(int32_t head_dim);

/*
 * A paged key/value cache in 8 bits.  A value is e4m3(code) * scale, with one FP32 scale
 * for each page and head:
 *   k, v            e4m3 bytes [pages][kv_heads][page][head_dim], 16-byte aligned
 *   k_scale, v_scale  FP32 [pages][kv_heads]
 * page (tokens): 16, 32, 64, 128 or 256.  head_dim: 64 or 128.  Nothing has to be
 * initialized: slots and scales are read only where tokens were appended.
 */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t pages;
  int32_t kv_heads;
  int32_t page;
  int32_t head_dim;
} dq4_kv8_cache;

/*
 * Append tokens to the cache, one launch.  Sequence b's new tokens are rows
 * cu[b] .. cu[b + 1] - 1 of k and v (cu: int32[seqs + 1], cu[0] = 0, cu[seqs] = tokens; NULL:
 * one token each) and its length with them is seq_lens[b] (int32), so that they take
 * positions seq_lens[b] - n_b .. seq_lens[b] - 1.  Token pos of sequence b lives in slot
 * pos % page of page block_table[b * table_stride + pos / page] (int32).
 *   k, v            tokens x kv_heads x head_dim of `dtype` (FP16 or BF16), a head's values
 *                   contiguous and aligned to 8 bytes (strides % 4 == 0)
 *   cos, sin        tables of the rotation of k (k is rotated by its position in FP32, then
 *                   quantized); NULL: k is stored as it is.  rotary % 8 == 0.
 * For each page and head that gets tokens, and for K and V each:
 *   fit   = the least power of two with max|x| <= 448 fit over the page's new tokens, at
 *           least 2^-100; NaN if one of them is not finite
 *   scale = max(the page's scale if it holds earlier tokens of the sequence, fit), NaN if
 *           either is
 *   code  = e4m3(x / scale), round to nearest even; the page's earlier codes become
 *           e4m3(code * (old scale / scale)), exact but for codes that get subnormal,
 *           as both scales are powers of two.
 * A page with a NaN scale holds no usable values until its first slot is written again.
 * No two sequences of one call may append to the same page.
 * bad counts tokens that were not stored (position negative or past the table's
 * table_width pages, or a page id outside [0, pages)) and keys past the rotation's
 * tables (stored as zeros), each once.
 */
int dq4_kv8_append(const dq4_kv8_cache* cache, const void* k, int64_t k_token_stride,
                   int64_t k_head_stride, const void* v, int64_t v_token_stride,
                   int64_t v_head_stride, int32_t dtype, int64_t tokens,
                   const int32_t* block_table, int64_t table_stride, int32_t table_width,
                   const int32_t* seq_lens, const int32_t* cu, int64_t seqs, const float* cos,
                   const float* sin, int64_t table_rows, int32_t rotary, int32_t interleaved,
                   int* bad, void* stream);

/*
 * Attention of new tokens over the cache.  Row i of sequence b (its tokens, cu, seq_lens
 * and block_table as for dq4_kv8_append) has position p = seq_lens[b] - n_b + i and sees the
 * keys j with 0 <= j < seq_lens[b], j <= p if causal, and j > p - window if window > 0:
 *   out = sum_j e_j v_j / sum_j e_j,  e_j = exp(scale * q . k_j),  lse = log sum_j e_j
 * A row that sees no key gets zeros and lse = -infinity.  Query head h reads kv head
 * h / (heads / kv_heads).
 *   q               tokens x heads x head_dim, FP16 or BF16, a head's values contiguous and
 *                   16-byte aligned (strides % 8 == 0)
 *   out             contiguous tokens x heads x head_dim of `dtype`, 16-byte aligned
 *   lse             optional FP32 tokens x heads (NULL to skip)
 *   max_new         the most new tokens of any sequence, or an estimate: it chooses the
 *                   kernel, and what the result means does not depend on it (its rounding
 *                   does)
 *   workspace       device memory, 256-byte aligned, of at least
 *                   dq4_kv8_attention_workspace_bytes bytes, the first 2048 zero before
 *                   its first use; a completed call leaves it ready for later calls of any
 *                   shape that it is large enough for, in the same stream (not for concurrent
 *                   calls or replays of captured ones).
 * The result does not depend on the order in which the SMs work.  Weights e_j times their pages'
 * V scales are FP16 in the product with V: relative to the row's largest, one has all its 11
 * bits down to 2^-27, a fixed step of 2^-37 below, and is nothing below 2^-38.  lse and the
 * sum in out's denominator take them in FP32, down to 2^-138 of the largest (what is less would
 * matter only with V scales of one sequence 2^100 apart).
 * pages * kv_heads and tokens * heads / kv_heads: at most 2^31 - 1.  Keys past the table's
 * table_width pages, and pages with an id outside [0, pages), are not seen; bad is
 * incremented for each part of the work that met one, and for a wait that ran out (never
 * expected; the workspace must then be cleared again).  Pages that lie wholly before
 * the windows of all of the sequence's rows are not looked at: they may have been given
 * back, their ids and what they hold may be anything.
 * A NaN code or scale of K or V reaches the rows that see its key, and no others.  Of V, a
 * scale that is NaN (append's mark of a page with a value that is not finite) makes out and
 * lse of such a row NaN; a NaN code beside a number (append writes none) makes the row's
 * value of that column NaN, or the whole row and its lse.
 */
int dq4_kv8_attention(const dq4_kv8_cache* cache, const void* q, int64_t q_token_stride,
                      int64_t q_head_stride, int32_t dtype, int64_t tokens, int32_t heads,
                      const int32_t* block_table, int64_t table_stride, int32_t table_width,
                      const int32_t* seq_lens, const int32_t* cu, int64_t seqs,
                      int32_t max_new, float scale, int32_t causal, int32_t window, void* out,
                      float* lse, void* workspace, int64_t workspace_bytes, int* bad,
                      void* stream);
int64_t dq4_kv8_attention_workspace_bytes(int64_t tokens, int64_t seqs, int32_t heads,
                                          int32_t kv_heads, int32_t head_dim);

#ifdef __cplusplus
}
#endif

#endif /* DQ4_ATTN_H */
