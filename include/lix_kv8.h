/*
 * lix_kv8.h - C ABI of liblix.so, attention over a paged cache held in 8 bits.
 *
 * The reader of the tokens that the indexer selects: keys and values of the
 * attended tokens lie in pages of e4m3 codes with one fp32 scale per page and
 * head.  Four steps: lix_kv8_append fills the cache, lix_kv8_attention
 * attends over it (all visible tokens, or those of the indexer's top-k),
 * lix_kv8_token_weights gives the weight that each token received, and
 * lix_kv8_evict keeps the heaviest in new pages.
 *
 * The conventions of lix.h hold: device memory of the current device owned by
 * the caller, nothing allocated or kept, work on the caller's stream,
 * synchronous validation, its status codes.  In addition:
 *
 * Cache.    k_pages, v_pages: e4m3 (OCP, 448 the largest) bytes
 *           [num_pages, Hkv, page, D]; k_scales, v_scales: fp32
 *           [num_pages, Hkv], finite and not negative.  A cached value is
 *           code * scale.  page is 16, 32, 64 or 128 tokens; D is 64, 128 or
 *           256; num_pages * Hkv * page < 2^31.
 * Tables.   block_table int32 [B, max_pages]: token s of sequence b lies in
 *           slot s % page of page block_table[b, s / page].  An entry
 *           outside [0, num_pages) is no page: its tokens are seen by no
 *           query, nothing is written to them, nothing is read out of
 *           bounds.  Sequences may share pages that are only read.
 * Lengths.  kv_lens int32 [B], tokens of each sequence, clamped to
 *           [0, max_pages * page].
 * Queries.  q [B, S, Hq, D] bf16 or fp16, strides q_sb, q_ss, q_sh in
 *           elements (multiples of 8), the last dimension contiguous.  Query
 *           head h reads key/value head h / (Hq / Hkv).
 * Visible.  q_start == NULL: query t of sequence b sees its kv_lens[b]
 *           tokens.  Otherwise it is at position q_start[b] + t and sees
 *           tokens [0, min(kv_lens[b], (q_start[b] + t + 1) / compress_ratio))
 *           (the indexer's range over compressed positions, page
 *           "...deepseek_v4.kernels.tilelang_indexer_fwd", section
 *           _make_causal_cu_seqlens; compress_ratio 1 is the causal mask).
 *           q_lens (NULL, or int32 [B]): queries t >= q_lens[b] are padding
 *           and see nothing.
 * Alignment. pages and q: 16 bytes; the others: their element.
 */
#ifndef LIX_KV8_H
#define LIX_KV8_H

#include "lix.h"
#include "lix_rotary.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * lix_kv8_append - quantises new tokens behind those of each sequence.
 *
 * Token i < new_lens[b] of k[b], v[b] becomes token kv_lens[b] + i of
 * sequence b (new_lens NULL: S of each; values are clamped to [0, S]; kv_lens
 * is not changed).  For each page that receives a token, per head and for
 * keys and values apart:
 *     need  = the smallest power of two >= max |x| / 448 over its finite new
 *             values, at least 2^-60
 *     scale = need                     where its first slot is new
 *             max(need, its scale)     otherwise
 *     code  = e4m3(x / scale), rounded to nearest even, saturating at 448
 *             (infinities too); NaN stays NaN
 * Where the scale of a page with older tokens grows, those are written again
 * as e4m3(code * old / new), exact for powers of two down to e4m3's smallest
 * value.  Slots behind the last new token keep their bytes.  Tokens that fall
 * on no page or behind max_pages are dropped.  Two sequences must not append
 * to the same page in one call.
 *
 *   k, v      dtype (LIX_BF16 or LIX_FP16) [B, S, Hkv, D], strides in
 *             elements (multiples of 8), 16-byte aligned
 *   new_lens  int32 [B] or NULL
 */
int lix_kv8_append(const void* k, long long k_sb, long long k_ss, long long k_sh,
                   const void* v, long long v_sb, long long v_ss, long long v_sh, int dtype,
                   int B, int S, int Hkv, int D,
                   void* k_pages, void* v_pages, float* k_scales, float* v_scales, int num_pages, int page,
                   const int32_t* block_table, int max_pages, const int32_t* kv_lens, const int32_t* new_lens,
                   hipStream_t stream);

/*
 * lix_kv8_attention - softmax attention over the cached tokens.
 *
 * With x[s] = scale * (q . k[s]) over the tokens that query (b, t) sees:
 *     lse = log(sum_s exp(x[s]))
 *     out = sum_s exp(x[s] - lse) v[s]
 * indices == NULL: over all visible tokens.  indices int32 [B, S, topk] (as
 * lix_topk gives them, shared by the heads): over the listed ones that are
 * visible; other entries (-1 among them) count nothing, a token listed twice
 * counts twice.  A query that sees nothing: out = 0, lse = -inf.  Products
 * accumulate in fp32; the weights exp(x - running maximum) are rounded once
 * to fp16 (11 bits) to multiply the values, not in their sum.  Hidden tokens
 * contribute nothing whatever their bytes are.  Results are the same bits on
 * every call.
 *
 *   scale      finite, >= 0
 *   out        dtype of q [B, S, Hq, D], contiguous, 16-byte aligned
 *   lse        fp32 [B, S, Hq]
 *   workspace  lix_kv8_attention_workspace_bytes bytes, 256-byte aligned
 *              (NULL where that is 0); contents unspecified before and after
 * LIX_ERR_SHAPE: a size < 1, Hq not a multiple of Hkv, topk < 1 with indices,
 * compress_ratio < 1, a negative or not finite scale, or a smaller workspace.
 */
int lix_kv8_attention(const void* q, long long q_sb, long long q_ss, long long q_sh, int dtype,
                      int B, int S, int Hq, int Hkv, int D,
                      const void* k_pages, const void* v_pages, const float* k_scales, const float* v_scales,
                      int num_pages, int page, const int32_t* block_table, int max_pages, const int32_t* kv_lens,
                      const int32_t* q_start, const int32_t* q_lens, int compress_ratio, float scale,
                      const int32_t* indices, int topk, void* out, float* lse,
                      void* workspace, long long workspace_bytes, hipStream_t stream);

/*
 * lix_kv8_attention_workspace_bytes - workspace of lix_kv8_attention for
 * these sizes (topk 0: no indices): the partial results of the parts that a
 * long sequence is split into where there are few queries, 0 where it is not
 * split; -1 for sizes that the call does not take.  Pure host function.
 */
long long lix_kv8_attention_workspace_bytes(int B, int S, int Hq, int Hkv, int D, int page, int max_pages, int topk);

/*
 * lix_kv8_token_weights - the attention weight that each cached token got.
 *
 *     w[b, n, s] = sum over queries t and the heads h of key head n of
 *                  exp(scale * (q[b,t,h] . k[s]) - lse[b,t,h])
 * over the queries that see token s; a query with lse = -inf gives nothing.
 * Written to (accumulate == 0) or added to weights[b, n, s] for
 * s < kv_lens[b]; entries behind stay as they were.  Sums are in fp32 in a
 * fixed order: the same bits on every call.
 *
 *   lse      fp32 [B, S, Hq], as lix_kv8_attention gave it for these queries
 *   weights  fp32 [B, Hkv, width], width >= max_pages * page
 *   workspace  lix_kv8_token_weights_workspace_bytes bytes, 256-byte aligned
 *            (NULL where that is 0); contents unspecified before and after
 */
int lix_kv8_token_weights(const void* q, long long q_sb, long long q_ss, long long q_sh, int dtype,
                          int B, int S, int Hq, int Hkv, int D,
                          const void* k_pages, const float* k_scales, int num_pages, int page,
                          const int32_t* block_table, int max_pages, const int32_t* kv_lens,
                          const int32_t* q_start, const int32_t* q_lens, int compress_ratio, float scale,
                          const float* lse, float* weights, int width, int accumulate,
                          void* workspace, long long workspace_bytes, hipStream_t stream);

/* Workspace of lix_kv8_token_weights for these sizes: the sums of the parts that many queries are split into where
 * there are few keys, 0 where they are not; -1 for sizes that the call does not take.  Pure host function. */
long long lix_kv8_token_weights_workspace_bytes(int B, int S, int Hq, int Hkv, int D, int page, int max_pages);

/*
 * lix_kv8_evict - keeps the tokens with the largest weights, in new pages.
 *
 * Of a sequence of n > keep tokens, for each key head: its first `sinks`, its
 * last `recent`, and of the others those with the largest weights, equal
 * weights by token, the lower first, `keep` in all; of a shorter sequence,
 * all.  They go in ascending order to the slots of the pages of
 * new_table[b], which no sequence may be using: the old pages are only read.
 * Each new page gets, per head, the scale that lix_kv8_append would give its
 * values.  Weights must not be NaN (which tokens are kept is then
 * unspecified).
 *
 *   weights      fp32 [B, Hkv, width], width >= max_pages * page
 *   new_table    int32 [B, new_max_pages], new_max_pages * page >= keep
 *   new_lens     int32 [B]             out: min(n, keep)
 *   kept         int32 [B, Hkv, keep]  out: the kept tokens, -1 behind them
 *   new_weights  fp32  [B, Hkv, keep]  out: their weights, 0 behind them
 *   workspace    lix_kv8_evict_workspace_bytes bytes, 256-byte aligned (NULL
 *                where that is 0)
 * LIX_ERR_SHAPE: a size < 1, sinks or recent < 0, sinks + recent > keep, a
 * width or new_max_pages that is too small, or a smaller workspace.
 */
int lix_kv8_evict(void* k_pages, void* v_pages, float* k_scales, float* v_scales,
                  int num_pages, int page, int B, int Hkv, int D,
                  const int32_t* block_table, int max_pages, const int32_t* kv_lens,
                  const float* weights, int width, const int32_t* new_table, int new_max_pages,
                  int keep, int recent, int sinks, int32_t* new_lens, int32_t* kept, float* new_weights,
                  void* workspace, long long workspace_bytes, hipStream_t stream);

/* Workspace of lix_kv8_evict: the selected tokens and ranges of rows beyond 32768 tokens, 0 for tables that hold no
 * more; -1 for sizes it does not take.  Pure host function. */
long long lix_kv8_evict_workspace_bytes(int B, int Hkv, int page, int max_pages, int width, int keep, int recent,
                                        int sinks);

#ifdef __cplusplus
}
#endif

#endif /* LIX_KV8_H */
