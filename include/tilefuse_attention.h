/*
 * tilefuse_attention.h -- C ABI of the attention that stands between a decoder
 * layer's quantized linears (tilefuse.h), and of the paged key-value cache
 * that it reads, for AMD MI355X (gfx950).
 *
 * A layer's step: the QKV linear -> tf_kv_append (rotate queries and keys,
 * write keys and values into the cache) -> tf_attn_decode (one new token per
 * sequence) or tf_attn_prefill_paged (many) -> the output linear.  The rotated
 * keys are in the pages alone: tf_kv_append leaves the QKV output as it was.
 * tf_attn_prefill is for keys that stand packed: whose positions are encoded in
 * another way, or that the caller has rotated.
 * tf_kv_fork and tf_kv_compact keep the pool of pages.
 *
 * Notation: T tokens, Hq query heads, Hkv key-value heads (Hq a multiple:
 * query head j reads key-value head j / (Hq / Hkv)), D channels of a head.
 *
 * The cache.  A plane is [pages][Hkv][page][D] 16-bit values: the keys, or the
 * values, of one layer.  `tables` is int32 [seqs][width]: entry (s, c) names
 * the page that holds tokens c * page .. of sequence s; entries past a
 * sequence's length may hold anything.  A page id outside [0, pages) inside a
 * sequence's length reads as zeros and is never written.
 *
 * Conventions shared with tilefuse.h: device pointers owned by the caller, the
 * library allocates nothing and keeps no pointer; calls are asynchronous on
 * `stream`; every argument the host can see is checked before any HIP work
 * and a call that returns anything but TF_OK has launched nothing.  Index
 * tensors (tables, lengths, positions) live on the device: the kernels clamp
 * or skip what lies outside the buffers, as each call says, and never read
 * or write out of them.  Outputs must not alias inputs unless a call allows
 * it.  `type` is TF_TYPE_BF16 or TF_TYPE_F16, of every 16-bit tensor of a call
 * (others: TF_ERR_UNSUPPORTED).  Tensors described with strides take them in
 * elements: multiples of 8, base 16-byte aligned (else TF_ERR_ALIGN), token
 * stride and (of several heads) head stride at least D and below 2^26 (else
 * TF_ERR_SHAPE); channels are contiguous.  All other tensors are contiguous;
 * 16-bit ones and rope 16-byte, int32 ones 4-byte, workspaces 256-byte
 * aligned.
 */
#ifndef TILEFUSE_ATTENTION_H
#define TILEFUSE_ATTENTION_H

#include "tilefuse.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { TF_TYPE_BF16 = 0, TF_TYPE_F16 = 1 };

/* ------------------------------------------------------------------------ */
/* Append: rotate and store new tokens.                                      */
/*                                                                           */
/*   qkv    [T][(Hq + 2 Hkv) D] of token stride qkv_token: the fused QKV      */
/*          output, query heads, then key heads, then value heads            */
/*   rope   fp32 [rope_rows][D]: for each position D/2 cosines, then D/2     */
/*          sines.  Channels i and i + D/2 are a pair:                       */
/*          (a, b) -> (a cos - b sin, b cos + a sin), fp32, rounded once      */
/*   seq, pos  int32 [T]: the sequence of a token and its position in it     */
/*   q      out [T][Hq][D]: the rotated query heads                          */
/*   k_pages, v_pages  out: rotated keys and copied values, at the page that */
/*          tables names for the position                                    */
/*                                                                           */
/* D is a multiple of 16, at most 1024; page a power of two, 16 .. 1024.  A   */
/* token whose sequence, position or page does not exist is not stored; a    */
/* position outside the rope rows has its heads turned to zeros.  Two tokens */
/* of one call at the same place: either's row may stay.  T is at most        */
/* 2^26 - 4 (else TF_ERR_SHAPE); T == 0: TF_OK.                              */
/* ------------------------------------------------------------------------ */
int tf_kv_append(int type, const uint16_t *qkv, int64_t qkv_token, const float *rope, int64_t rope_rows,
                 const int32_t *seq, const int32_t *pos, int64_t T, const int32_t *tables, int64_t seqs, int64_t width,
                 uint16_t *q, uint16_t *k_pages, uint16_t *v_pages, int64_t pages, int64_t page, int64_t Hq,
                 int64_t Hkv, int64_t D, void *stream);

/* ------------------------------------------------------------------------ */
/* Attention.  Scores are scale q . k with fp32 sums, the softmax statistics */
/* and the outputs' sums are fp32, probabilities are rounded to the tensors' */
/* type (nearest even) before they meet V, outputs are rounded once.  scale  */
/* is positive and scale * log2(e) finite, D is 64 or 128, Hq / Hkv at most  */
/* 1024 (else TF_ERR_UNSUPPORTED).  A row that sees no key is zero.  Keys    */
/* and values that a row does not see do not reach it, whatever they hold,   */
/* infinities and NaN included.                                              */
/* ------------------------------------------------------------------------ */

/* One new token per sequence over its pages.
 *   q      [seqs][Hq][D], strides q_token, q_head
 *   lens   int32 [seqs]: tokens in the cache, the new one included; read as
 *          clamped to [0, min(longest, width * page)].  0: the row is zero.
 *   longest  an upper bound of lens: it sets how the cache's length is split
 *          over workgroups
 *   out    [seqs][Hq][D]
 * page is a power of two, 16 .. 1024; seqs <= 65535 (0: TF_OK); longest and
 * width * page at most 2^30.  The workspace
 * holds the split's partial results; the size depends on the device's compute
 * units.  Results do not depend on what it held. */
size_t tf_attn_decode_workspace_bytes(int64_t seqs, int64_t Hq, int64_t Hkv, int64_t D, int64_t longest);
int tf_attn_decode(int type, const uint16_t *q, int64_t q_token, int64_t q_head, const uint16_t *k_pages,
                   const uint16_t *v_pages, int64_t pages, int64_t page, const int32_t *tables, int64_t width,
                   const int32_t *lens, uint16_t *out, int64_t seqs, int64_t Hq, int64_t Hkv, int64_t D,
                   int64_t longest, float scale, void *workspace, size_t ws_bytes, void *stream);

/* Causal attention of packed prompts.  Sequence s has tokens cu_q[s] ..
 * cu_q[s + 1] - 1 of q and keys cu_k[s] .. cu_k[s + 1] - 1 of k and v; its last
 * token sees every key, the one before it one fewer, and so on.
 *   q      [T][Hq][D], strides q_token, q_head
 *   k, v   [keys][Hkv][D] with strides of their own: all three may be parts of
 *          one fused QKV output.  They are taken as they are: beside queries
 *          that tf_kv_append has rotated, the QKV output's keys, which it has
 *          not, are the wrong ones
 *   cu_q, cu_k  int32 [seqs + 1], ascending; clamped to the tensors
 *   longest  an upper bound of the new tokens of a sequence (tokens past it
 *          are not computed), at most T
 *   out    [T][Hq][D]; rows of no sequence are not written
 * T and keys are at most 2^30, and seqs * Hkv * ceil(longest * (Hq / Hkv) / 128)
 * is below 2^24 (else TF_ERR_SHAPE).  The workspace holds partial results where few
 * rows meet many keys and the keys are cut into ranges; the size depends on
 * the device's compute units, results do not depend on what it held. */
size_t tf_attn_prefill_workspace_bytes(int64_t seqs, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t longest,
                                       int64_t keys);
int tf_attn_prefill(int type, const uint16_t *q, int64_t q_token, int64_t q_head, const uint16_t *k, int64_t k_token,
                    int64_t k_head, const uint16_t *v, int64_t v_token, int64_t v_head, const int32_t *cu_q,
                    const int32_t *cu_k, uint16_t *out, int64_t seqs, int64_t T, int64_t keys, int64_t Hq, int64_t Hkv,
                    int64_t D, int64_t longest, float scale, void *workspace, size_t ws_bytes, void *stream);

/* The same over the pages of a cache that already holds the sequences' lens[s]
 * tokens, the new ones included (prompts in chunks, shared prefixes).  `keys`
 * of the workspace's size is width * page, and the work is ordered and split for
 * that many: a single short prompt over a table for 131072 tokens takes 2 to 4 us
 * longer than over one cut to its length. */
int tf_attn_prefill_paged(int type, const uint16_t *q, int64_t q_token, int64_t q_head, const uint16_t *k_pages,
                          const uint16_t *v_pages, int64_t pages, int64_t page, const int32_t *tables, int64_t width,
                          const int32_t *cu_q, const int32_t *lens, uint16_t *out, int64_t seqs, int64_t T, int64_t Hq,
                          int64_t Hkv, int64_t D, int64_t longest, float scale, void *workspace, size_t ws_bytes,
                          void *stream);

/* ------------------------------------------------------------------------ */
/* The pool.  refs int32 [pages] counts the table entries that name a page;  */
/* a page of 0 or less is free.  cache is [planes][pages][Hkv][page][D], any  */
/* 16-bit type, D a multiple of 8; page is 1 .. 1024.                        */
/* ------------------------------------------------------------------------ */

/* Each children[i] becomes a copy of parents[i]: it shares the parent's full
 * pages (refs_out + 1) and gets a copy of the partial page, if there is one, in
 * the lowest free pages in the order of i (zeros, where the entry of the partial
 * page names none, as the parent reads it).  Its table row is replaced (pages
 * it held are not released; unused entries become -1).
 *   refs_out, tables_out, lens_out  the whole new state; may be the inputs
 *   status  int32 [1]: 0, or how many free pages were missing; then nothing is
 *           forked and the outputs equal the inputs
 * A pair with an index outside [0, seqs) is skipped.  A child is named once
 * and is no parent of the same call.  (planes + 1) * forks + seqs is below
 * 2^24 (else TF_ERR_SHAPE). */
size_t tf_kv_fork_workspace_bytes(int64_t forks);
int tf_kv_fork(uint16_t *cache, int64_t planes, int64_t pages, int64_t Hkv, int64_t page, int64_t D,
               const int32_t *refs, const int32_t *tables, const int32_t *lens, int64_t seqs, int64_t width,
               const int32_t *parents, const int32_t *children, int64_t forks, int32_t *refs_out, int32_t *tables_out,
               int32_t *lens_out, int32_t *status, void *workspace, size_t ws_bytes, void *stream);

/* With L pages in use (refs > 0), the pages in use at or past L move to the free
 * ones before L, both in ascending order, in every plane.
 *   refs_out, tables_out  the new state; may be the inputs
 *   moved   int32 [pages]: where each page is now; -1 for a free page
 * A table entry outside [0, pages) or naming a free page becomes -1. */
size_t tf_kv_compact_workspace_bytes(int64_t pages);
int tf_kv_compact(uint16_t *cache, int64_t planes, int64_t pages, int64_t Hkv, int64_t page, int64_t D,
                  const int32_t *refs, const int32_t *tables, int64_t seqs, int64_t width, int32_t *refs_out,
                  int32_t *tables_out, int32_t *moved, void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TILEFUSE_ATTENTION_H */
