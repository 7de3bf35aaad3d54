/*
 * splitzip_kv4.h -- a paged KV cache held in 4 bits and the operators on it, for AMD MI355X
 * (gfx950): append, read, attend, weigh, evict.  Part of libsplitzip.so; status codes and
 * splitzip_last_error() as in splitzip.h.
 *
 * Format.  32 channels of one token and head form a block: one scale byte b and 32 codes.
 * A code is a sign bit over one of the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 (E2M1) and stands
 * for itself times 2^(b - 127).  A block whose largest value is m 2^E (1 <= m < 2) takes the
 * scale 2^(E - 2), or 2^(E - 1) for m >= 1.75: the smallest power of two under which that value
 * rounds to at most 6.  Codes are rounded to nearest, ties to the even code.  b stays within
 * [2, 252], so every value is a finite and normal BF16 number or zero (values past
 * 6 * 2^125 become that).  A block that holds an infinity or a NaN has b = 255 and reads as NaN.
 *
 * Buffers.  P pages of page_size tokens (a power of two, 16 .. 1024), H KV heads, D channels a
 * head (64, 128 or 256):
 *
 *   k_codes  u8 [P][H][page_size][D / 2]            even channel in the low nibble
 *   k_scales u8 [P][H][page_size][D / 32]
 *   v_codes  u8 [P][H][page_size / 4][16][4][D / 32] tokens interleaved in fours: 16 runs of
 *                                                   D / 16 channels, of each run four tokens
 *   v_scales u8 [P][H][D / 32][page_size]
 *   weights  f32 [P][H][page_size]                  accumulated attention weights
 *   status   u32 [1]                                SPLITZIP_KV4_BAD_* bits, set by kernels
 *
 * all contiguous and 16-byte aligned.  Token j of sequence s lies in page
 * table[s * table_stride + j / page_size] at j % page_size.
 *
 * Conventions
 *   - Pointers are DEVICE pointers on cache->device, structs are host memory read before the
 *     call returns.  Work is enqueued on `stream`; no call waits, allocates or copies to the
 *     host, so each may be captured into a graph.
 *   - What only the GPU sees (table, lens, cu_seqlens) is checked there: a page number outside
 *     [0, num_pages), a length outside the table and offsets that decrease or leave [0, total]
 *     set a bit of *status.  Such a page is never read or written: its tokens are left out of
 *     append and of attention, read as NaN and evicted as zeros; a length is cut to the table's.
 *   - Sequences may share pages in attend, read and weigh; append and evict write to pages that no
 *     other sequence of the call has.
 */
#ifndef SPLITZIP_KV4_H
#define SPLITZIP_KV4_H

#include "splitzip.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPLITZIP_KV4_BF16 0
#define SPLITZIP_KV4_FP16 1
#define SPLITZIP_KV4_FP32 2   /* append and read only */

#define SPLITZIP_KV4_BAD_PAGE 1u     /* bits of *status */
#define SPLITZIP_KV4_BAD_LENGTH 2u
#define SPLITZIP_KV4_BAD_OFFSETS 4u

typedef struct splitzip_kv4_cache {
    uint8_t *k_codes;
    uint8_t *k_scales;
    uint8_t *v_codes;
    uint8_t *v_scales;
    float *weights;
    uint32_t *status;
    int64_t num_pages;
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t device;
} splitzip_kv4_cache;

/*
 * The sequences of one call.  lens[s] counts the tokens of sequence s, the new ones among
 * them; its n = cu_seqlens[s + 1] - cu_seqlens[s] new tokens or queries are rows
 * cu_seqlens[s] .. of the call's tensors and stand at its last n tokens (cu_seqlens NULL: one
 * row a sequence).  total: rows of those tensors.  max_q and max_len say how many queries and
 * tokens a sequence is expected to have; they choose the launch and with it attend's workspace,
 * and the results hold whatever they say.  max_q 0: not known.
 */
typedef struct splitzip_kv4_batch {
    const int32_t *table;
    const int32_t *lens;
    const int32_t *cu_seqlens;
    int64_t table_stride;
    int64_t total;
    int32_t table_width;
    int32_t n_seqs;
    int32_t max_q;
    int32_t max_len;
} splitzip_kv4_batch;

/*
 * Queries [total][q_heads][head_dim] with strides in elements (channels adjacent).  Query head
 * f reads KV head f / (q_heads / kv_heads).  Query i of a sequence stands at token
 * p = len - n + i and sees tokens j <= p with j > p - window or j < sinks; window 0: no window.
 * scale 0: attend counts all of them alike, whatever the query holds; weigh gives NaN for a query
 * that is not finite.
 */
typedef struct splitzip_kv4_queries {
    const void *q;
    int64_t token_stride;
    int64_t head_stride;
    int32_t q_heads;
    int32_t dtype;
    int32_t window;
    int32_t sinks;
    float scale;
} splitzip_kv4_queries;

/*
 * Quantizes k and v [total][kv_heads][head_dim] (strides in elements) into the cache at the
 * sequences' last tokens and sets those tokens' weights to 0.  New tokens at negative positions
 * (more rows than the length) are left out.
 */
int splitzip_kv4_append(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch, const void *k,
                        int64_t k_token_stride, int64_t k_head_stride, const void *v,
                        int64_t v_token_stride, int64_t v_head_stride, int32_t dtype, void *stream);

/*
 * The other way: k and v [total][kv_heads][head_dim], contiguous, from the sequences' last
 * tokens.  Rows at no token of a sequence read as NaN.
 */
int splitzip_kv4_read(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch, void *k, void *v,
                      int32_t dtype, void *stream);

/* Bytes of the workspace that splitzip_kv4_attend wants for this call (0: none; at most 512 MiB). */
int splitzip_kv4_attend_workspace(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch,
                                  const splitzip_kv4_queries *queries, uint64_t *bytes);

/*
 * out [total][q_heads][head_dim] (of the queries' type, contiguous) = softmax over the tokens a
 * query sees of scale q.k, times v; lse f32 [total][q_heads] (optional) = the logarithm of the
 * sum of exp(scale q.k).  A query that sees nothing, or belongs to no sequence, gets out = 0 and
 * lse = -infinity.
 * Sums are held in 32 bits: out is finite where sum exp(s - max s) |v| over those tokens is below 2^128.
 */
int splitzip_kv4_attend(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch,
                        const splitzip_kv4_queries *queries, void *out, float *lse, void *workspace,
                        uint64_t workspace_bytes, void *stream);

/*
 * Adds to the weight of every token and KV head the attention it got: the sum over the queries
 * and the heads of the group of exp(scale q.k - lse), for queries that see the token.  lse f32
 * [total][q_heads] is what splitzip_kv4_attend gave for these queries; one of -infinity adds
 * nothing.  A page that sequences share gets the sum over all of them, added in no fixed order (its
 * last bits may differ from call to call); elsewhere results do not depend on timing.
 */
int splitzip_kv4_weigh(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch,
                       const splitzip_kv4_queries *queries, const float *lse, void *stream);

/*
 * Cuts every sequence to budget tokens a KV head.  A sequence of at most budget tokens keeps
 * all of them; another keeps its first `sinks`, its last `recent` and, of those between, the
 * budget - sinks - recent of the largest weights (equal weights: the lowest token first; a NaN
 * counts as the lowest weight), each KV head for itself.  What is kept moves, in token order,
 * with its weights, to tokens 0 .. of the pages of out_table [n_seqs][>= budget / page_size
 * rounded up], which must share no page with `table`.  out_lens i32 [n_seqs], apart from
 * batch->lens; kept i32 [n_seqs][kv_heads][budget], -1 behind the last.  budget is below 2^31 - 65536.
 * batch->cu_seqlens, total, max_q are not read.
 */
int splitzip_kv4_evict(const splitzip_kv4_cache *cache, const splitzip_kv4_batch *batch,
                       const int32_t *out_table, int64_t out_table_stride, int32_t out_table_width,
                       int32_t budget, int32_t sinks, int32_t recent, int32_t *out_lens, int32_t *kept,
                       void *stream);

#ifdef __cplusplus
}
#endif
#endif
