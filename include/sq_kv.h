/*
 * sq_kv.h - a microscaled (MX) cache of keys and values: rotary positions and
 * the quantized write in one call, the way back, and the attention over the
 * cache.  Same library (libsq.so), conventions and status codes as sq.h:
 * device pointers owned by the caller, work enqueued on `stream`, arguments
 * checked on the host before anything is enqueued, no allocation, no
 * synchronization, capturable in a HIP graph.
 *
 * The cache is `pages` pages of `page` tokens.  For each page and head the
 * rows of its tokens follow one another:
 *   kq, vq  [pages, heads, page, dim / 2] (SQ_MX_E2M1) or [.., dim]
 *           (SQ_MX_E4M3) code bytes
 *   ks, vs  [pages, heads, page, dim / 32] scale bytes
 * with the codes, blocks of 32 channels and quantization of sq_mx.h.  dim is
 * 64, 128 or 256; page a power of two from 16 to 2^20; 1 <= pages,
 * 1 <= heads <= 65535, and pages * page < 2^31.  A token's slot is its page's
 * number times `page` plus its place in the page.  A block table [B, width]
 * of int32 names the pages of B sequences in order: token t of sequence b is
 * at place t % page of page table[b, t / page].  Of a row only the entries
 * that its sequence's tokens need are read.
 *
 * Alignment: all of q, k, v, y, kq, vq, their rows' strides in bytes, the
 * multipliers and the workspace 16 bytes; ks, vs 4 bytes; other arrays their
 * element size.  What a call writes (the workspace and, in a write, the cache's
 * four arrays among it) shares no byte with what it reads or with one another:
 * SQ_ERR_ARG.
 */
#ifndef SQ_KV_H
#define SQ_KV_H

#include "sq_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct sq_kv_cache {
    uint8_t *kq, *ks, *vq, *vs;
    int64_t pages, heads, page, dim;
    int fmt; /* SQ_MX_E2M1 or SQ_MX_E4M3 */
} sq_kv_cache;

typedef enum { SQ_ROPE_HALF = 0, SQ_ROPE_INTERLEAVED = 1 } sq_rope_layout;

/*
 * Rotary positions of queries and keys, and the quantized write of keys and
 * values.  For token t at position p = positions[t], with x one head's row:
 *   a_i = fl64(p * inv_freq[i]), c_i = fl32(cos(a_i) * amplitude),
 *   s_i = fl32(sin(a_i) * amplitude), i < rotary / 2
 *   pairs (x1, x2) = (x[i], x[i + rotary / 2]) (SQ_ROPE_HALF) or
 *   (x[2 i], x[2 i + 1]) (SQ_ROPE_INTERLEAVED) become
 *   y1 = fl(fl(x1 c_i) - fl(x2 s_i)), y2 = fl(fl(x2 c_i) + fl(x1 s_i)) in fp32;
 *   channels from `rotary` on stay as they are
 *   q_out[t] = y, times q_mul (in fp32), rounded to the type
 *   the key's row at slots[t] holds y, times k_mul (in fp32), quantized; the
 *   value's row v as it is, quantized
 *   q       [T, q_heads, dim] of dt (SQ_F32, SQ_F16, SQ_BF16) or NULL (keys
 *           and values alone); rows at q + t * q_stride[0] + head * q_stride[1]
 *           elements; k, v [T, heads, dim] of dt with strides of their own
 *   positions int64 [T], inv_freq fp64 [rotary / 2]: NULL with rotary == 0
 *           (nothing is rotated)
 *   rotary  0, or a multiple of 16 up to dim
 *   q_mul   fp32 [q_heads, dim] or NULL, k_mul fp32 [heads, dim] or NULL
 *           (smoothing: a key's large channels divided, the query's multiplied)
 *   slots   int64 [T]; a token whose slot is negative or past the cache is
 *           not written (its query is)
 *   q_out   [T, q_heads, dim] dense, of dt
 * Two tokens of a call with the same slot leave that row undefined.
 * T <= 2^24, q_heads <= 65535.
 */
int sq_rope_quantize_kv_mx(const void *q, const int64_t q_stride[2], const void *k,
                           const int64_t k_stride[2], const void *v, const int64_t v_stride[2],
                           int dt, int64_t T, int64_t q_heads, const int64_t *positions,
                           const double *inv_freq, int64_t rotary, double amplitude, int layout,
                           const float *q_mul, const float *k_mul, const int64_t *slots,
                           const sq_kv_cache *cache, void *q_out, void *stream);

/*
 * The values of cached tokens, dense: row cu[b] + t of k and v [total, heads,
 * dim] is token t of sequence b, for t < cu[b + 1] - cu[b], in dt with
 * round-to-nearest-even.
 *   table int32 [B, width], cu int32 [B + 1], not descending from 0
 * Rows from cu[B] on are left as they were.  A token whose page is not in the
 * cache, or that lies past the table, gives NaN.  B, total <= 2^24.
 */
int sq_dequantize_kv_mx(const sq_kv_cache *cache, const int32_t *table, int64_t B, int64_t width,
                        const int32_t *cu, int64_t total, void *k, void *v, int dt, void *stream);

/*
 * Attention of new tokens over the cache, new tokens included (they are
 * written before).  Sequence b has n_k = seq_lens[b] tokens in the cache, the
 * last n_q = cu_q[b + 1] - cu_q[b] of them the queries q[cu_q[b] ..].  Query i
 * is at place p = n_k - n_q + i and sees the keys j with
 *   j <= p (causal != 0) or j < n_k (causal == 0), and
 *   j > p - window (window > 0)
 *   y = sum_j w_j v_j, w = softmax over those j of scale * (q . k_j)
 * A query that sees no key gets 0, one that sees keys but scores all of them
 * -inf NaN (0 / 0).  Query head h reads key head h / (q_heads /
 * heads).  Keys and values are the cache's, read in dt (round-to-nearest-even;
 * bf16 holds all in its range but those of e4m3 blocks with e < 3; in fp16
 * magnitudes from 65520 on become infinite).  Products are summed in fp32, the softmax's
 * maximum and sum are fp32; its weights are rounded to dt for the product with
 * the values (in fp16 those below 2^-21 of a row's largest by up to 2^-32 of
 * it).  They are at most 2^15 in fp16 and 2^8 in bf16 before they are divided by
 * their sum, so that bf16 values of 2^120 over their number and more may give
 * an infinity for a finite mean.
 *   q        [T, q_heads, dim] of dt (SQ_F16 or SQ_BF16), strides as above
 *   table    int32 [B, width], seq_lens int32 [B]
 *   cu_q     int32 [B + 1], not descending from 0, cu_q[B] <= T; or NULL: T ==
 *            B, one query a sequence
 *   max_q    no sequence has more queries (1 with cu_q NULL): rows of a
 *            sequence that has more may be left as they were
 *   y        [T, q_heads, dim] dense, of dt; rows from cu_q[B] on are left as
 *            they were
 *   workspace of sq_attention_kv_mx_workspace(..) bytes, used by this call
 *            alone while it runs
 * A key or value whose page is not in the cache counts as NaN; the queries of
 * a sequence with seq_lens[b] > width * page get NaN; a negative length counts
 * as 0.  An infinity or NaN of a key or value reaches the queries that
 * see it and no others.  The same call gives the same bits every time; a
 * sequence's bits may depend on the others of the call.
 * q_heads % heads == 0, q_heads <= 65535, T <= 2^24, T * q_heads <= 2^29,
 * B * heads <= 2^22, width * page <= 2^30, width * page / 128 * heads <= 2^30
 * (SQ_ERR_UNSUPPORTED above), finite scale, max_q >= 1 where T, B > 0.  T == 0
 * or B == 0 enqueues nothing.
 */
int sq_attention_kv_mx(const void *q, const int64_t q_stride[2], int dt, int64_t T,
                       int64_t q_heads, const sq_kv_cache *cache, const int32_t *table, int64_t B,
                       int64_t width, const int32_t *seq_lens, const int32_t *cu_q, int64_t max_q,
                       float scale, int causal, int64_t window, void *y, void *workspace,
                       size_t workspace_bytes, void *stream);

/* Bytes of workspace for such a call; 0 for arguments that it would refuse. */
size_t sq_attention_kv_mx_workspace(int64_t T, int64_t q_heads, const sq_kv_cache *cache,
                                    int64_t B, int64_t width, int64_t max_q);

#ifdef __cplusplus
}
#endif

#endif /* SQ_KV_H */
