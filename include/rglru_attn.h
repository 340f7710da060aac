/*
 * rglru_attn.h -- local attention beside the RG-LRU layer: the other temporal
 * mixing of a Griffin stack (S. De's thread on Griffin: recurrent blocks mixed
 * with local multi-query attention; "Beyond Transformer Architecture: Griffin
 * and Google RecurrentGemma", "Core Components of Griffin", 2. Local
 * multi-query attention: a fixed window of past tokens). Three operators, each
 * in the forms of the layer (over a sequence, its backward, one new token):
 *
 *   queries and keys   n = x * rsqrt(mean_d(x^2) + eps) * w          per head
 *                      (n_i, n_{i+r/2}) turned by the angle
 *                      position * base^(-2i/r), i < r/2; the dims r.. stay n
 *   visibility         key j is visible to position p when j <= p and
 *                      (window == 0 or j > p - window or j < sinks)
 *   attention          out = sum_j p_j v_j, p = softmax_j(scale * q . k_j) over
 *                      the visible keys; lse = log sum_j exp(scale * q . k_j);
 *                      a query that sees no key has out = 0, lse = -inf
 *
 * The conventions of rglru.h hold (device pointers owned by the caller,
 * 16-byte alignment, asynchronous calls on `stream`, rglru_status codes, no
 * allocation and no state kept between calls), and
 *   - io is the storage type of every activation, weight and cache; statistics,
 *     log-sums, softmax and accumulators are float.
 *   - Every size is 1 or more; a row without tokens is a length of 0.
 *   - Query head h reads key head h / (Hq / Hkv); Hq is a multiple of Hkv.
 *   - dh is a multiple of 8, at most 256.
 *   - Tensors with strides: element (b, t, h, d) lies at
 *     b * batch + t * token + h * head + d, in elements, each stride a multiple
 *     of 16 bytes and at least dh, so that slices of a fused projection, or
 *     head-major tensors, are read in place. A NULL stride pointer means dense
 *     (B, T, H, dh). Everything else is dense in the shape given.
 *   - Outputs must not overlap inputs.
 *   - dev_status (device int or NULL) as in rglru.h. A page number outside
 *     [0, num_pages), a position past max_pages * page_size or a length past
 *     what its table can name sets RGLRU_ERR_INVALID_ARG there; what it names is
 *     neither read nor written (a key is treated as hidden, and a window stays
 *     where the length puts it). The tensor-core
 *     attention reports RGLRU_ERR_TIMEOUT when one of its bounded waits expires.
 */
#ifndef RGLRU_B200_ATTN_H
#define RGLRU_B200_ATTN_H

#include "rglru.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  long long batch, token, head;
} rglru_strides;

/*
 * Norm of every head of q and k, and the rotation, in one pass.
 *   q (B, T, Hq, dh), k (B, T, Hkv, dh)  io, strided
 *   w_q, w_k (dh)      io, the norms' weights, or NULL for ones
 *   positions (B, T)   int, any sign, or NULL for 0..T-1
 *   q_out, k_out       io, dense (written)
 * rot is the number of rotated dims: 0 <= rot <= dh, a multiple of 16. The angle
 * is formed modulo one turn in 64-bit integers, so far positions lose nothing;
 * sine and cosine are good to 2^-21 for bf16 rows and to the last places for fp32.
 * base > 1 (base >= 1 allowed), eps >= 0, both finite.
 */
int rglru_qk_norm_rope_fwd(const void *q, const rglru_strides *q_strides, const void *k,
                           const rglru_strides *k_strides, const void *w_q, const void *w_k,
                           const int *positions, void *q_out, void *k_out, int B, int T, int Hq,
                           int Hkv, int dh, int rot, double base, float eps, int io,
                           void *stream);

/*
 * The serving form: as rglru_qk_norm_rope_fwd, but the keys, and the values v
 * (B, T, Hkv, dh; strided, copied as they are), go to their slots of a paged
 * cache instead of k_out. Position p of row b lives in page
 * page_table[b * max_pages + p / page_size], slot p % page_size.
 *   k_cache, v_cache (num_pages, page_size, Hkv, dh)  io, written in place
 *   page_table (B, max_pages) int; positions (B, T) int, required
 * A token at a negative position is padding: it is not read, its row of q_out
 * becomes zeros and no slot is written.
 * Two tokens of a call with the same slot leave either one's values there, each
 * 16 bytes of it for themselves.
 */
int rglru_qk_norm_rope_append(const void *q, const rglru_strides *q_strides, const void *k,
                              const rglru_strides *k_strides, const void *v,
                              const rglru_strides *v_strides, const void *w_q, const void *w_k,
                              const int *positions, void *q_out, void *k_cache, void *v_cache,
                              const int *page_table, int num_pages, int page_size, int max_pages,
                              int B, int T, int Hq, int Hkv, int dh, int rot, double base,
                              float eps, int io, int *dev_status, void *stream);

/*
 * Backward of rglru_qk_norm_rope_fwd from its inputs and the gradients of its
 * outputs. dq_out, dk_out, dq, dk: io, dense; dw_q, dw_k (dh) float, written
 * (not added to), or NULL when not wanted. Sums over tokens and heads are taken
 * in a fixed order: the same inputs give the same bits.
 */
size_t rglru_qk_norm_rope_bwd_workspace_bytes(int B, int T, int Hq, int Hkv, int dh, int io);

int rglru_qk_norm_rope_bwd(const void *q, const rglru_strides *q_strides, const void *k,
                           const rglru_strides *k_strides, const void *w_q, const void *w_k,
                           const int *positions, const void *dq_out, const void *dk_out, void *dq,
                           void *dk, float *dw_q, float *dw_k, int B, int T, int Hq, int Hkv,
                           int dh, int rot, double base, float eps, int io, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * Attention of T queries over S keys: query t stands at position t + S - T, so
 * that S > T continues a sequence whose first S - T keys are given (with S < T
 * the first T - S queries see no key).
 *   q (B, T, Hq, dh), k, v (B, S, Hkv, dh)  io, strided
 *   lens (B) int or NULL: row b has only its first lens[b] tokens (S == T then;
 *       values outside [0, T] are clamped). Rows past them are not read, and
 *       out and lse are left as they were there.
 *   out (B, T, Hq, dh) io, lse (B, Hq, T) float or NULL, both dense (written)
 * window >= 0 (0: none), sinks >= 0, scale finite and positive.
 * What lies in key rows that no query of the call sees has no effect, whatever
 * it is. A NaN in q is that query's output, a NaN in k that of the queries that
 * see the key, and so is a score of +inf; a score of -inf counts as a hidden key.
 * A value row that some query sees is taken to be finite (one that
 * is not may reach, with weight zero, queries of the same call that do not see
 * it). bf16 with dh 64, 128 or 256 runs on the tensor cores (weights rounded
 * to bf16 for the product with v, an eighth of them good to 2.6e-6 before that, in
 * lse too), everything else in fp32 on CUDA cores.
 */
int rglru_local_attn_fwd(const void *q, const rglru_strides *q_strides, const void *k,
                         const rglru_strides *k_strides, const void *v,
                         const rglru_strides *v_strides, const int *lens, void *out, float *lse,
                         int B, int T, int S, int Hq, int Hkv, int dh, int window, int sinks,
                         float scale, int io, int *dev_status, void *stream);

/*
 * Backward of rglru_local_attn_fwd, from its inputs, its out and lse and
 * dout = dL/dout (B, T, Hq, dh; dense), with lse constant. (Row sums of dout and out
 * come from out, but for queries that see few keys, 16 at most, from those: the
 * rounding of out would tell there.)
 *   dq (B, T, Hq, dh), dk, dv (B, S, Hkv, dh)  io, dense (written; with lens,
 *   rows past a sequence are left as they were).
 * Key heads shared by several query heads get the sum of their gradients, taken
 * in a fixed order: the same inputs give the same bits.
 * As in the forward, rows past a sequence and keys that no query sees may hold
 * anything, and so may q, out and dout of queries that see no key. All other rows
 * are taken to be finite: one that is not reaches the gradients it has a part in,
 * and may reach, with weight zero, others of its batch row and key head.
 * bf16 with dh 64, 128 or 256 runs on the tensor cores (weights and score
 * gradients rounded to bf16 for their products), everything else in fp32.
 */
size_t rglru_local_attn_bwd_workspace_bytes(int B, int T, int S, int Hq, int Hkv, int dh,
                                            int window, int sinks, int io);

int rglru_local_attn_bwd(const void *q, const rglru_strides *q_strides, const void *k,
                         const rglru_strides *k_strides, const void *v,
                         const rglru_strides *v_strides, const void *out, const float *lse,
                         const void *dout, const int *lens, void *dq, void *dk, void *dv, int B,
                         int T, int S, int Hq, int Hkv, int dh, int window, int sinks,
                         float scale, int io, void *workspace, size_t workspace_bytes,
                         int *dev_status, void *stream);

/*
 * Attention of one new token of each of B sequences over its paged cache (the
 * layout of rglru_qk_norm_rope_append). The token is the last of its sequence:
 * lens[b] counts it, its key and value are in the cache already, and it stands
 * at position lens[b] - 1.
 *   q (B, Hq, dh) io, dense; lens (B) int (0 or less: out row = 0)
 *   out (B, Hq, dh) io, dense (written)
 * Only visible keys are read: pages that hold none may be absent (any entry).
 * The visible keys of a sequence are split over thread blocks when there are
 * few sequences, and the parts are joined in a fixed order. bf16 with dh 64, 128
 * or 256 runs on the tensor cores (weights rounded to bf16 for the product with
 * v), everything else in fp32 on CUDA cores.
 */
size_t rglru_paged_attn_decode_workspace_bytes(int B, int Hq, int Hkv, int dh, int page_size,
                                               int max_pages, int window, int sinks, int io);

int rglru_paged_attn_decode(const void *q, const void *k_cache, const void *v_cache,
                            const int *page_table, const int *lens, void *out, int num_pages,
                            int page_size, int max_pages, int B, int Hq, int Hkv, int dh,
                            int window, int sinks, float scale, int io, void *workspace,
                            size_t workspace_bytes, int *dev_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RGLRU_B200_ATTN_H */
