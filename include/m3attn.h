/*
 * m3attn.h -- C ABI of libm3scan, attention next to the recurrent core: causal attention over whole
 * prompts with its gradient, and for decoding a paged cache of keys and values that is appended to (with
 * the rotation of positions on the way) and attended to by one token per sequence.
 *
 * (Stacks of this core are described as hybrids with an attention layer without positions after every five of
 * the core's: papernotes.org summary of Mamba-3, retrieval; bud-325 notes.)
 *
 * The conventions of m3scan.h hold for every entry point here: device pointers owned by the caller,
 * validation on the host, kernels enqueued on `stream` and nothing else (no allocation, no
 * synchronisation; all calls may be captured into a HIP graph), m3_status results with m3_last_error(), a
 * gfx950 GPU as the current device.  Further:
 *  - Heads.  `heads` query heads share `kv_heads` key heads in groups of heads / kv_heads consecutive
 *    ones.  A head has head_dim elements: a multiple of 8, at most 128.
 *  - Strides.  Tensors of heads ([b, L, H, D] or packed [T, H, D]) are given by the distances in elements between
 *    consecutive sequences, tokens and heads; the D elements of a head are dense.  {0, 0, 0} means dense
 *    [b, L, H, D].  Heads before tokens ([b, H, L, D]) or slices of a wider projection are other
 *    strides.  Strides are not negative, and tokens are less than 2^24 bytes apart.
 *  - Alignment.  Heads start on 16-byte boundaries (pointers and strides); other pointers are aligned to their
 *    element size, workspaces to 16 bytes.
 *  - Outputs must not overlap inputs or one another, except where a call allows it, nor themselves (a stride of 0
 *    over more than one element is for inputs).  Tensors may be slices of one buffer whose tokens are equally far
 *    apart.
 *  - Packed batches.  cu_seqlens [b + 1] int32: sequence s holds tokens cu[s] .. cu[s+1]-1, cu[0] = 0,
 *    nondecreasing, cu[b] <= T.  Rows at and past cu[b] are neither read nor written.  The distance between
 *    sequences is not used.
 *  - Workspaces are scratch: nothing in them has to survive the call or to be cleared before it.  Two
 *    calls that may run at the same time need a workspace each.
 *  - Equal inputs give equal bits: no result depends on scheduling.
 */
#ifndef M3ATTN_H
#define M3ATTN_H

#include "m3scan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t batch, token, head;
} m3_head_strides;

/* ------------------------------------------------------------------------ whole prompts */

typedef struct {
    int64_t batch;      /* b: sequences                                                       */
    int64_t seqlen;     /* L: tokens per sequence; packed: T, the tokens of the whole batch   */
    int64_t heads;      /* Hq, a multiple of kv_heads                                         */
    int64_t kv_heads;
    int64_t head_dim;   /* D                                                                  */
    m3_head_strides q, k, v, o;
    m3_head_strides dout, dq, dk, dv; /* backward                                             */
    int32_t io;         /* m3_dtype of q, k, v, o and their gradients                         */
    uint32_t flags;     /* 0                                                                  */
    float scale;        /* positive, at most 2.3e38; 0: 1 / sqrt(D)                           */
} m3_attn_dims;

/*
 * m3_attention -- causal attention of every token to itself and the tokens before it in its sequence:
 *
 *   s_ij = scale q_i . k_j  (j <= i),  lse_i = log sum_j exp(s_ij),  o_i = sum_j exp(s_ij - lse_i) v_j
 *
 * For: the forward pass of training, prefill.  Scores, maxima, sums and o are fp32; with bf16 io the
 * probabilities are rounded to bf16 for their product with v (relative to the largest score of their row so
 * far, within 2^8).  q . k may be any fp32 number; beyond them it is infinite.  A row whose scores are all
 * -infinity is NaN (0 / 0).  What later tokens hold, infinities and NaN included, does not reach a row.
 *
 *   q        [b, L, Hq, D] or [T, Hq, D] io;  k, v with Hkv heads            required
 *   o        like q                                                         required
 *   lse      [b, Hq, L], packed [Hq, T] f32, dense: read by m3_attention_backward    NULL: not wanted
 */
m3_status m3_attention(const m3_attn_dims* dims, const int32_t* cu_seqlens, const void* q, const void* k,
                       const void* v, void* o, float* lse, hipStream_t stream);

/*
 * m3_attention_backward -- gradients of m3_attention.  With p_ij = exp(s_ij - lse_i) and the loss's gradient
 * dout of o:
 *
 *   delta_i = dout_i . o_i,  ds_ij = p_ij (dout_i . v_j - delta_i)
 *   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dout_i
 *
 * dk and dv are summed over the query heads of their group.  With bf16 io, p and ds are rounded to bf16 for
 * their products, and delta of a row that sees at most 128 keys is sum_j p_ij (dout_i . v_j) / sum_j p_ij, the same
 * but for o's rounding; sums are fp32.  p is off by |lse| 2^-23 of itself, as much as lse is: it has no digits
 * where scores reach 2^24, and from 2^30 on gradients may not be finite.  An infinity or NaN in a row of an input
 * makes gradients of up to 31 other rows of its block of 32 tokens NaN beside those that the formulas make so.
 *
 *   o, lse     what m3_attention wrote for the same dims, offsets and inputs      required
 *   dout       like o                                                            required
 *   dq, dk, dv like q, k, v                                                      required
 *   workspace  m3_attention_backward_workspace_bytes(dims, packed) bytes
 */
size_t m3_attention_backward_workspace_bytes(const m3_attn_dims* dims, int packed);
m3_status m3_attention_backward(const m3_attn_dims* dims, const int32_t* cu_seqlens, const void* q,
                                const void* k, const void* v, const void* o, const float* lse,
                                const void* dout, void* dq, void* dk, void* dv, void* workspace,
                                size_t workspace_bytes, hipStream_t stream);

/* -------------------------------------------------------------------------- paged cache */

/*
 * A cache is num_pages pages of page_size tokens.  Page p, head h and place i in the page are p * page + h *
 * head + i * token elements from the cache's start ({0, 0, 0}: dense [num_pages, kv_heads, page_size, D]).
 * page_table [b, table_width] int32 holds each sequence's pages in order: position t of sequence s is in page
 * page_table[s][t / page_size] at place t % page_size.  A page number outside 0 .. num_pages - 1 is no page:
 * nothing is written there, and nothing is attended to.
 */
typedef struct {
    int64_t page, token, head;
} m3_page_strides;

typedef struct {
    int64_t batch;      /* b: sequences                                                       */
    int64_t seqlen;     /* append: new tokens per sequence; packed: T, those of the batch; step: 1 */
    int64_t heads;      /* Hq, a multiple of kv_heads                                         */
    int64_t kv_heads;
    int64_t head_dim;   /* D                                                                  */
    int64_t num_pages;
    int64_t page_size;
    int64_t table_width;
    int64_t rotary_dim; /* append: elements of a head that are rotated, a multiple of 8       */
    m3_page_strides k_cache, v_cache;
    m3_head_strides q, k, v, q_out, k_out; /* append                                          */
    m3_head_strides o;  /* step (token is not used)                                           */
    int32_t io;         /* m3_dtype of the caches and of q, k, v, q_out, k_out, o             */
    uint32_t flags;     /* append: M3_ROTATE_HALVES or 0; step: 0                             */
    float scale;        /* step: positive, at most 2.3e38; 0: 1 / sqrt(D)                     */
} m3_cache_dims;

/* m3_cache_dims.flags: pairs are elements (k, k + rotary_dim / 2), else (2k, 2k + 1), as the core's are */
#define M3_ROTATE_HALVES 1u

/*
 * m3_cache_append -- new keys and values into the cache, with the rotation of positions on the way:
 * token i of sequence s's n new ones has position t = lens[s] - n + i; its pair number k of keys and queries
 * is turned by the angle t * inv_freq[k],
 *
 *   (a, b) -> (a cos - b sin, a sin + b cos),
 *
 * and elements from rotary_dim on are copied.  Angles are computed in fp64, products in fp32.  With the
 * frequencies' signs turned it is the rotation's inverse, and with it its gradient.
 *
 *   lens       [b] int32: tokens of each sequence in the cache, the new ones counted in; NULL: n
 *   inv_freq   [rotary_dim / 2] f32                               required when rotary_dim is not 0
 *   q, q_out   [b, n, Hq, D] io, packed [T, Hq, D]; q_out may be q itself (same strides)
 *                                                                 both NULL: no queries
 *   k, v       [b, n, Hkv, D] io, packed [T, Hkv, D]              k required, v with the caches
 *   k_out      like k: the rotated keys; may be k itself (same strides)  NULL: not wanted
 *   k_cache, v_cache, page_table    all NULL: only q_out and k_out are written
 * Tokens whose position is negative, past the table or on no page are not cached; a place that two tokens
 * of one call belong to holds either (pages of different sequences may be shared, as long as no new token
 * is written to a shared page).
 */
m3_status m3_cache_append(const m3_cache_dims* dims, const int32_t* cu_seqlens, const int32_t* lens,
                          const float* inv_freq, const void* q, const void* k, const void* v, void* q_out,
                          void* k_out, void* k_cache, void* v_cache, const int32_t* page_table,
                          hipStream_t stream);

/*
 * m3_attention_step -- one token per sequence over the cache: with s_j = scale q . k_j over the positions j <
 * lens[s] (m3_cache_append's lens, so that a token attends to itself),
 *
 *   lse = log sum_j exp(s_j),  o = sum_j exp(s_j - lse) v_j;  no position: o = 0, lse = -infinity
 *
 * For: decoding.  Reads every page once; long sequences are cut into pieces that run at the same time.
 * Scores, sums and partial results are fp32, their range as m3_attention's; with bf16 io the probabilities are
 * rounded to bf16 for their product with v.  Positions whose scores are all -infinity make o NaN, as a prompt's
 * row, and lse -infinity.  lens[s] past table_width * page_size counts as that.
 *
 *   q          [b, Hq, D] io, strides dims->q (batch, head)              required
 *   o          like q, strides dims->o; may be q itself (same strides)   required
 *   lse        [b, Hq] f32                                               NULL: not wanted
 *   workspace  m3_attention_step_workspace_bytes(dims) bytes; the size is for the current device
 */
size_t m3_attention_step_workspace_bytes(const m3_cache_dims* dims);
m3_status m3_attention_step(const m3_cache_dims* dims, const void* q, const void* k_cache,
                            const void* v_cache, const int32_t* page_table, const int32_t* lens, void* o,
                            float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* M3ATTN_H */
