/*
 * gdn_attention.h -- the attention layers beside the recurrent ones, on a paged
 * key/value cache, for AMD Instinct MI355X (gfx950).  C ABI, in the same
 * library as gdn_paged.h and with its conventions: device memory owned by the
 * caller, calls asynchronous on `stream` that only launch kernels (so they can
 * be captured into a HIP graph), no host synchronization, no allocation; GDN_OK
 * or a negative status set before any launch for what the host can check, the
 * message in gdn_last_error().  Device-side contents (page ids, cu_seqlens,
 * last_page_len) are not validated.
 *
 * The page table is the CSR form of the recurrent layers: sequence b owns the
 * pages page_indices[page_indptr[b] .. page_indptr[b+1]) and holds, after the
 * call's new tokens, (pages - 1) * page_size + last_page_len[b] tokens (none
 * when it has no page; fewer than 2^31 - 4096 in all).  Its n new tokens are the
 * last n of them.  Any page_size >= 1 is served.
 */
#ifndef GDN_ATTENTION_H
#define GDN_ATTENTION_H

#include "gdn_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of queries, keys and values. */
enum { GDN_TYPE_BF16 = 0, GDN_TYPE_F16 = 1, GDN_TYPE_F32 = 2 };

/*
 * Rows [tokens, heads, head_dim] in device memory: the last dimension is dense,
 * tokens and heads sit token_stride and head_stride elements apart (views of a
 * fused projection are such rows).
 */
typedef struct {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} gdn_rows_t;

/*
 * A paged key/value cache: element d of head h of the token at offset i of page
 * p is at k (or v) + p * page_stride + i * token_stride + h * head_stride + d,
 * in elements.  The keys and the values have the same strides, so pages laid
 * out [tokens, heads, dim] and [heads, tokens, dim], apart or interleaved in one
 * allocation, are all such caches.  page_stride and (of pages of more than one token)
 * token_stride are 0 or more, GDN_EUNSUPPORTED otherwise; head_stride may be negative.
 */
typedef struct {
  void* k;
  void* v;
  int64_t page_stride;
  int64_t token_stride;
  int64_t head_stride;
  int32_t page_size;
  int32_t num_seqs;
  const int32_t* page_indices;  /* [page_indptr[num_seqs]] */
  const int32_t* page_indptr;   /* [num_seqs + 1] */
  const int32_t* last_page_len; /* [num_seqs] */
} gdn_kv_cache_t;

/*
 * Rotary positions.  The first rot_dim values of a head form rot_dim / 2 pairs:
 * (x_i, x_{i + rot_dim/2}), or (x_{2i}, x_{2i+1}) when interleaved.  At position
 * t pair i becomes
 *     (a c - b s, b c + a s),  c = table[t][i], s = table[t][rot_dim/2 + i],
 * or, when transposed, (a c + b s, b c - a s): the transposed map, which takes
 * the gradient of the rotated rows to the gradient of the rows.  Values past
 * rot_dim pass unchanged.  Arithmetic in fp32, one rounding at the end.
 * A position outside the table's rows gives NaN in the rotated values (the
 * table is never read there).
 */
typedef struct {
  const float* table; /* [table_rows, rot_dim], dense: cosines, then sines */
  int64_t table_rows;
  int32_t rot_dim;     /* even, 2 .. head_dim */
  int32_t interleaved;
  int32_t transposed;
} gdn_rope_t;

/*
 * gdn_rope_table -- the table of a gdn_rope_t for positions 0 .. rows - 1:
 * angles position * f_i, f_i = base^(-2 i / rot_dim), computed in fp64 and
 * stored as fp32(magnitude * cos), fp32(magnitude * sin).  For contexts longer
 * than the model was trained on the frequencies are changed:
 *   GDN_ROPE_PLAIN   none.
 *   GDN_ROPE_LINEAR  f_i / factor.
 *   GDN_ROPE_BASE    base * factor^(rot_dim / (rot_dim - 2)): the lowest
 *                    frequency divided by factor, the highest unchanged.
 *   GDN_ROPE_BANDS   by the turns r_i = original * f_i / (2 pi) that a pair makes
 *                    over the original context: f_i * ((1 - w) / factor + w),
 *                    w = (r_i - low_turns) / (high_turns - low_turns) clamped to
 *                    0 .. 1.
 * Errors: GDN_EINVAL for a null table, rows < 0, rot_dim odd, < 2 or > 1024,
 * base <= 0, factor <= 0, magnitude not finite, an unknown scaling, BASE with
 * rot_dim 2, BANDS without original > 0 and high_turns > low_turns.
 */
enum { GDN_ROPE_PLAIN = 0, GDN_ROPE_LINEAR = 1, GDN_ROPE_BASE = 2, GDN_ROPE_BANDS = 3 };
typedef struct {
  int32_t scaling;
  double base;
  double factor;
  double original;
  double low_turns;
  double high_turns;
  double magnitude;
} gdn_rope_scaling_t;
int gdn_rope_table(const gdn_rope_scaling_t* scaling, float* table, int64_t rows, int32_t rot_dim,
                   hipStream_t stream);

/*
 * gdn_rope -- rotates the rows of q (num_q_heads heads) and k (num_k_heads; 0:
 * none) at the given positions into q_out and k_out, which may be the inputs.
 *   positions [num_tokens], int32, or int64 when index_dtype is GDN_INDEX_INT64.
 * Errors: GDN_EINVAL (null pointers, negative sizes, head_dim < 1, rot_dim odd
 * or outside 2 .. head_dim, unknown types; more than 65536 heads, a head_dim over
 * 65536, or so many values a token that its threads pass 2^31), GDN_ELAUNCH.
 */
int gdn_rope(const gdn_rope_t* rope, int32_t dtype, int32_t head_dim, int32_t num_q_heads,
             int32_t num_k_heads, int64_t num_tokens, const void* positions, int32_t index_dtype,
             const gdn_rows_t* q, const gdn_rows_t* k, const gdn_rows_t* q_out,
             const gdn_rows_t* k_out, hipStream_t stream);

/*
 * Norms of query and key heads, before the rotation: a head's row x becomes
 *     x (sum x^2 / head_dim + eps)^(-1/2) (offset + weight),
 * sums in fp32, with one rounding after the rotation.  head_dim at most 512.
 */
typedef struct {
  const void* q_weight; /* [head_dim], any alignment; NULL: queries are not normed */
  const void* k_weight; /* [head_dim]; NULL: keys are not normed */
  int32_t weight_dtype; /* the rows' type, or GDN_TYPE_F32 */
  float eps;            /* >= 0 */
  float offset;
} gdn_norm_t;

/*
 * gdn_norm_rope -- gdn_rope of the normed rows of q and k, in one pass.  q_out
 * and k_out may be the inputs.  Errors as gdn_rope, and GDN_EINVAL for a null
 * norm, a null weight of a tensor that has heads, a weight_dtype that is neither
 * the rows' nor fp32, eps < 0 or not finite, offset not finite;
 * GDN_EUNSUPPORTED for a head_dim over 512.
 */
int gdn_norm_rope(const gdn_norm_t* norm, const gdn_rope_t* rope, int32_t dtype, int32_t head_dim,
                  int32_t num_q_heads, int32_t num_k_heads, int64_t num_tokens, const void* positions,
                  int32_t index_dtype, const gdn_rows_t* q, const gdn_rows_t* k,
                  const gdn_rows_t* q_out, const gdn_rows_t* k_out, hipStream_t stream);

/*
 * gdn_norm_rope_backward -- from the inputs q and k of a gdn_norm_rope call and
 * the gradients of its outputs, those of q and k (q_grad, k_grad: rows that may
 * lie over the inputs' or the outputs' gradients', with the same strides, and
 * otherwise share no memory with them) and of the weights (q_weight_grad,
 * k_weight_grad: [head_dim] of the weights' type, sums over all rows in fp32 in
 * an order that the sizes fix, so equal inputs give equal sums; zeros for no
 * tokens).  The workspace is 256-byte aligned, of
 * gdn_norm_rope_backward_workspace_size bytes (0 on bad sizes).
 * Errors as gdn_norm_rope, GDN_EWORKSPACE, and GDN_EINVAL for gradients whose rows
 * share memory they must not (where strides differ: whose spans do), the queries' with
 * the keys' rows among it.
 */
size_t gdn_norm_rope_backward_workspace_size(int32_t head_dim, int32_t num_q_heads,
                                             int32_t num_k_heads, int64_t num_tokens);
int gdn_norm_rope_backward(const gdn_norm_t* norm, const gdn_rope_t* rope, int32_t dtype,
                           int32_t head_dim, int32_t num_q_heads, int32_t num_k_heads,
                           int64_t num_tokens, const void* positions, int32_t index_dtype,
                           const gdn_rows_t* q, const gdn_rows_t* k, const gdn_rows_t* q_out_grad,
                           const gdn_rows_t* k_out_grad, const gdn_rows_t* q_grad,
                           const gdn_rows_t* k_grad, void* q_weight_grad, void* k_weight_grad,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * gdn_kv_append_paged -- writes the keys and values of a batch's new tokens to
 * the cache, the keys rotated on the way when `rope` is not NULL, and rotates
 * the queries of the same tokens into q_out in the same launch when q is not
 * NULL.  The position of a new token is its place in its sequence.
 *   cu_seqlens [num_seqs + 1]: sequence b's new tokens are rows cu_seqlens[b] ..
 *   cu_seqlens[b+1]; NULL: one new token per sequence (total_tokens = num_seqs).
 *   k, v: rows of the new tokens, cache->num heads = num_kv_heads.
 * A new token whose place in its sequence is negative (more new tokens than the
 * page table holds) is not written to the cache.
 * Errors: GDN_EINVAL (null pointers, negative sizes, page_size < 1, unknown
 * types, rotary arguments as in gdn_rope), GDN_ELAUNCH.
 */
int gdn_kv_append_paged(const gdn_rope_t* rope, int32_t dtype, int32_t head_dim,
                        int32_t num_q_heads, int32_t num_kv_heads, const int32_t* cu_seqlens,
                        int64_t total_tokens, const gdn_rows_t* k, const gdn_rows_t* v,
                        const gdn_kv_cache_t* cache, const gdn_rows_t* q, const gdn_rows_t* q_out,
                        hipStream_t stream);

/*
 * A cache of 8 bits: the gdn_kv_cache_t holds e4m3 codes (1 sign, 4 exponent, 3
 * fraction bits; no infinities), its strides in codes, rows 16-byte aligned, and
 * a value is its code times the scale of its block of `block` tokens of a page
 * and head: scale j of head h of page p, for the tokens j * block .. of the page,
 * is at k (or v) + p * page_stride + j * block_stride + h * head_stride.  Scales
 * are powers of two between 2^-100 and 2^120, as the append writes them; readers
 * take nothing else.  The block is a multiple of 16 tokens that divides the page.
 */
typedef struct {
  float* k;
  float* v;
  int64_t page_stride;
  int64_t block_stride;
  int64_t head_stride;
  int32_t block;
} gdn_kv_scales_t;

/*
 * gdn_kv_append_paged_ext -- gdn_kv_append_paged with the queries and keys normed
 * before the rotation (norm; NULL: neither) and, where scales is not NULL, into a
 * cache of 8 bits.  There a block's scale is the least power of two with which
 * the largest magnitude of the new tokens' (normed, rotated) values in it is at
 * most 448, and no less than the block's own where tokens before them lie in it:
 * if the scale grows their codes are rounded to the new one.  A block that the
 * new tokens open takes a new scale, whatever it held.  A value is rounded once,
 * to nearest, ties to even; values that are not finite are stored as NaN and count
 * for no scale, and none is stored over 15/8 of the rows' type's highest power of two
 * (61,440 in fp16: the next code is beyond it).  Slots behind the new tokens are left as
 * they are, and with norm or scales also rows of q_out behind the last sequence.
 * Errors as gdn_kv_append_paged and gdn_norm_rope (but that a null weight leaves
 * its heads as they are), GDN_EINVAL for null or unaligned scales, a bad block,
 * or an 8-bit cache that is not 16-byte aligned in every stride and address;
 * GDN_EUNSUPPORTED for an 8-bit cache of fp32 rows, of heads other than 64, 128
 * or 256, with rows of k, v, q or q_out that are not 4-byte aligned, a rot_dim that
 * is not a multiple of 4 or a rope table that is not 8-byte aligned.
 */
int gdn_kv_append_paged_ext(const gdn_norm_t* norm, const gdn_rope_t* rope, int32_t dtype,
                            int32_t head_dim, int32_t num_q_heads, int32_t num_kv_heads,
                            const int32_t* cu_seqlens, int64_t total_tokens, const gdn_rows_t* k,
                            const gdn_rows_t* v, const gdn_kv_cache_t* cache,
                            const gdn_kv_scales_t* scales, const gdn_rows_t* q,
                            const gdn_rows_t* q_out, hipStream_t stream);

/*
 * gdn_kv_read_paged -- the last tokens of each sequence, as the append counts its
 * new ones, back from a cache of 8 bits: rows cu_seqlens[b] .. of k and v (of
 * `dtype`, 16-byte aligned) get the values of the last cu_seqlens[b+1] -
 * cu_seqlens[b] tokens of sequence b (cu_seqlens NULL: one each), exact in bf16 and
 * fp32 and rounded in fp16.  A row whose sequence holds fewer tokens is zeros, rows
 * behind the last sequence are left as they are.
 * Errors: GDN_EINVAL (null pointers, negative sizes, num_kv_heads < 1, an unknown
 * type, total_tokens other than num_seqs without cu_seqlens, null or unaligned
 * scales, a bad block, a cache or rows of k and v that are not 16-byte aligned in every
 * stride and address), GDN_EUNSUPPORTED (heads other than 64, 128 or 256), GDN_ELAUNCH.
 */
int gdn_kv_read_paged(int32_t dtype, int32_t head_dim, int32_t num_kv_heads,
                      const int32_t* cu_seqlens, int64_t total_tokens, const gdn_kv_cache_t* cache,
                      const gdn_kv_scales_t* scales, const gdn_rows_t* k, const gdn_rows_t* v,
                      hipStream_t stream);

/*
 * What the attention calls compute, for query row i (position t in its
 * sequence) and q-head h, which reads kv-head h / (num_q_heads / num_kv_heads):
 *     x_j = scale * q . k_j                 (scale <= 0: 1/sqrt(head_dim))
 *     x_j = softcap * tanh(x_j / softcap)   (softcap > 0)
 *     o   = sum_j e^{x_j} v_j / sum_j e^{x_j},   lse = log sum_j e^{x_j}
 * over the tokens j of the sequence with j <= t (causal; otherwise all of them)
 * and, for window > 0, j > t - window.  A row that sees no token gives o = 0 and
 * lse = -inf; one whose scores are all -inf gives o = NaN (0 / 0) and lse = -inf.
 * Scores, references, sums and the output accumulate in fp32.  In the chunk call
 * e^{x} enters the product with v rounded to the element type, as the scores'
 * matrix product takes q and k in theirs (bf16: 2.2e-3 of the output in the mean,
 * where the output's own rounding is 1.6e-3; in fp16, whose least step is 2^-24,
 * each weight is off by up to 2^-32 of the row's sum besides); the decode call
 * passes it as the sum of two such values and adds nothing visible.  A capped score
 * is off by up to 2^-19 of itself, or, in the chunk call and for caps of up to 64, by
 * up to 2^-21 of the cap; caps over 1e30 count as none.  Cache slots that no sequence
 * holds are never read, whatever they contain; keys and values a row does not see do
 * not reach it, and infinities and NaN it sees enter it as themselves.
 */
typedef struct {
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim; /* 64, 128 or 256 */
  int32_t dtype;    /* GDN_TYPE_BF16 or GDN_TYPE_F16: q, the cache and o */
  float scale;
  float softcap;
  int32_t window;
  int32_t causal;
} gdn_attention_dims_t;

/*
 * Workspace bytes of any attention call for at most total_tokens query rows
 * in at most num_seqs sequences (an upper bound that never decreases as either
 * grows), 256-byte aligned.  0 on bad dims.  The second form: of calls over 16-bit
 * caches alone (codes 0), or over 8-bit caches alone.
 */
size_t gdn_attention_workspace_size(const gdn_attention_dims_t* dims, int64_t total_tokens,
                                    int32_t num_seqs);
size_t gdn_attention_workspace_size_ext(const gdn_attention_dims_t* dims, int32_t codes,
                                        int64_t total_tokens, int32_t num_seqs);

/*
 * gdn_attention_prefill_paged -- attention of the batch's new tokens (q rows
 * cu_seqlens[b] .. cu_seqlens[b+1], any count per sequence, none included) over
 * everything their sequences hold in the cache, the new tokens themselves
 * among it: append first, then attend.
 *   out: rows of total_tokens tokens that share no memory with q (with strides other
 *   than q's: nor lie among its rows); lse [total_tokens, num_q_heads] or NULL.
 * Errors: GDN_EINVAL (null pointers, negative sizes or window, page_size < 1,
 * rows or a cache that are not 16-byte aligned in every stride and address, out
 * over q),
 * GDN_EUNSUPPORTED (head_dim, dtype, num_q_heads not a multiple of
 * num_kv_heads), GDN_EWORKSPACE, GDN_ELAUNCH.
 */
int gdn_attention_prefill_paged(const gdn_attention_dims_t* dims, const gdn_rows_t* q,
                                const int32_t* cu_seqlens, int64_t total_tokens,
                                const gdn_kv_cache_t* cache, const gdn_rows_t* out, float* lse,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * gdn_attention_decode_paged -- one token per sequence: q and out hold num_seqs
 * rows, the query of sequence b sits at its last position.  A sequence without a
 * page gives o = 0 and lse = -inf.  out may be q itself (the same address and
 * strides).  Errors as gdn_attention_prefill_paged.
 */
int gdn_attention_decode_paged(const gdn_attention_dims_t* dims, const gdn_rows_t* q,
                               const gdn_kv_cache_t* cache, const gdn_rows_t* out, float* lse,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * The same calls with first tokens that stay visible beside a window, and over
 * caches of 8 bits.
 *   sinks: with a window a row sees token j <= t (causal) also if j < sinks.
 *     Without one it means nothing.
 *   scales: of an 8-bit cache, or NULL for one of dims->dtype.  The result is that
 *     of a cache that holds the values, code times scale, rounded to dims->dtype
 *     (exact in bf16; in fp16 magnitudes over 65,504 become infinite, and an output
 *     that sees one infinite or NaN).
 * Errors as the calls above, and GDN_EINVAL for sinks < 0 or over 2^30, null or
 * unaligned scales or a bad block; GDN_EUNSUPPORTED for chunks over an 8-bit cache
 * whose token stride reaches 2^30 / page_size.
 */
int gdn_attention_prefill_paged_ext(const gdn_attention_dims_t* dims, int32_t sinks,
                                    const gdn_rows_t* q, const int32_t* cu_seqlens,
                                    int64_t total_tokens, const gdn_kv_cache_t* cache,
                                    const gdn_kv_scales_t* scales, const gdn_rows_t* out, float* lse,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream);
int gdn_attention_decode_paged_ext(const gdn_attention_dims_t* dims, int32_t sinks,
                                   const gdn_rows_t* q, const gdn_kv_cache_t* cache,
                                   const gdn_kv_scales_t* scales, const gdn_rows_t* out, float* lse,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTENTION_H */
