/*
 * smla_prompt — prompts in the expanded form of latent attention. Where a prompt
 * is dense (no selection), the cached latent rows are turned into keys and
 * values of each head (a product with the model's up-projection, the caller's own)
 * and attention runs over those: cheaper per key than the latent form of smla_serve.h
 * once many query tokens share a key. These calls are what stands around that product:
 * rotation tables, the rotation of queries and keys, cache rows read back as
 * bf16 values, and the attention over packed prompts.
 *
 * The conventions of smla.h and smla_serve.h hold.
 */
#ifndef SMLA_PROMPT_H_
#define SMLA_PROMPT_H_

#include "smla_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * smla_rope_table — cosines and sines of the positions first .. first + n - 1.
 *
 *   w_i = base^(-2 i / dim), i = 0 .. dim / 2 - 1, and for long contexts
 *   original = 0:  w'_i = w_i / factor                         (factor 1: as it is)
 *   original > 0:  w'_i = w_i (1 - r_i) + w_i / factor r_i,  r_i = clamp((i - low) / (high - low), 0, 1),
 *                  low  = max(floor(dim ln(original / (2 pi beta_fast)) / (2 ln base)), 0),
 *                  high = min(ceil(dim ln(original / (2 pi beta_slow)) / (2 ln base)), dim - 1)
 *                  (high - low at least 0.001): pairs that turn more than beta_fast times
 *                  over `original` positions keep their speed, slow ones are stretched.
 *   cos_sin[k][i] = magnitude cos((first + k) w'_i),  cos_sin[k][dim / 2 + i] = magnitude sin(...)
 *
 *   cos_sin  [n][dim] fp32 out. With dim = 64 it is what smla_rope takes.
 *   dim      a multiple of 8, 8 .. 256.
 * Angles are exact fractions of a turn (64-bit fixed point; the w' are computed in 64-bit
 * floating point), so far positions lose nothing: within 2^-22 of the formula below
 * 2^27 positions. base > 1, factor >= 1, beta_fast >= beta_slow > 0, magnitude finite,
 * first + n at most 2^31. No workspace, no device errors.
 * ------------------------------------------------------------------------- */
int smla_rope_table(float* cos_sin, int64_t first, int32_t n, int32_t dim, double base, double factor,
                    int32_t original, double beta_fast, double beta_slow, float magnitude, void* stream);

/* ---------------------------------------------------------------------------
 * smla_rope_apply — turns `dim` values of each head (a whole head, or the part of it that
 * x points at).
 *
 *   cos_sin   [max_pos][dim] fp32 as smla_rope_table makes it. Pair i is values 2i
 *             and 2i + 1 (interleaved != 0) or i and i + dim / 2:
 *             (a, b) -> (a cos - b sin, a sin + b cos), in fp32, rounded once.
 *   positions [rows] int32; -1: the row is skipped (padding).
 *   x         head h of row i at x + i * x_row + h * x_head bf16 values.
 *   out       the same with out_row and out_head. out may be x with the same strides (in
 *             place); otherwise the two do not overlap. No two heads of out share a value
 *             (SMLA_ERR_INVALID_ARG).
 * dim: a multiple of 8, 8 .. 256. Strides: multiples of 8 values, head strides at
 * least dim (where there are several heads), row strides not negative. Device errors:
 * another position outside [0, max_pos): the row is skipped. Workspace: 256 bytes.
 * ------------------------------------------------------------------------- */
int smla_rope_apply(const float* cos_sin, int32_t max_pos, int32_t dim, int32_t interleaved, int32_t rows,
                    const int32_t* positions, const void* x, int64_t x_row, int64_t x_head, int32_t n_heads,
                    void* out, int64_t out_row, int64_t out_head, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * smla_cache_read — rows of the paged cache as bf16 values, packed: row cu_rows[b] + j of
 * the outputs is token starts[b] + j of request b.
 *
 *   page_tables [n_seqs][max_pages] int32.
 *   cu_rows     [n_seqs + 1] int32 (device), not decreasing: first output row of each
 *               request, and the number of rows.
 *   rows        rows of the outputs (host bound on cu_rows[n_seqs]). Rows before cu_rows[0]
 *               and from cu_rows[n_seqs] on are left as they are.
 *   starts      [n_seqs] int32 (device) or NULL: 0.
 *   latent      [rows] rows of 512 bf16 values, latent_stride values apart, or NULL:
 *               values 0..511 of the cache's latent rows: e4m3 codes times their scale in
 *               fp32, rounded once.
 *   pe          [rows] rows of 64, pe_stride apart, or NULL: the rope values.
 *   keys        [rows] rows of d_idx, keys_stride apart, or NULL: the indexer keys, times
 *               their scale where the cache has one.
 * Strides: multiples of 8, at least the row's width. Device errors: a token outside the
 * request's table or whose page is not in the pool: zeros; rows of an interval that runs
 * backwards: left as they are, as are rows past `rows`. Workspace: 256 bytes. The cache
 * is device memory; a part of it that no output needs may be NULL. One output at least, rows, n_seqs and
 * max_pages at least 1: a step that has no rows makes no call.
 * ------------------------------------------------------------------------- */
int smla_cache_read(const smla_paged_cache* cache, const int32_t* page_tables, int32_t max_pages, int32_t n_seqs,
                    const int32_t* cu_rows, int32_t rows, const int32_t* starts, void* latent, int64_t latent_stride,
                    void* pe, int64_t pe_stride, void* keys, int64_t keys_stride, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Heads of packed tokens: head h of token i at data + i * row_stride + h * head_stride
 * bf16 values. data on a 16-byte boundary, strides multiples of 8 values and below 2^35,
 * row_stride at least a head's width, head_stride as well (where there are several heads). */
typedef struct smla_heads {
  const void* data;
  int64_t row_stride, head_stride;
} smla_heads;

/* ---------------------------------------------------------------------------
 * smla_prompt_fwd — attention over packed prompts: request b has the query tokens
 * cu_q[b] .. cu_q[b + 1] - 1 and the keys cu_k[b] .. cu_k[b + 1] - 1, and
 *   o = softmax(sm_scale q K^T) V,  lse = ln sum exp(sm_scale q k)
 * over the keys that a token sees: all of its request's (causal = 0), or, of nq tokens and nk
 * keys, token i sees keys 0 .. nk - nq + i (causal != 0: the tokens are the last ones of
 * the context). Query head h uses key head h / (n_heads / n_kv_heads).
 *
 *   q      [total_q][n_heads][d_qk].  v [total_k][n_kv_heads][128].
 *   k      [total_k][n_kv_heads][d_qk], or, with k_pe, [..][d_qk - 64]: the last 64 values of every
 *   k_pe   head's key are those of [total_k] rows of 64 bf16 values, k_pe_stride apart
 *          (the rope part, which all heads share), or NULL.
 *   cu_q, cu_k  [n_seqs + 1] int32 (device), not decreasing, within [0, total]. Query rows
 *          outside every request's (padding) are left as they are. A request whose bounds
 *          run backwards or leave [0, total] counts as empty and is reported
 *          (SMLA_ERR_DEVICE_BOUNDS).
 *   prev_out, prev_lse  [total_q][n_heads][128] and [total_q][n_heads] fp32, or both NULL: the
 *          result of the same queries over other keys. The two are joined:
 *          L = ln(e^prev_lse + e^lse), out = e^(prev_lse - L) prev_out + e^(lse - L) o, lse = L.
 *          A prev_lse of -inf adds nothing, whatever prev_out holds. prev_out may be out
 *          (where that is fp32) and prev_lse may be lse.
 *   out    [total_q][n_heads][128] bf16, or fp32 (out_fp32 != 0: to be joined by a later call
 *          without rounding in between).
 *   lse    [total_q][n_heads] fp32 natural log, or NULL. A row that sees no key, or none whose logit is above
 *          -inf, has o = 0 and lse = -inf.
 * Operands are bf16, sums, maxima and partial results fp32; probabilities are rounded
 * to bf16 for their product with V, the sum of them is not. Keys and values that a row does
 * not see never reach it, whatever they hold; a value that is not finite reaches the rows that
 * see it, however small its probability: NaN as NaN, an infinity as itself or, where its probability or a joined
 * part's weight is zero in fp32, as either (how a request's keys are cut decides).
 * total_q, total_k and n_seqs are at least 1 (requests of no tokens or keys are fine; where no request has
 * any, there is no call to make: prev_out and prev_lse are the result).
 * Supported: d_qk 128 and 192; 1 <= n_heads <= 1024, a multiple of n_kv_heads. sm_scale is finite.
 * Workspace: the returned size (status word, the plan of the work, and partial results of
 * rows whose keys are cut: two pieces of 133 KB for each SM). The size is that of the current device.
 * ------------------------------------------------------------------------- */
size_t smla_prompt_fwd_workspace_size(int32_t total_q, int32_t total_k, int32_t n_seqs, int32_t n_heads,
                                      int32_t n_kv_heads);
int smla_prompt_fwd(const smla_heads* q, const smla_heads* k, const smla_heads* v, const void* k_pe,
                    int64_t k_pe_stride, int32_t total_q, int32_t total_k, int32_t n_seqs, const int32_t* cu_q,
                    const int32_t* cu_k, int32_t n_heads, int32_t n_kv_heads, int32_t d_qk, int32_t causal,
                    float sm_scale, const float* prev_out, const float* prev_lse, void* out, int32_t out_fp32,
                    float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SMLA_PROMPT_H_ */
