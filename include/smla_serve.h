/*
 * smla_serve — what a serving step needs around the paged latent cache of
 * smla.h: block tables and slot maps from request lengths, the rows of new
 * tokens normed, rotated, quantised and written into the cache, the queries
 * prepared for the indexer and the attention, and attention of a batch over a
 * prompt that all of its requests share.
 *
 * The conventions of smla.h hold: device pointers, caller-owned buffers, work
 * enqueued on `stream`, no allocation and no synchronisation, argument checks
 * on the host before anything is enqueued, device-side errors as bits of the
 * status word at the head of the workspace (smla_read_status). Arrays of int32
 * and float need their natural alignment only; rows of bf16 or e4m3 values, norm
 * weights and cos_sin start on 16-byte boundaries.
 */
#ifndef SMLA_SERVE_H_
#define SMLA_SERVE_H_

#include "smla.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * smla_build_tables — pages and slots of the next new_lens[b] tokens of every
 * request, from lengths that live on the device. (free_pages begins with the page to
 * be handed out first: a caller that keeps one list for many calls moves it on by
 * pages_used.)
 *
 * Request b holds ctx_lens[b] tokens in ceil(ctx / 64) pages, listed first in
 * page_tables[b]. Its new tokens continue its last page and then take pages
 * from free_pages in order, requests in the order of b:
 *   need[b]  = ceil((ctx + new) / 64) - ceil(ctx / 64)
 *   page p of b (p >= ceil(ctx / 64)) = free_pages[sum_{a<b} need[a] + p - ceil(ctx / 64)]
 *   slot of the token at position t   = page(t / 64) * 64 + t % 64
 *
 *   ctx_lens    [n_seqs] int32, >= 0.     new_lens [n_seqs] int32, >= 0 (0: idle).
 *   page_tables [n_seqs][max_pages] int32, in and out: the entries of the new
 *               pages are written, all others are left as they are.
 *   free_pages  [n_free] int32: page ids to hand out (may be NULL if n_free = 0).
 *   max_new     rows of the per-token outputs (host bound on the sum of new_lens).
 *   seq_lens    [n_seqs] int32 out: tokens of b that have a page afterwards
 *               (ctx + new); what smla_sparse_mla_decode and
 *               smla_shared_prefix_fwd take. Not the same array as ctx_lens.
 *   cu_new      [n_seqs + 1] int32 out: first output row of each request, and
 *               the number of rows in use.
 *   positions   [max_new] int32 out or NULL: position of each new token.
 *   slots       [max_new] int32 out: pool row of each new token.
 *   row_seq     [max_new] int32 out or NULL: its request.
 *   pages_used  [1] int32 out: entries of free_pages that were taken.
 * Rows past cu_new[n_seqs] get -1 in all three (a batch padded to a captured
 * size: smla_cache_append skips slot -1, smla_query_prep position -1).
 * Device errors (SMLA_ERR_DEVICE_BOUNDS): negative lengths, or more than
 * max_pages * 64 tokens (or 2^31 - 64): the request counts as empty (seq_lens 0, no rows).
 * Rows past max_new: dropped, as if new_lens were smaller. Free list exhausted:
 * the tokens without a page get slot -1 and seq_lens stops before them. A page id
 * that no pool can have (negative, or 2^25 and more), of a continued page or taken
 * from free_pages: the page's tokens get slot -1; the id stays in the table and
 * seq_lens counts the tokens (the attention skips and reports the page again).
 * Workspace: 256 bytes.
 * ------------------------------------------------------------------------- */
int smla_build_tables(const int32_t* ctx_lens, const int32_t* new_lens, int32_t n_seqs, int32_t* page_tables,
                      int32_t max_pages, const int32_t* free_pages, int32_t n_free, int32_t max_new,
                      int32_t* seq_lens, int32_t* cu_new, int32_t* positions, int32_t* slots, int32_t* row_seq,
                      int32_t* pages_used, void* workspace, size_t workspace_bytes, void* stream);

/* Rotation of the rope values. cos_sin [max_pos][64] fp32: for each position the
 * cosines of its 32 angles, then their sines. Pair i of 64 values is turned by
 * angle i: (a, b) -> (a cos - b sin, a sin + b cos). interleaved != 0: pair i is
 * values 2i and 2i + 1; 0: values i and i + 32. */
typedef struct smla_rope {
  const float* cos_sin;
  int32_t max_pos;
  int32_t kv_interleaved;  /* the latent row's 64 rope values and the attention query's */
  int32_t idx_interleaved; /* the first 64 values of an indexer key or query */
} smla_rope;

/* ---------------------------------------------------------------------------
 * smla_cache_append — writes the rows of new tokens into the cache, in one pass
 * over them: norm, rotation, quantisation to the cache's formats, paged write.
 *
 *   slots     [rows] int32 pool rows (page * 64 + slot in page); -1: skipped.
 *             No two rows may have the same slot.
 *   positions [rows] int32 for the rotation (row of cos_sin).
 *   ckv       [rows] rows of 576 bf16 values, ckv_stride values apart (a
 *             multiple of 8), or NULL: leave cache->kv alone. Values 0..511:
 *               y = x * rsqrt(mean(x^2) + eps) * kv_norm   (kv_norm [512] fp32;
 *               NULL: y = x), values 512..575: the rotated rope values.
 *             Written as cache->kv_dtype says: bf16; e4m3 with one scale over
 *             the 576 values into kv_scale; or the 656-byte row with a scale per
 *             128 latent values and bf16 rope. scale = amax / 448 (at least 2^-126; 1 if
 *             all are zero), code = e4m3(y / scale), rounded to nearest even.
 *   k_raw     [rows] rows of d_idx bf16 values, k_stride apart (a multiple of
 *             8), or NULL: leave cache->k_idx alone.
 *               idx_norm and idx_bias ([d_idx] fp32): layer norm
 *                 y = (x - mean) * rsqrt(var + eps) * idx_norm + idx_bias;
 *               idx_norm alone: y = x * rsqrt(mean(x^2) + eps) * idx_norm;
 *               neither: y = x.
 *             The first 64 values are then rotated. bf16 keys are rounded; e4m3
 *             keys get such a scale in k_idx_scale, or, where that array
 *             is NULL, are rounded as they are (beyond +-448: saturated).
 * All arithmetic in fp32, rounded once. Device errors: a slot outside the pool
 * or a position outside [0, max_pos): the row is skipped. Workspace: 256 bytes.
 * Supported: d_idx 128 (e4m3) and 64 (bf16), as in smla.h.
 * ------------------------------------------------------------------------- */
int smla_cache_append(const smla_paged_cache* cache, const smla_rope* rope, int32_t rows, const int32_t* slots,
                      const int32_t* positions, const void* ckv, int64_t ckv_stride, const float* kv_norm,
                      const void* k_raw, int64_t k_stride, const float* idx_norm, const float* idx_bias, float eps,
                      void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * smla_query_prep — the queries of new tokens as the attention and the indexer
 * take them, every head in one pass.
 *
 *   positions [rows] int32 (row of cos_sin); -1: the row is skipped (padding).
 *   q_pe      the 64 rope values of each attention head, bf16: head h of row i
 *             at q_pe + i * pe_row_stride + h * pe_head_stride values (multiples
 *             of 8), or NULL: no attention queries. Rotated and written to
 *   q         [rows][n_heads][576] bf16, values 512..575 of each head (values
 *             0..511, the latent part, are left alone).
 *   q_raw     [rows][h_idx][d_idx] bf16 indexer queries, rows q_raw_stride
 *             values apart (a multiple of 8), or NULL: no indexer queries. Each
 *             head: y = x * rsqrt(mean(x^2) + eps) * idx_norm ([d_idx] fp32;
 *             NULL: y = x), first 64 values rotated, then
 *   q_idx     [rows][h_idx][d_idx]: bf16, or e4m3 with scale and codes of the head
 *             as smla_cache_append makes them; the scale goes into
 *   w_out     [rows][h_idx] fp32 = w * (scale * w_scale) (bf16: w * w_scale),
 *             so that w_out * ReLU(q_idx . k) is the score's term: a positive
 *             scale passes through the ReLU. w [rows][h_idx] fp32; w_out may be w.
 * Device errors: another position outside [0, max_pos): the row is skipped.
 * Workspace: 256 bytes. Supported: n_heads 16 and 64, h_idx 4, 8, 16, 32, 64,
 * d_idx 128 (e4m3) and 64 (bf16).
 * ------------------------------------------------------------------------- */
int smla_query_prep(const smla_rope* rope, int32_t rows, const int32_t* positions, const void* q_pe,
                    int64_t pe_row_stride, int64_t pe_head_stride, int32_t n_heads, void* q, const void* q_raw,
                    int64_t q_raw_stride, int32_t h_idx, int32_t d_idx, int32_t idx_dtype, const float* idx_norm,
                    float eps, const float* w, float w_scale, void* q_idx, float* w_out, void* workspace,
                    size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * smla_shared_prefix_fwd — attention of a batch over a prompt that all of its
 * requests share and over each request's own tokens, with no selection: every
 * new token sees every key up to its own position (MLA in MQA form: QK over 576
 * values, PV over the first 512, as smla_sparse_mla_fwd).
 *
 * Tokens 0 .. shared_len - 1 are the same for every request. They are read
 * through page_tables[0] only, once for all query rows of the batch together
 * (so row 0 lists the shared pages even where request 0 is idle; pages past every
 * request's length are not looked at);
 * tokens from shared_len on are read through each request's own table. The two
 * parts are joined by their log-sum-exp. shared_len need not end on a page: the
 * page that holds the border is read through row 0 before it and through
 * the request's own table after it. shared_len = 0: plain causal attention.
 *
 *   page_tables [n_seqs][max_pages] int32.
 *   seq_lens    [n_seqs] int32 (device): keys of each request including the
 *               shared ones and its q_per_seq new tokens. Query j of request b
 *               sits at position seq_lens[b] - q_per_seq + j and sees keys
 *               0..that position; a position < 0 sees nothing (an idle request:
 *               seq_lens[b] = 0). A length above max_seq_len is taken as
 *               max_seq_len and reported (SMLA_ERR_DEVICE_BOUNDS).
 *   max_seq_len host bound of seq_lens; shared_len <= max_seq_len.
 *   q           [n_seqs * q_per_seq][n_heads][576] bf16.
 *   out         [n_seqs * q_per_seq][n_heads][512] bf16.
 *   lse         [n_seqs * q_per_seq][n_heads] fp32 natural log, or NULL. A row
 *               that sees no key gets out = 0 and lse = -inf.
 * Keys of a page outside the pool are skipped and reported. The latent cache is
 * device memory. The MMAs accumulate in fp32. BF16 rows and per-token FP8 codes:
 * bf16 operands (q, rows and codes as they are, the probabilities rounded to bf16;
 * the scales multiply logits and probabilities in fp32). Tile-scaled FP8 rows: f16
 * operands (values and probabilities rounded to f16), so |q| and the values must
 * stay below 65504; beyond it, in a row that sees a key or a key that a row sees,
 * smla_read_status gives SMLA_ERR_UNSUPPORTED, as for smla_sparse_mla_fwd. Values
 * below f16's normals (2^-14) are off by up to 2^-25 (and below that zero).
 * Keys that a row does not see never reach it, whatever they hold (an unused
 * slot of a page may hold NaN).
 * Supported: n_heads 16 and 64; any q_per_seq >= 1; the three cache formats.
 * Workspace: the returned size (status word, the partial results of the pieces that
 * the keys are cut into, 265 KB each: two pieces for each pair of SMs where nothing is
 * shared, else one for each 128 rows of the batch, one for each 128 rows or part
 * of them of each request, and one for each pair; and, for FP8 caches whose shared part
 * is read by more than 128 query rows of several requests, a 16-bit copy of the shared
 * rows, 1,152 bytes a token and 16 a page). The size is that of the current device.
 * ------------------------------------------------------------------------- */
size_t smla_shared_prefix_fwd_workspace_size(int32_t n_seqs, int32_t max_seq_len, int32_t shared_len,
                                             int32_t q_per_seq, int32_t n_heads, int32_t kv_dtype);
int smla_shared_prefix_fwd(const smla_paged_cache* cache, const int32_t* page_tables, int32_t max_pages,
                           int32_t n_seqs, const int32_t* seq_lens, int32_t max_seq_len, int32_t shared_len,
                           int32_t q_per_seq, const void* q, int32_t n_heads, float sm_scale, void* out, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SMLA_SERVE_H_ */
