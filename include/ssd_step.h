/*
 * ssd_step.h -- C ABI of the operators around the Mamba2 SSD scan in a model
 * step, on MI355X (gfx950): the mixer's projections, its gated norm, the
 * log probabilities of tokens, and the pages and slots of the exact-replay
 * cache. The scan itself, its cache and the conv are in ssd_replay.h, whose
 * conventions hold here too: device pointers, contiguous row-major arrays,
 * asynchronous on `stream`, no allocation, every argument check on the host
 * before any launch, ssd_status codes, no exception across the ABI.
 *
 * One property is shared by all of them. A row's result depends on that
 * row's inputs alone: not on how many rows the call has, where the row
 * stands, or which kernel the size selects. So a step over one token gives
 * the bits that the same token gets in a prompt, as the scan and its replay
 * decode do (vLLM RFC "Mamba2: exact-replay decode so that prefill, chunked
 * prefill and decode produce identical bits").
 */
#ifndef SSD_STEP_H
#define SSD_STEP_H

#include "ssd_replay.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SSD_ACT_NONE = 0,
    SSD_ACT_SILU = 1,  /* v / (1 + exp(-v)) */
    SSD_ACT_GELU = 2,  /* tanh form: v / (1 + exp(-2 sqrt(2/pi) (v + 0.044715 v^3))) */
    SSD_ACT_RELU2 = 3  /* max(v, 0)^2 */
} ssd_activation;

/* Matrix product with bias, activation and residual in its epilogue:
 *   out[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + residual[m][n]
 *   x         [M,K] io_dtype
 *   w         [N,K] io_dtype
 *   bias      [N] fp32, or NULL
 *   residual  [M,N] io_dtype, or NULL
 *   out       [M,N] out_dtype (SSD_F32 or SSD_BF16); may be `residual`
 *             itself when the dtypes agree, and aliases nothing else
 * The sum is an fp32 chain over k in a fixed order (matrix-core steps of 32
 * k in bf16, of 4 in fp32, where every 512 k are a chain of their own and the
 * chains are added in order; a bf16 product is exact in fp32), the epilogue
 * is fp32, and the result is rounded once. The bits of a row do not depend on M.
 * M >= 0, N >= 0, K >= 1. K a multiple of 8 (bf16) or 4 (fp32) and at most
 * 1048576, and at most 4194304 tiles of 128 x 128 outputs, else
 * SSD_ERR_UNSUPPORTED. x and w 16-byte aligned (the others need their natural
 * alignment). One launch, or two over the columns. */
int ssd_linear(int64_t M, int64_t N, int64_t K, int32_t io_dtype,
               int32_t out_dtype, int32_t activation, const void *x,
               const void *w, const float *bias, const void *residual,
               void *out, hipStream_t stream);

/* The mixer's in-projection: ssd_linear of u [M, d_model] with
 * w [2*H*P + 2*G*N + H, d_model], its columns written to the three arrays
 * that the gate, the conv and the scan take:
 *   z    [M,H,P]       io_dtype   columns [0, H*P)
 *   xBC  [M,conv_dim]  io_dtype   the next H*P + 2*G*N
 *   dt   [M,H]         dt_dtype   the last H (raw dt)
 * bias [2*H*P + 2*G*N + H] fp32 or NULL. Same arithmetic and limits as
 * ssd_linear. shape->chunk_size is not used (any valid value). */
int ssd_in_proj(const ssd_shape *shape, int64_t M, int64_t d_model,
                const void *u, const void *w, const float *bias, void *z,
                void *xBC, void *dt, hipStream_t stream);

/* Gated RMS norm of the scan's output, before the out-projection. With
 * groups of gs = H*P / groups channels and g(v) = v / (1 + exp(-v)):
 *   norm_before_gate = 0:  v = y g(z);  out = v r w,  r = 1 / sqrt(mean_gs(v^2) + eps)
 *   norm_before_gate = 1:  out = (y r w) g(z),        r = 1 / sqrt(mean_gs(y^2) + eps)
 *   y, z  [T,H,P] io_dtype; z NULL: no gate
 *   w     [H*P] fp32
 *   out   [T,H,P] io_dtype; may be y or z itself
 * fp32 inside, rounded once. groups divides H; gs at most 32768 and T*H*P at
 * most 2^34, else SSD_ERR_UNSUPPORTED; eps >= 0 and finite, else
 * SSD_ERR_SHAPE. All arrays 16-byte aligned. */
int ssd_gated_norm(const ssd_shape *shape, int64_t T, int32_t groups, float eps,
                   int32_t norm_before_gate, const void *y, const void *z,
                   const float *w, void *out, hipStream_t stream);

/* Log probabilities of one given token per row, with the distribution's
 * entropy, the token's rank and the best alternatives. p = softmax(logits[t]):
 *   logits        [T,V] SSD_F32 or SSD_BF16 (natural alignment is enough)
 *   tokens        [T] int32
 *   logprob       [T] fp32    log p[token]; NaN for a token outside [0, V)
 *   entropy       [T] fp32    -sum p log p (nats), 0 log 0 = 0; or NULL
 *   rank          [T] int32   tokens ahead of this one, by logit descending
 *                             and index ascending (0 = greedy choice); -1 for
 *                             a token outside [0, V); or NULL
 *   top_ids       [T,top_k] int32, top_logprobs [T,top_k] fp32: the first
 *                             top_k tokens in that order (ties to the lower
 *                             index); both NULL when top_k is 0
 * Logits of -inf are masked tokens (p = 0). A row with nothing left (all
 * -inf) has logprob and top_logprobs -inf, entropy 0, and ranks by index. A
 * row that holds a NaN or +inf has no distribution: logprob, entropy and
 * top_logprobs are NaN, rank and top_ids -1.
 * 0 <= T <= 16777208, 1 <= V < 2^31 - 65536, 0 <= top_k <= min(64, V). One
 * launch, no workspace; sums in fp32 over a fixed split of the row. */
int ssd_token_logprobs(int64_t T, int64_t V, int32_t dtype, const void *logits,
                       const int32_t *tokens, int32_t top_k, float *logprob,
                       float *entropy, int32_t *rank, int32_t *top_ids,
                       float *top_logprobs, hipStream_t stream);

/* ---- pages and slots of an exact-replay cache ----
 *
 * The page table (cache->buf_pages, which the calls that say so write
 * despite its const) is the only record of who holds which page: a page is
 * free when no table entry names it, entries outside [0, num_pages) are "no
 * page". Nothing else is kept between calls, so a table that the caller
 * edits stays right. Slot lists must be distinct unless stated, list entries
 * outside [0, num_slots) are skipped. cache->work is not used (may be NULL).
 * num_pages at most 1048576, num_slots * Q / page_tokens below 2^31 and lists
 * of copy and free up to 16777208 entries (SSD_ERR_UNSUPPORTED). One table may
 * serve the caches of several layers (reserve and trim through any one of
 * them, copy and free each), but not a pool that is compacted, since that
 * moves one cache's pages. A contiguous cache (buf_pages NULL) is
 * SSD_ERR_NULL for the page calls and fine for copy and free.
 * Calls on one cache must be ordered (one stream, or events). */

/* Hands out pages so that each listed slot can take tokens: slot =
 * slot_idx[b] (NULL = b) gets a page for every position below
 * min(buf_len[like] + tokens[b], Q) that has none, where like = like_idx[b]
 * (NULL = the slot itself; otherwise the slot that will be copied into it,
 * and may repeat). tokens NULL: tokens_all for every slot; a negative count
 * is taken as 0. With tokens = 1 the next decode step, with tokens = n any
 * prefill, verification or acceptance of up to n tokens finds its pages.
 * Requests are served in list order, lowest free page first: with need[b]
 * the pages that b lacks, b is served when need[0] + .. + need[b] (the
 * skipped and the unserved counted too) is at most the number of free
 * pages, and gets all of them; otherwise its table row stays as it is.
 * granted[n] int32 (or NULL): 1 when the slot has all its pages now (also
 * when it lacked none), 0 when it was not served or the entry (slot or
 * like) is skipped or its buf_len is outside [0, Q). Writes the table. */
int ssd_replay_pages_reserve(const ssd_shape *shape, const ssd_replay_cache *cache,
                             int32_t n, const int32_t *slot_idx,
                             const int32_t *like_idx, const int32_t *tokens,
                             int32_t tokens_all, int32_t *granted, hipStream_t stream);

/* Returns the pages past each listed slot's buffered tokens (entries
 * ceil(buf_len / page_tokens) and up become -1): after a chunk completed or
 * drafts were refused. Writes the table. */
int ssd_replay_pages_trim(const ssd_shape *shape, const ssd_replay_cache *cache,
                          int32_t n, const int32_t *slot_idx, hipStream_t stream);

/* Ends the listed slots: state, its bf16 copy, buf_len and boundary_pos
 * become zero (a fresh slot) and, in a paged cache, the slot's pages are
 * returned. Buffered rows are left as they are. Writes the table. */
int ssd_replay_cache_free(const ssd_shape *shape, const ssd_replay_cache *cache,
                          int32_t n, const int32_t *slot_idx, hipStream_t stream);

/* Copies slots: dst->slot[dst_idx[b]] becomes what src->slot[src_idx[b]] is
 * (state, bf16 copy, the buf_len buffered rows, buf_len, boundary_pos), so
 * it decodes on with the same bits. The caches may be the same one (a fork)
 * or two of the same shape and chunk size that differ in slots, pages,
 * page size or layout (moving to a larger or smaller pool). Sources may
 * repeat; destinations are distinct and, within one cache, no destination
 * is another entry's source. Buffered C is copied when both caches keep it;
 * dst keeping C that src lacks is SSD_ERR_NULL. An entry is skipped (its
 * destination left as it is) when a slot is out of range, the source's
 * buf_len is outside [0, Q), a page that its buffered positions need is
 * missing on either side, or source and destination are the same slot.
 * copied[n] int32 (or NULL): 1 for an entry that was copied (or is the
 * same slot), 0 for one that was skipped. The tables are only read. */
int ssd_replay_cache_copy(const ssd_shape *shape, const ssd_replay_cache *dst,
                          const ssd_replay_cache *src, int32_t n,
                          const int32_t *dst_idx, const int32_t *src_idx,
                          int32_t *copied, hipStream_t stream);

/* Compacts the pool: with U pages in use, the used pages numbered U and up
 * move, in order, to the free pages below U, in order, and the table
 * follows, so that pages 0..U-1 hold everything. used[1] int32 receives U.
 * workspace: ssd_replay_pages_compact_workspace_bytes(cache) bytes, 4-byte
 * aligned, contents irrelevant before and after. Writes the table and pages. */
size_t ssd_replay_pages_compact_workspace_bytes(const ssd_replay_cache *cache);
int ssd_replay_pages_compact(const ssd_shape *shape, const ssd_replay_cache *cache,
                             int32_t *used, void *workspace, size_t workspace_bytes,
                             hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_STEP_H */
