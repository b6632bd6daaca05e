/*
 * specverify_cache.h - operators of libspecverify on the paged key/value cache
 * of a round (include/specverify.h): what happens to the cache between one
 * verify step and the next.
 *
 *   sv_plan_round    after a round: lengths move by the tokens that it kept
 *                    (num_accepted + 1, or sv_truncate_emitted's count), pages
 *                    that hold only rejected drafts go back to the free list,
 *                    the next round's pages come from it, and every row of the
 *                    next round gets its slot and its position
 *   sv_append_kv4    the round's keys and values, quantised to 4 bits, into
 *                    their slots
 *   sv_read_kv4      the values that slots hold
 *   sv_attend_kv4    the attention of the round's gamma+1 rows over the pages
 *                    ("11.1 核心原理: Draft + Verify 与 Rejection Sampling",
 *                    section 11.1.1: one forward pass of the target gives the
 *                    gamma+1 distributions that the verify step takes)
 *
 * Memory, execution and error conventions are those of specverify.h: device
 * memory owned by the caller, asynchronous on `stream` of the current device,
 * arguments validated on the host before any launch, data problems never
 * fault.  B = 0 is a valid empty call.
 *
 * The cache.  cache [pages][heads][page * (D + 8)] bytes, 16-byte aligned; a
 * page holds `page` tokens (a multiple of 16, at most 256), D is 64 or 128.
 * Slot s is token s % page of page s / page.  A head's block of a page holds,
 * one after another,
 *   the codes of its keys     token t: D/2 bytes at t * D/2; channel 2j is the
 *                             low half of byte j, channel 2j+1 the high half
 *   the codes of its values   tokens 2u and 2u+1 interleaved by units of four
 *                             channels: unit j of token t is the two bytes at
 *                             (t / 2) * D + 4 j + 2 (t % 2), its channels in
 *                             the order of a key's
 *   four numbers per token    of the model's type (bf16 or fp16): scale and
 *                             offset of the key, scale and offset of the value
 * A held element is scale * code + offset.  A row x of D elements is held with
 *   offset = min x
 *   scale  = (max x - min x) / 15, in float32, rounded to the model's type
 *   code   = (x - offset) * (1 / scale) in float32, rounded to the nearest
 *            whole number (ties to even), at most 15; 0 where scale is below
 *            2^-126
 * A row with a NaN or an infinity, or whose scale is not finite, is held as
 * NaN: scale and offset NaN, codes 0.
 * The bytes do not say which type they are of: a cache is read and attended with
 * the type that was appended.
 */
#ifndef SPECVERIFY_CACHE_H
#define SPECVERIFY_CACHE_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits checked by the entry points. */
#define SV_MAX_PLAN_SEQUENCES 8192 /* sequences of one sv_plan_round */
#define SV_MAX_CACHE_PAGE 256      /* tokens of a page */
#define SV_MAX_CACHE_SLOTS (1 << 30) /* pages * page, and block table entries of a call */
#define SV_MAX_CACHE_ROWS (1 << 24) /* rows B * (gamma+1) of one call */
#define SV_MAX_CACHE_HEADS 1024    /* key/value heads */
#define SV_MAX_CACHE_GROUP 64      /* query heads that share a key/value head */

/* Per-sequence status of sv_plan_round. */
#define SV_PLAN_NO_PAGES 1  /* the free list has too few pages for it */
#define SV_PLAN_TOO_LONG 2  /* it needs more pages than its table row has entries */

/*
 * The bookkeeping between two rounds, in place on the state.
 *
 *   lengths      [B] int32, in and out: tokens whose keys and values are valid.
 *                lengths[b] += kept[b] (at least 0, at most 2^31 - 1, as
 *                positions are)
 *   kept         [B] int32 or NULL (none): tokens of the last round that stay,
 *                negative: tokens taken back
 *   gamma_b      [B] int32 or NULL (gamma): drafts of the next round, clamped to
 *                [-1, gamma]; it has n_b = gamma_b[b] + 1 rows
 *   block_table  [B][N] int32, in and out: the pages of a sequence in order,
 *                behind them -1
 *   blocks       [B] int32, in and out: how many it has.  It needs
 *                ceil((lengths[b] + n_b) / page)
 *   free_blocks  [pool] int32, in and out: the free pages are the first
 *                free_count[0] entries, the last of them is taken first
 *   free_count   [1] int32, in and out
 *   slots        [B][gamma+1] int32, out: block_table[b][p / page] * page +
 *                p % page for row i at position p = lengths[b] + i; -1 behind
 *                row n_b - 1, and for all rows of a sequence with a status
 *   positions    [B][gamma+1] int32, out: lengths[b] + i; 0 behind row n_b - 1
 *   status       [B] int32, out: SV_PLAN_ bits; such a sequence neither gives
 *                nor takes pages
 *
 * All sequences give before any takes.  Taking goes in the order of the
 * sequences and of their pages; the first one that the free list cannot serve
 * in full, and all that want pages behind it, get none.  Giving goes in the
 * reverse order, so that a round that is taken back leaves the free list as it
 * was.  A count outside its array is clamped to it; a page id outside
 * [0, 2^30 / page) gives slot -1.  Giving never writes behind `pool`.
 *
 * A sequence with a status has moved to lengths[b] all the same, but nothing of
 * this round is stored for it, and what its last page holds behind lengths[b] are
 * rejected drafts: give sv_attend_kv4 gamma_b = -1 for it, and the next
 * sv_plan_round kept = 0 (as for every sequence without rows in a round).
 *
 * SV_ERR_INVALID_ARG for bad sizes (B * N and pool * page above
 * SV_MAX_CACHE_SLOTS among them) and NULL arrays.
 */
sv_status sv_plan_round(int B, int gamma, int page, int N, int pool, int32_t* lengths, const int32_t* kept,
                        const int32_t* gamma_b, int32_t* block_table, int32_t* blocks, int32_t* free_blocks,
                        int32_t* free_count, int32_t* slots, int32_t* positions, int32_t* status, sv_stream_t stream);

/*
 * Keys and values of R = B * (gamma+1) rows into their slots.
 *
 *   k, v       element (b, i, h, d) at b * strides[0] + i * strides[1] +
 *              h * strides[2] + d; strides (in elements, on the host) are
 *              multiples of 8 and not negative, k and v 16-byte aligned
 *   dtype      SV_DTYPE_BF16 or SV_DTYPE_F16
 *   slots      [B][gamma+1] int32: a row whose slot is outside
 *              [0, pages * page) is not written.  No slot is given twice
 *   cache      overlaps neither k nor v (SV_ERR_INVALID_ARG)
 */
sv_status sv_append_kv4(int B, int gamma, int heads, int D, int page, int pages, const void* k,
                        const int64_t* k_strides, const void* v, const int64_t* v_strides, sv_dtype dtype,
                        const int32_t* slots, void* cache, sv_stream_t stream);

/*
 * What R slots hold: k, v [R][heads][D] of the model's type, contiguous and
 * 16-byte aligned, apart from each other and from cache: scale * code + offset
 * rounded to it; 0 where the slot is outside [0, pages * page).
 */
sv_status sv_read_kv4(int R, int heads, int D, int page, int pages, const void* cache, sv_dtype dtype,
                      const int32_t* slots, void* k, void* v, sv_stream_t stream);

/*
 * Attention of a round's rows over the cache.  Row i of sequence b sees the
 * positions 0 .. lengths[b] + i (the round's own tokens are appended before):
 *   z_t = scale * (q . k_t),  out = sum_t softmax(z)_t v_t,
 *   lse = log sum_t exp(z_t)
 *
 *   G            query heads per key/value head; query head h * G + g reads
 *                key/value head h
 *   gamma        at most SV_MAX_GAMMA
 *   q            [B][gamma+1][heads * G][D] through q_strides (batch, row,
 *                head), as k's in sv_append_kv4.  A row with an element that
 *                is beyond 2^100 or is so times scale, an infinity or a NaN may
 *                give NaN; the rows beside it are not touched by it
 *   block_table  [B][N] int32: an entry outside [0, pages) hides its tokens,
 *                as does a position at N * page and behind.  N * page bounds
 *                the sequences' lengths: few sequences take one launch instead
 *                of two, and about half of the time, where it is at most 16640,
 *                so a table of no more columns than its longest sequence has
 *                pages serves short sequences best
 *   lengths      [B] int32: tokens cached before the round (negative: 0)
 *   gamma_b      [B] int32 or NULL (gamma): rows i <= gamma_b[b] take part;
 *                -1: none
 *   scale        positive and finite
 *   out          [B][gamma+1][heads * G][D] of q's type, contiguous, 16-byte
 *                aligned, overlapping neither q nor cache.  A row that sees no
 *                token is 0
 *   lse          [B][gamma+1][heads * G] float32 or NULL; -inf where a row
 *                sees no token
 *   fill         nonzero: rows behind gamma_b become 0 in out and lse; 0: they
 *                stay as they are
 *   workspace    of sv_attend_kv4_workspace_bytes(gamma, heads, G, D) bytes
 *                (0 for sizes that are not supported) on the current device,
 *                16-byte aligned, any contents; one per concurrent call
 *
 * Sums and softmax statistics are float32, of weights up to 2^8: held values
 * beyond 2^100 may give infinities or NaN.  A token's weight times its value's
 * scale is rounded to float16 (bf16 results, where the rounding counts for what
 * an element is away from the middle of its row alone) or to two float16 parts
 * (fp16 results), relative to the largest scale of a value that the sequence
 * has in that head: beside the relative error, 2^-30 of the largest value for
 * each token.  Results do not depend on the order in which CTAs run.
 */
size_t sv_attend_kv4_workspace_bytes(int gamma, int heads, int G, int D);

sv_status sv_attend_kv4(int B, int gamma, int heads, int G, int D, int page, int pages, int N, const void* q,
                        const int64_t* q_strides, sv_dtype dtype, const void* cache, const int32_t* block_table,
                        const int32_t* lengths, const int32_t* gamma_b, float scale, void* out, float* lse, int fill,
                        void* workspace, size_t workspace_bytes, sv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_CACHE_H */
