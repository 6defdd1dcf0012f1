/*
 * q4_serve.h -- C ABI of libq4, the turn of a serving loop around a model's layers, for AMD
 * Instinct MI355X (gfx950): the plan of a batch on the paged cache of q4_attn.h (offsets,
 * positions, slots and pages of the new tokens, from the requests' lengths) and the choice
 * of the next tokens from the logits. All of it runs on the device, so that a decode step
 * can be captured and replayed without the host. Same library, status codes and conventions
 * as q4.h (device pointers owned by the caller, enqueue-only on `stream`, host-side
 * validation before any HIP call, q4_last_error() for details).
 */
#ifndef Q4_SERVE_H
#define Q4_SERVE_H

#include "q4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- the plan of a batch ---------------------------------------------------------
 * Sequence s holds kv_lens[s] tokens, its block table's first ceil(kv_lens[s] / page_size)
 * entries their pages, and gets new_lens[s] more (NULL: one each). In this order:
 *   1. where reset[s] != 0 (NULL: nowhere), the sequence's pages are pushed on the stack of
 *      free pages, in the order of sequences and blocks, and its length becomes 0: a request
 *      that has ended, its place empty (no new tokens) or taken by the next one;
 *   2. the new tokens are the call's rows, one sequence's behind the other's: rows
 *      q_offsets[s] .. q_offsets[s + 1] - 1; row i of them is token t = kv_lens[s] + i;
 *   3. each page that the new tokens need beyond those held is popped from the stack's top,
 *      in the order of sequences and blocks, into the block table;
 *   4. of each row: positions = starts[s] + t (starts NULL: t; a shared prefix's length, for
 *      q4_paged_attention_shared), slots = page * page_size + t % page_size;
 *   5. kv_lens_out[s] = kv_lens[s] + new_lens[s].
 * These are the arguments of q4_qk_norm_rope_append and q4_paged_attention.
 *   free_pages: int32 [pages], the stack, free_count[0] pages deep (its top is entry
 *   free_count[0] - 1); free_count_out[0] its depth afterwards. free_pages NULL: a block
 *   table that holds all pages already; nothing is pushed or popped, free_count and
 *   free_count_out are unused.
 *   block_table: int32 [seqs][max_blocks]; entries of tokens that are not stored keep what
 *   they held. tokens: rows that positions and slots (int32 [tokens]) hold; those behind the
 *   last sequence's get slot -1 (which the append skips) and position 0.
 *   kv_lens, new_lens, reset, starts: int32 [seqs]; q_offsets: int32 [seqs + 1].
 * lacking[0] (int32) counts the pages that were needed and not there: the stack was empty or
 * the block table too short. Their tokens have slot -1 and do not count in kv_lens_out (the
 * rows stay; such a sequence's attention is not to be used). New tokens beyond `tokens` rows
 * are dropped, sequence by sequence from the last. Lengths outside [0, max_blocks *
 * page_size] are cut to it, negative new_lens to 0; a page number outside [0, pages) gives
 * slot -1: no contents of these arrays lead outside the buffers.
 * kv_lens_out may be kv_lens, free_count_out may be free_count (a captured loop keeps its
 * state so); no other buffers may overlap. With other output buffers and nothing reset, a
 * call changes none of its own inputs and may be repeated. max_blocks * page_size <= 2^30, pages *
 * page_size < 2^31; seqs <= 65536. `workspace` (8-byte aligned) must hold
 * q4_paged_plan_workspace_bytes() bytes (NULL when that is 0). */
size_t q4_paged_plan_workspace_bytes(int64_t seqs, int64_t tokens);
q4_status q4_paged_plan(const int32_t* kv_lens, const int32_t* new_lens, const int32_t* reset, const int32_t* starts,
                        int64_t seqs, int64_t tokens, int32_t page_size, int64_t pages, int32_t* block_table,
                        int64_t max_blocks, int32_t* free_pages, const int32_t* free_count, int32_t* q_offsets,
                        int32_t* positions, int32_t* slots, int32_t* kv_lens_out, int32_t* free_count_out,
                        int32_t* lacking, void* workspace, size_t workspace_bytes, void* stream);

/* ---- the next tokens -------------------------------------------------------------
 * One token of each row of logits [rows][vocab], rows `stride` >= 0 elements apart (0: all
 * draws from the same logits), for a given uniform random number u in [0, 1) a row. With m the row's largest logit:
 *   w_i = exp((l_i - m) / temperature), tokens ranked by logit, equal ones by index;
 *   top_k: the first k stay (k <= 0 or >= vocab: all);
 *   top_p: of those the shortest run of first ones whose w sum to top_p times theirs or
 *     more stays (>= 1 or NaN: all; <= 0: the first);
 *   min_p: of those w_i >= min_p stays (<= 0 or NaN: all; > 1: as 1);
 *   the token is the first, by index, up to which the w that stayed sum to more than u
 *   times their total.
 * temperature <= 0 or NaN: the first by rank (no draw). A temperature of +infinity weighs
 * all alike. u below 0 or NaN is taken as 0, 1 or more as the last token that stayed.
 * A NaN logit counts as -infinity; tokens at -infinity are never chosen; with +infinity
 * among the logits only those have weight. A row with nothing above -infinity: token -1,
 * prob 0.
 *   temperature, top_p, min_p: float32 [rows], top_k: int32 [rows], each NULL: 1, 1, 0, all.
 *   tokens: int32 [rows]; probs: float32 [rows] or NULL, the chosen token's w over the total
 *   of those that stayed.
 * Differences are taken in float64 and weights kept in fixed point, 2^-s of the largest a
 * step, s = min(50, 62 - ceil(log2(vocab))) (45 for 131072 tokens), so that sums are exact
 * in any order. A weight is off by half a step at most, so the choice is that of exact
 * arithmetic but where u * total or a cut comes within vocab * 2^-(s + 1) of the largest weight
 * (2e-12 for 4096 tokens, 2e-9 for 131072, 1.2e-7, two steps of a float32 u, for 2^20) and
 * 2^-47 of the sum of a border; a token whose weight rounds to 0 is never drawn.
 * Deterministic. vocab <= 2^20, rows < 2^22, rows *
 * ceil(vocab / 4096) < 2^24 (Q4_ERR_SHAPE). `workspace` (16-byte aligned) must hold
 * q4_sample_workspace_bytes() bytes (NULL when that is 0), which serve fewer rows too: where rows are split (above
 * 32768 logits, or above 16384 for up to 32 rows) 8 bytes a logit for the tokens that a cut may list, with or without
 * cuts, and some more (67 MB for 64 rows of 128256), else none. */
typedef enum { Q4_F16 = 0, Q4_BF16 = 1, Q4_F32 = 2 } q4_dtype;

size_t q4_sample_workspace_bytes(int64_t rows, int64_t vocab);
q4_status q4_sample(const void* logits, int32_t dtype, int64_t stride, int64_t rows, int64_t vocab,
                    const float* uniforms, const float* temperature, const int32_t* top_k, const float* top_p,
                    const float* min_p, int32_t* tokens, float* probs, void* workspace, size_t workspace_bytes,
                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4_SERVE_H */
