/*
 * q4_attn.h -- C ABI of libq4, the attention side of a decoder layer on a paged INT4
 * KV cache, for AMD Instinct MI355X (gfx950): norm and rotation of q and k, the
 * append of k and v into the pages, and the attention of new tokens over them. Same
 * library, status codes and conventions as q4.h (device pointers owned by the
 * caller, enqueue-only on `stream`, host-side validation before any HIP call,
 * q4_last_error() for details).
 *
 * Sources (cited by page title and section):
 *  [WIKI] "压缩算法" (cs-knowledge-wiki.pages.dev), section 7.4.1.2: INT4 KV cache,
 *         groups along head_dim, scale = group amax / 7, codes in [-8, 7].
 *  [YBB]  "LLM 后训练量化深度实战…" (www.ybb.press), section 七: scales must be at least
 *         per head and follow the tokens, and the pages, they belong to.
 *
 * Tokens. The rows of all sequences lie one behind the other: q [tokens][q_heads]
 * [head_dim], k and v [tokens][kv_heads][head_dim], float16. The heads of a token are
 * contiguous, the tokens `stride` elements apart, so q, k and v may be slices of one
 * fused projection's rows. Row pointers are 16-byte aligned and strides multiples of
 * 8. head_dim is 64, 128 or 256; q_heads is a multiple of kv_heads, and query head h
 * reads KV head h / (q_heads / kv_heads).
 *
 * The paged cache. A page holds page_size tokens (a multiple of 16) of every KV head;
 * token row i of page p is slot p * page_size + i. Per page and head, K and V lie as
 * tiles of 16 tokens in the operand order of v_mfma_f32_16x16x32_f16, so attention
 * loads them straight into registers. With T = page_size / 16, D = head_dim,
 * M = D / 32, I = min(M, 4), tile = (p * kv_heads + h) * T + i / 16 and t = i % 16:
 *   K code of channel 32m + 8c + e (c < 4, e < 8): nibble p(e) of dword
 *     tile * 2D + ((m / I) * 64 + t + 16c) * I + m % I,
 *     p(e) = e / 2 (e even), 4 + (e - 1) / 2 (e odd);
 *   V code of channel 32m + 16n + r (n < 2, r < 16): nibble n of byte b(t % 4) of dword
 *     tile * 2D + ((m / I) * 64 + r + 16 (t / 4)) * I + m % I,
 *     b = 0, 2, 1, 3 (the float16 pairs of the conversion are then adjacent tokens);
 *   K and V scale of group j: float16 element (tile * D / group + j) * 16 + t.
 * Codes are stored offset-binary (q + 8). Rounding is q4_kv.h's: scale =
 * float16_rne(float32(amax) / 7), q = clamp(rint_half_even(x / scale), -8, 7), 0 for a
 * zero scale; a group that holds an infinity or a NaN gets a NaN scale. group is 32, 64
 * or 128 and divides head_dim; pages * page_size < 2^31.
 * Nothing reads the contents of a slot that no sequence's length covers.
 */
#ifndef Q4_ATTN_H
#define Q4_ATTN_H

#include "q4.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  void* k_codes;  /* q4_paged_codes_bytes() bytes, 16-byte aligned     */
  void* k_scales; /* q4_paged_scales_count() float16, 8-byte aligned   */
  void* v_codes;
  void* v_scales;
  int64_t pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t group;
} q4_paged_kv;

/* Bytes of k_codes (and of v_codes), and float16 elements of k_scales (and of
 * v_scales); 0 for sizes the cache does not take (q4_last_error() says why). */
size_t q4_paged_codes_bytes(int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim);
size_t q4_paged_scales_count(int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim, int32_t group);

/* Rotation table of `positions` positions: float32 [positions][rot_dim / 2][2], the
 * cosine and sine of position * theta^(-2 i / rot_dim), angles taken in float64 (far
 * positions keep their phase). Models with scaled frequencies fill a table of the
 * same layout themselves. rot_dim is a positive multiple of 16; table 16-byte aligned. */
q4_status q4_rope_table(int64_t positions, int32_t rot_dim, double theta, float* table, void* stream);

/* RMS norm of every q and k head and the rotation by position, in one pass:
 *   h = x * w / sqrt(mean(x^2) + eps)            (weight NULL: h = x),
 *   (h_a, h_b) -> (h_a c - h_b s, h_b c + h_a s)  for the pairs of the first rot_dim
 * channels, (i, i + rot_dim / 2), or (2i, 2i + 1) with `interleaved`; c, s =
 * table[position][i]. The result is float16: q from float32 arithmetic, k from
 * float64 (quantized next, its values decide codes), rounded to float32 and then to
 * float16. q_weight and k_weight: float16 [head_dim], 16-byte aligned, each may be
 * NULL. positions: int32 [tokens]; one outside [0, table_positions) is taken as the nearest inside. table NULL or
 * rot_dim 0: no rotation (positions unused). q_heads or kv_heads may be 0. q_out and
 * k_out may be q and k themselves with the same stride; any other overlap gives
 * unspecified values. At most 2^26 - 4 tokens a call (here and in the append). */
q4_status q4_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens,
                          int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void* q_weight,
                          const void* k_weight, float eps, const int32_t* positions, const float* table,
                          int64_t table_positions, int32_t rot_dim, int32_t interleaved, void* q_out,
                          int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream);

/* q4_qk_norm_rope with k, rounded to float16 as above, and v quantized into the cache
 * at `slots` (int32 [tokens]) instead of k written out: the same bits as the two steps
 * one after the other. A slot outside [0, pages * page_size), -1 say, is a padded row:
 * its q is written, its k and v are not. Slots inside must differ from each other
 * (equal ones leave unspecified codes there). No other slot is touched. q_heads may
 * be 0. */
q4_status q4_qk_norm_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, int64_t tokens, int32_t q_heads, const void* q_weight,
                                 const void* k_weight, float eps, const int32_t* positions, const float* table,
                                 int64_t table_positions, int32_t rot_dim, int32_t interleaved, void* q_out,
                                 int64_t q_out_stride, const q4_paged_kv* cache, const int32_t* slots,
                                 void* stream);

/* Quantize k and v as they are into the cache at `slots` (rules as above). */
q4_status q4_paged_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t tokens,
                             const q4_paged_kv* cache, const int32_t* slots, void* stream);

/* The values of `slots` (int32 [tokens], any order, repeats allowed): k_out and v_out
 * float16 [tokens][kv_heads][head_dim] contiguous, 16-byte aligned, each code * scale
 * rounded once; zeros for a slot outside the cache. */
q4_status q4_paged_kv_dequant(const q4_paged_kv* cache, const int32_t* slots, int64_t tokens, void* k_out,
                              void* v_out, void* stream);

/* Attention of each sequence's newest tokens over its pages, causal:
 *   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale * q . k_t),
 * k and v the cache's code * scale unrounded. Rows q_offsets[n] .. q_offsets[n + 1] - 1
 * of q are sequence n's, the last of its kv_lens[n] tokens, whose k and v are in the
 * cache already: row i of n_q sees the keys t <= p = kv_lens[n] - n_q + i, and with
 * window > 0 only those with t > p - window. A decode step has one row a sequence, a
 * chunk of a prompt many; both may be mixed in a call. Token t of sequence n lies in
 * page block_table[n][t / page_size]; entries behind the length are not read. Pages may
 * be shared between sequences.
 *   q: float16 [tokens][q_heads][head_dim], q_stride elements from token to token;
 *   out: the same shape, contiguous, 8-byte aligned, overlapping no input; scale: within
 *   +-2e38 (0 and negative ones too), and within float32 times log2(e) and any K scale;
 *   block_table: int32 [seqs][max_blocks]; q_offsets: int32 [seqs + 1], ascending;
 *   kv_lens: int32 [seqs].
 *   max_q and max_kv bound the rows and the length of every sequence; they size the
 *   launch and the workspace, so a captured graph serves any lengths up to them. They
 *   also pick one form of the kernel for the whole call: beside long chunks a single
 *   token's context is read by one workgroup per KV head, several times slower than
 *   among single tokens, so long chunks are better given a call of their own.
 * A row that sees no key (an empty sequence, a row ahead of its sequence's start) is
 * zero; one whose scores are all -infinity, or one of them +infinity (infinities in q,
 * scores beyond float32), is NaN, as its softmax is. Rows of no sequence are left as
 * they were. Lengths, offsets and rows beyond the bounds are cut to them, and the keys
 * of a page number outside [0, pages) count as hidden, so no contents of these arrays
 * lead outside the buffers. q . k is taken with the exact codes and held in float32, as
 * the softmax is; the weights are rounded to float16 with the V scale in them before they
 * meet the codes (11 bits down to 2^-26 of the largest product of weight and V scale, in
 * steps of 2^-36 of it below), out is rounded once. The result does not depend on timing:
 * partial results of a split context are joined in a fixed order. Where a context is
 * split depends on the bounds, on the other sequences' lengths and on the device's
 * size, so a row's last bits may differ between batches it is part of.
 * `workspace` (16-byte aligned) must hold q4_paged_attention_workspace_bytes() bytes
 * on the device that the call runs on, taken there with the call's own bounds (NULL
 * when that is 0, else Q4_ERR_WORKSPACE); contents as q4_gemm's. seqs, heads and max_q
 * whose launch would need 2^24 workgroups are refused (Q4_ERR_SHAPE). */
size_t q4_paged_attention_workspace_bytes(int64_t seqs, int64_t tokens, int64_t max_q, int64_t max_kv,
                                          int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t group,
                                          int64_t window);
q4_status q4_paged_attention(const void* q, int64_t q_stride, const q4_paged_kv* cache, const int32_t* block_table,
                             int64_t max_blocks, const int32_t* q_offsets, const int32_t* kv_lens, int64_t seqs,
                             int64_t tokens, int64_t max_q, int64_t max_kv, int32_t q_heads, float scale,
                             int64_t window, void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Attention of requests that share long prefixes (a system prompt, a document), each prefix
 * stored once and read once for all rows behind it (for each sequence's by themselves where the
 * sequences have 640 or more of a KV head's rows and are of like sizes, at least a third of max_q tokens or
 * 2048 rows on average): q4_paged_attention, without a window, of sequences whose first keys are their group's prefix. Sequences group_offsets[g] ..
 * group_offsets[g + 1] - 1 (int32 [groups + 1], ascending) are group g's; token t <
 * prefix_lens[g] (int32 [groups]) of its prefix lies in page prefix_table[g][t / page_size]
 * (int32 [groups][max_prefix_blocks]). Every row of the group sees all of them, and its own
 * sequence's keys as q4_paged_attention has them: kv_lens, block_table and max_kv count the
 * keys behind the prefix only. A sequence of no group has no prefix. A prefix need not end
 * where a page does; the rotation of the keys behind it counts from its length (starts of
 * q4_paged_plan).
 * max_group_q and max_prefix (with max_kv below 2^30) bound the rows of a group's sequences together
 * and the prefixes' lengths; rows of a group beyond max_group_q are taken as having no prefix, longer prefixes
 * are cut. With few rows behind a short prefix, or hundreds in every sequence, a plain call whose
 * block tables begin with the prefix's pages is about as fast or faster (64 heads over 8: nine chunks of up to
 * 251 tokens behind 6001 keys 492 us, 496 here; all of 251: 586, 688). Everything else, rows that see no key, infinities and what
 * results depend on among it, is q4_paged_attention's. groups * heads * max_group_q
 * is refused as seqs * heads * max_q is. */
size_t q4_paged_attention_shared_workspace_bytes(int64_t seqs, int64_t groups, int64_t tokens, int64_t max_q,
                                                 int64_t max_kv, int64_t max_group_q, int64_t max_prefix,
                                                 int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t group);
q4_status q4_paged_attention_shared(const void* q, int64_t q_stride, const q4_paged_kv* cache,
                                    const int32_t* prefix_table, int64_t max_prefix_blocks,
                                    const int32_t* prefix_lens, const int32_t* group_offsets, int64_t groups,
                                    const int32_t* block_table, int64_t max_blocks, const int32_t* q_offsets,
                                    const int32_t* kv_lens, int64_t seqs, int64_t tokens, int64_t max_q,
                                    int64_t max_kv, int64_t max_group_q, int64_t max_prefix, int32_t q_heads,
                                    float scale, void* out, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4_ATTN_H */
