// C ABI front end of the attention side (include/q4_attn.h): argument validation and
// launch-shape selection on the host, before any HIP call.
#include <algorithm>

#include <hip/hip_runtime.h>

#include "../../include/q4_attn.h"
#include "q4_check.h"
#include "q4_internal.h"

using q4::aligned;
using q4::fail;
using q4::hip_status;
using q4::kMaxDim;
using q4::kMaxGroups256;
using q4::ok;

namespace {

q4_status check_paged_dims(int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim, int32_t group) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(Q4_ERR_UNSUPPORTED, "head_dim=%d: the paged cache takes 64, 128 or 256", (int)head_dim);
  if (group != 32 && group != 64 && group != 128)
    return fail(Q4_ERR_GROUP, "KV group %d unsupported (32, 64 or 128)", (int)group);
  if (head_dim % group != 0)
    return fail(Q4_ERR_GROUP, "head_dim=%d must be a multiple of group %d", (int)head_dim, (int)group);
  if (pages <= 0 || pages >= kMaxDim || kv_heads <= 0 || kv_heads > 65535)
    return fail(Q4_ERR_SHAPE, "pages=%lld, kv_heads=%d out of range", (long long)pages, (int)kv_heads);
  if (page_size <= 0 || page_size % 16 != 0)
    return fail(Q4_ERR_SHAPE, "page_size=%d must be a positive multiple of 16", (int)page_size);
  if (pages * page_size >= (int64_t(1) << 31))
    return fail(Q4_ERR_SHAPE, "pages * page_size = %lld must be below 2^31", (long long)(pages * page_size));
  return Q4_OK;
}

q4_status check_paged(const q4_paged_kv* cache, q4::PagedArgs* c) {
  if (!cache) return fail(Q4_ERR_NULL, "cache must be non-NULL");
  q4_status st = check_paged_dims(cache->pages, cache->page_size, cache->kv_heads, cache->head_dim, cache->group);
  if (st != Q4_OK) return st;
  if (!cache->k_codes || !cache->k_scales || !cache->v_codes || !cache->v_scales)
    return fail(Q4_ERR_NULL, "the cache's k_codes, k_scales, v_codes, v_scales must be non-NULL");
  if (!aligned(cache->k_codes, 16) || !aligned(cache->v_codes, 16) || !aligned(cache->k_scales, 8) ||
      !aligned(cache->v_scales, 8))
    return fail(Q4_ERR_ALIGN, "the cache's codes need 16-byte, its scales 8-byte alignment");
  *c = q4::PagedArgs{cache->k_codes, cache->k_scales, cache->v_codes,  cache->v_scales, cache->pages,
                     cache->page_size, cache->kv_heads, cache->head_dim, cache->group};
  return Q4_OK;
}

// A [tokens][heads][head_dim] operand: strides cover a row and keep 16-byte rows.
q4_status check_rows(const char* name, const void* p, int64_t stride, int64_t heads, int64_t head_dim) {
  if (!p) return fail(Q4_ERR_NULL, "%s must be non-NULL", name);
  if (stride < heads * head_dim || stride >= (int64_t(1) << 40))
    return fail(Q4_ERR_SHAPE, "%s: stride %lld is not in [heads * head_dim = %lld, 2^40)", name, (long long)stride,
                (long long)(heads * head_dim));
  if (stride % 8 != 0 || !aligned(p, 16))
    return fail(Q4_ERR_ALIGN, "%s needs 16-byte alignment and a stride that is a multiple of 8", name);
  return Q4_OK;
}

// Checks and launch shared by the norm / rotation entry points; a.cache.head_dim etc.
// are set where a.append.
q4_status rope_common(q4::RopeArgs& a, void* stream) {
  if (a.tokens < 0 || a.tokens > 4 * kMaxGroups256)  // a wavefront per token or more of them
    return fail(Q4_ERR_SHAPE, "tokens=%lld out of range", (long long)a.tokens);
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256)
    return fail(Q4_ERR_UNSUPPORTED, "head_dim=%d unsupported (64, 128 or 256)", a.head_dim);
  if (a.q_heads < 0 || a.kv_heads < 0 || a.q_heads > 65535 || a.kv_heads > 65535)
    return fail(Q4_ERR_SHAPE, "q_heads=%d, kv_heads=%d out of range", a.q_heads, a.kv_heads);
  if (!a.table) a.rot = 0;
  if (a.rot < 0 || a.rot > a.head_dim || a.rot % 16 != 0)
    return fail(Q4_ERR_UNSUPPORTED, "rot_dim=%d must be a multiple of 16 in [0, head_dim]", a.rot);
  if (a.rot > 0 && (a.table_positions <= 0 || a.table_positions >= kMaxDim))
    return fail(Q4_ERR_SHAPE, "table_positions=%lld out of range", (long long)a.table_positions);
  if ((a.q_weight || a.k_weight) && !(a.eps >= 0.0f && a.eps <= 3.0e38f))
    return fail(Q4_ERR_SHAPE, "eps must be a finite number >= 0");
  if (a.tokens == 0 || (a.q_heads == 0 && a.kv_heads == 0)) return ok();
  q4_status st;
  if (a.q_heads > 0) {
    if ((st = check_rows("q", a.q, a.q_stride, a.q_heads, a.head_dim)) != Q4_OK) return st;
    if ((st = check_rows("q_out", a.q_out, a.q_out_stride, a.q_heads, a.head_dim)) != Q4_OK) return st;
  }
  if (a.kv_heads > 0) {
    if ((st = check_rows("k", a.k, a.k_stride, a.kv_heads, a.head_dim)) != Q4_OK) return st;
    if (a.append) {
      if ((st = check_rows("v", a.v, a.v_stride, a.kv_heads, a.head_dim)) != Q4_OK) return st;
    } else if ((st = check_rows("k_out", a.k_out, a.k_out_stride, a.kv_heads, a.head_dim)) != Q4_OK) {
      return st;
    }
  }
  if (a.append && !a.slots) return fail(Q4_ERR_NULL, "slots must be non-NULL");
  if (a.rot > 0 && !a.positions) return fail(Q4_ERR_NULL, "positions must be non-NULL");
  if ((a.q_weight && !aligned(a.q_weight, 16)) || (a.k_weight && !aligned(a.k_weight, 16)) ||
      (a.rot > 0 && (!aligned(a.table, 16) || !aligned(a.positions, 4))) || (a.append && !aligned(a.slots, 4)))
    return fail(Q4_ERR_ALIGN, "weights and table need 16-byte, positions and slots 4-byte alignment");
  return hip_status(q4::launch_rope(a, static_cast<hipStream_t>(stream)), "norm and rotation launch");
}

// Sizes of an attention call; q_heads in whole shares of kv_heads.
q4_status check_attn(int64_t seqs, int64_t tokens, int64_t max_q, int64_t max_kv, int32_t q_heads, int32_t kv_heads,
                     int64_t window) {
  if (seqs < 0 || tokens < 0 || max_q < 0 || max_kv < 0 || seqs >= kMaxDim || tokens >= kMaxDim || max_q >= kMaxDim ||
      max_kv >= kMaxDim)
    return fail(Q4_ERR_SHAPE, "seqs=%lld, tokens=%lld, max_q=%lld, max_kv=%lld out of range", (long long)seqs,
                (long long)tokens, (long long)max_q, (long long)max_kv);
  if (window < 0 || window >= kMaxDim) return fail(Q4_ERR_SHAPE, "window=%lld out of range", (long long)window);
  if (kv_heads <= 0 || q_heads <= 0 || q_heads > 65535 || q_heads % kv_heads != 0)
    return fail(Q4_ERR_SHAPE, "q_heads=%d must be a positive multiple of kv_heads=%d", (int)q_heads, (int)kv_heads);
  const int64_t rows = std::min(max_q, tokens) * (q_heads / kv_heads);
  if (rows >= kMaxDim || (rows / 16 + 1) * kv_heads >= kMaxDim / std::max<int64_t>(seqs, 1))
    return fail(Q4_ERR_SHAPE, "seqs * heads * max_q too large for one call");
  return Q4_OK;
}

// Launch shape (q4_attn.hip), from the bounds alone and one for all sequences of the call (a 512-token
// chunk and 47 single tokens over 8K contexts: 995 us together, 327 in two calls); the rows are those
// that a KV head's new tokens of one sequence have.
//   up to 16: the 16-row kernel (one tile holds them all);
//   more: 128 a workgroup where those workgroups are two or more a CU, so that nothing has to
//     be cut but the last round (sixteen 509-token chunks of 64 heads over 8: 870 TFLOP/s, 32-row
//     tiles 760);
//   else 32-row tiles (8 sequences of 5 tokens over 8K: 42 us; 128-row workgroups would leave
//     three quarters of the chip idle), or 16-row ones where the 32-row kernel is not built.
// The 16- and 32-row kernels take equal shares of all the work, cut anywhere (48 rows over
// unequal 8K contexts 77 -> 68 us against a fixed number of cuts); where the keys of a row are
// at most 512, one share's smallest piece, a workgroup takes a whole job and no join
// is launched (16 rows over 512 keys: 7.0 us, 2 us less than with the join).
// Workgroups of 128 rows that fill the chip a whole number of times take their jobs whole; the
// jobs left over are cut, so that their last round is full too, into pieces of 1536 keys
// or more by the bounds (1024 jobs of up to 8190 keys 626 -> 512 us, 896 of 4096 246 -> 204;
// pieces of 1280 keys: 142 -> 150 us for 896 jobs of up to 2600; of 1024: 102 -> 117 us for 1024 jobs
// of up to 2048, whose partial results cost more than the round has left to give).
q4_status pick_attn(int64_t seqs, int64_t tokens, int64_t max_q, int64_t max_kv, int32_t q_heads, int32_t kv_heads,
                    int32_t head_dim, int32_t group, int64_t window, q4::AttnArgs* a) {
  const int64_t rows = std::min(max_q, tokens) * (q_heads / kv_heads);
  const int64_t groups = kv_heads * seqs;
  const bool fill = (rows + 127) / 128 * groups >= 2 * q4::device_cu_count_cached();
  a->rows_group = rows > 32 && fill ? 128 : rows <= 16 || !q4::has_attn32(head_dim, head_dim / group) ? 16 : 32;
  const int64_t span = window > 0 ? std::min(max_kv, window + std::min(max_q, tokens)) : max_kv;
  a->shares = a->rows_group == 128 || span <= 512 ? 0 : q4::attention_resident(head_dim, group, a->rows_group);
  const int64_t jobs = (rows + a->rows_group - 1) / a->rows_group * groups;
  int64_t grid = a->shares > 0 ? a->shares : jobs;
  if (a->rows_group == 128) {
    const int64_t slots = q4::attention_resident(head_dim, group, 128), rest = jobs % slots;
    const int64_t pieces = rest > 0 ? std::min(slots / rest, span / 1536) : 0;
    if (pieces > 1) a->tail = (int)rest, a->pieces = (int)pieces;
    grid = jobs - a->tail + (int64_t)a->tail * a->pieces;
    a->whole = (int)std::min(jobs - a->tail, kMaxDim);
  }
  if (grid > kMaxGroups256) return fail(Q4_ERR_SHAPE, "seqs * heads * max_q too large for one call");
  return Q4_OK;
}

size_t attn_parts(const q4::AttnArgs& a) {
  return (size_t)a.shares * 2 * a.rows_group + (size_t)a.tail * a.pieces * a.rows_group;
}
size_t attn_workspace(const q4::AttnArgs& a, int32_t head_dim) {
  return attn_parts(a) * (head_dim + 2) * 4 + (size_t)a.shares * 32;
}

// The checks of an attention call and its arguments with the launch shape; *any: whether there is something
// to launch.
q4_status attn_args(const void* q, int64_t q_stride, const q4_paged_kv* cache, const int32_t* block_table,
                    int64_t max_blocks, const int32_t* q_offsets, const int32_t* kv_lens, int64_t seqs, int64_t tokens,
                    int64_t max_q, int64_t max_kv, int32_t q_heads, float scale, int64_t window, void* out,
                    q4::AttnArgs* to, bool* any) {
  q4::AttnArgs& a = *to;
  q4_status st = check_paged(cache, &a.cache);
  if (st != Q4_OK) return st;
  if ((st = check_attn(seqs, tokens, max_q, max_kv, q_heads, a.cache.kv_heads, window)) != Q4_OK) return st;
  if (max_blocks < 0 || max_blocks >= kMaxDim)
    return fail(Q4_ERR_SHAPE, "max_blocks=%lld out of range", (long long)max_blocks);
  // times log2(e) it has to stay finite
  if (!(scale > -2.0e38f && scale < 2.0e38f)) return fail(Q4_ERR_SHAPE, "scale must be within +-2e38");
  *any = seqs > 0 && tokens > 0 && max_q > 0;
  if (!*any) return Q4_OK;
  if ((st = check_rows("q", q, q_stride, q_heads, a.cache.head_dim)) != Q4_OK) return st;
  if (!q_offsets || !kv_lens || !out || (!block_table && max_blocks > 0 && max_kv > 0))
    return fail(Q4_ERR_NULL, "block_table, q_offsets, kv_lens, out must be non-NULL");
  if (!aligned(out, 8) || !aligned(block_table, 4) || !aligned(q_offsets, 4) || !aligned(kv_lens, 4))
    return fail(Q4_ERR_ALIGN, "out needs 8-byte, block_table, q_offsets and kv_lens 4-byte alignment");
  a.q = q, a.q_stride = q_stride, a.block_table = block_table, a.max_blocks = (int)max_blocks;
  a.q_offsets = q_offsets, a.kv_lens = kv_lens, a.seqs = (int)seqs, a.tokens = (int)tokens;
  a.max_q = (int)std::min(max_q, tokens), a.max_kv = (int)max_kv, a.q_heads = q_heads;
  a.scale = scale, a.window = (int)window, a.out = out;
  return pick_attn(seqs, tokens, max_q, max_kv, q_heads, a.cache.kv_heads, a.cache.head_dim, a.cache.group, window, &a);
}

q4_status check_workspace(const void* workspace, size_t bytes, size_t need, const char* from) {
  if (!workspace || bytes < need)
    return fail(Q4_ERR_WORKSPACE, "this call needs %zu bytes of workspace (%s), got %zu", need, from,
                workspace ? bytes : (size_t)0);
  if (!aligned(workspace, 16)) return fail(Q4_ERR_ALIGN, "workspace needs 16-byte alignment");
  return Q4_OK;
}

void place_parts(q4::AttnArgs* a, void* workspace) {
  const size_t parts = attn_parts(*a);
  a->part_o = static_cast<float*>(workspace);
  a->part_ml = a->part_o + parts * a->cache.head_dim;
  a->cuts = reinterpret_cast<int32_t*>(a->part_ml + 2 * parts);
}

// Shared prefixes: sizes beyond those of check_attn.
q4_status check_prefix(int64_t groups, int64_t tokens, int64_t max_kv, int64_t max_group_q, int64_t max_prefix,
                       int32_t q_heads, int32_t kv_heads) {
  if (groups < 0 || max_group_q < 0 || max_prefix < 0 || groups >= kMaxDim || max_group_q >= kMaxDim ||
      max_prefix + max_kv >= kMaxDim)
    return fail(Q4_ERR_SHAPE, "groups=%lld, max_group_q=%lld, max_prefix=%lld (and max_kv) out of range", (long long)groups,
                (long long)max_group_q, (long long)max_prefix);
  return check_attn(groups, tokens, max_group_q, max_prefix, q_heads, kv_heads, 0);
}
bool has_prefix(int64_t groups, int64_t tokens, int64_t max_group_q, int64_t max_prefix) {
  return groups > 0 && tokens > 0 && max_group_q > 0 && max_prefix > 0;
}

// Launch shape of an attention call with shared prefixes, whose own keys' shape pick_attn has picked already.
//   Up to 256 rows of a group a KV head: one launch of 16-row tiles over prefixes and own keys, cut
//     into pieces of equal length until they are one round of the chip, then a join (8 sequences
//     behind 4000 keys, 64 heads over 8: 42 -> 20 us against prefixes first and own keys from there;
//     of 256 rows behind 8000 keys 40 -> 33, of 512 57 -> 67). Counted are the tiles that the call's rows can
//     fill at most, not those that the bounds allow: empty ones end at once (five groups of 41 rows in all,
//     bound 26: 50 us when the bounds' were counted). Not for long sequences outside the groups that are
//     eight tiles a CU and more, each of which would convert the same codes and leave partial results (8 rows
//     behind 8190 keys beside a prompt of 320, 640, 4000 tokens, this form / prefixes first: 80 / 100, 129 / 115,
//     971 / 441 us; 32 rows in 8 groups beside 8 prompts of 40, 80, 640: 57 / 53, 96 / 54, 634 / 159).
//   Else, 640 or more of a sequence: its rows fill tiles by themselves, so prefix and own keys are walked as
//     one line of keys, 128 rows a workgroup; jobs that do not fill the chip a whole number of times are
//     cut and joined (nine chunks of up to 251 rows behind 6001 keys: 552 us with the prefix first). A line reads its
//     prefix by itself, for one row as for 128, so only where the sequences have a third of max_q tokens each on
//     average, or 2048 rows (max_q may be a loose bound), and none longer than a group's lies outside the groups. Lines /
//     prefix first, us: behind 8190 keys 1 chunk of 512 tokens and 63 single ones 1302 / 465; 16 and 48 (1030 rows on
//     average) 3723 / 3381; 32 and 32 6120 / 6493; 64 chunks of 100 2277 / 2553, 32 and 32 single tokens 1382 /
//     1370; 1 of 4000 and 8 single (3562 rows) 1770 / 1856; behind 4000 1 of 2000 and 8 (1784) 628 / 505, 2 and 8 (3206)
//     918 / 976; 8 prompts of 640 in no group beside 32 single tokens 319 / 159. With max_q eight times the chunks'
//     length: 5 of 150 262 / 230, 64 of 100 782 / 880, 6 of 300 (2400) 390 / 446.
//   Else: 128-row workgroups over the prefixes, cut until they fill the chip, and the rows behind start
//     from those pieces. There a workgroup takes all of a row's own keys up to 4096 (64 rows behind 8190
//     keys, own keys up to 513: 75 us with equal shares of them and a join, 57 so; up to 2000: 90, 69).
constexpr int64_t kMaxPieces = 64;
q4_status pick_shared(int64_t groups, int64_t max_group_q, int64_t max_prefix, q4::AttnArgs* a) {
  const int heads = a->cache.kv_heads, share = a->q_heads / heads, d = a->cache.head_dim, g = a->cache.group;
  a->groups = (int)groups, a->max_group_q = (int)std::min<int64_t>(max_group_q, a->tokens), a->max_prefix = (int)max_prefix;
  const int64_t rows = (int64_t)a->max_group_q * share, own_rows = (int64_t)a->max_q * share;
  const bool prompts = own_rows > 256 && (int64_t)a->tokens * a->q_heads / 16 > 8 * q4::device_cu_count_cached();
  if (rows <= 256 && !prompts) {
    a->rows_group = 16, a->shares = 0, a->whole = 0, a->tail = 0, a->pieces = 0;
    const int64_t tiles = (rows + 15) / 16, own = (own_rows + 15) / 16 * heads * a->seqs;
    const int64_t filled = (int64_t)a->tokens * share / 16;
    const int64_t jobs = std::min(tiles * groups, filled + groups) * heads;
    const int64_t own_jobs = std::min(own, (filled + a->seqs) * heads);
    const int64_t slots = q4::prefix_attention_resident(d, g, 16);
    auto pieces = [](int64_t keys, int64_t units) { return std::max<int64_t>(1, (keys + 128 * units - 1) / (128 * units)); };
    int64_t lo = (std::max<int64_t>(max_prefix, a->max_kv) + 128 * kMaxPieces - 1) / (128 * kMaxPieces);
    int64_t hi = std::max<int64_t>(max_prefix, a->max_kv) / 128 + 1;  // units of 128 keys a piece
    lo = std::max<int64_t>(lo, 1);
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (jobs * pieces(max_prefix, mid) + own_jobs * pieces(a->max_kv, mid) <= slots) hi = mid; else lo = mid + 1;
    }
    a->prefix_pieces = (int)pieces(max_prefix, lo), a->own_pieces = (int)pieces(a->max_kv, lo);
    a->prefix_rows = (int)(tiles * 16);
    if (tiles * groups * heads * a->prefix_pieces + own * a->own_pieces > kMaxGroups256 || own > kMaxGroups256 / 2)
      return fail(Q4_ERR_SHAPE, "groups * heads * max_group_q too large for one call");
    return Q4_OK;
  }
  a->own_pieces = 0;
  const bool alike = 3 * (int64_t)a->tokens >= (int64_t)a->seqs * a->max_q ||
                     (int64_t)a->tokens * share >= 2048 * (int64_t)a->seqs;
  if (own_rows >= 640 && alike && a->max_group_q >= a->max_q) {
    const int64_t jobs = (own_rows + 127) / 128 * heads * a->seqs, slots = q4::line_attention_resident(d, g);
    // of these the call's rows fill about so many; the last round's share of them is cut, and a tenth of a round
    // more, so that no whole job is left for it where the lengths are ragged (9 chunks of up to 251 tokens behind 6001
    // keys 626 -> 496 us, 12 of up to 160 behind 8190 803 -> 555). Chunks of one length, whose number is
    // estimated well, lose up to a tenth by it (all of 251 624 -> 688, of 160 678 -> 737, 16 of 200 1100 -> 1133).
    const int64_t full = std::min(jobs, ((int64_t)a->tokens * share / 128 + (a->seqs + 1) / 2) * heads);
    int64_t rest = full % slots;
    if (full > slots && rest > 0) rest = std::min(rest + slots / 10, slots);
    const int64_t pieces = rest > 0 ? std::min(slots / rest, (max_prefix + a->max_kv) / 512) : 0;
    a->prefix_pieces = a->prefix_rows = 0;
    a->rows_group = 128, a->shares = 0;
    a->tail = pieces > 1 ? (int)std::min<int64_t>(rest * jobs / full, kMaxDim) : 0;
    a->pieces = pieces > 1 ? (int)pieces : 0;
    a->whole = (int)std::min(jobs - a->tail, kMaxDim);
    if (jobs > kMaxGroups256 || a->whole + a->tail * (int64_t)a->pieces > kMaxGroups256 ||
        a->tail * int64_t(32) > kMaxGroups256)
      return fail(Q4_ERR_SHAPE, "seqs * heads * max_q too large for one call");
    return Q4_OK;
  }
  if (a->max_kv <= 4096 && a->shares > 0) {  // then a workgroup a tile, which pick_attn has not counted
    a->shares = 0;
    if ((own_rows + a->rows_group - 1) / a->rows_group * heads * a->seqs > kMaxGroups256)
      return fail(Q4_ERR_SHAPE, "seqs * heads * max_q too large for one call");
  }
  const int64_t jobs = (rows + 127) / 128 * heads * groups;
  const int64_t slots = q4::prefix_attention_resident(d, g, 128);
  const int64_t pieces = std::max<int64_t>(1, std::min(slots / jobs, (max_prefix + 255) / 256));
  if (jobs * pieces > kMaxGroups256 / 2) return fail(Q4_ERR_SHAPE, "groups * heads * max_group_q too large for one call");
  a->prefix_pieces = (int)pieces, a->prefix_rows = (int)((rows + 127) / 128 * 128);
  return Q4_OK;
}

// Partial results over the prefixes; those over the keys behind them follow.
size_t prefix_parts(const q4::AttnArgs& a) {
  return (size_t)a.prefix_pieces * a.groups * a.cache.kv_heads * a.prefix_rows;
}
size_t prefix_bytes(const q4::AttnArgs& a) {
  return (size_t)q4::round_up(prefix_parts(a) * (a.cache.head_dim + 2) * 4, 256);
}
size_t shared_workspace(const q4::AttnArgs& a) {
  const size_t own = (size_t)a.own_pieces * a.tokens * a.q_heads * (a.cache.head_dim + 2) * 4;
  return prefix_bytes(a) + (a.own_pieces > 0 ? own : attn_workspace(a, a.cache.head_dim));
}

}  // namespace

extern "C" {

size_t q4_paged_codes_bytes(int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim) {
  if (check_paged_dims(pages, page_size, kv_heads, head_dim, 32) != Q4_OK) return 0;
  return (size_t)pages * page_size * kv_heads * (head_dim / 2);
}

size_t q4_paged_scales_count(int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim, int32_t group) {
  if (check_paged_dims(pages, page_size, kv_heads, head_dim, group) != Q4_OK) return 0;
  return (size_t)pages * page_size * kv_heads * (head_dim / group);
}

q4_status q4_rope_table(int64_t positions, int32_t rot_dim, double theta, float* table, void* stream) {
  if (positions < 0 || positions >= kMaxDim) return fail(Q4_ERR_SHAPE, "positions=%lld out of range", (long long)positions);
  if (rot_dim <= 0 || rot_dim % 16 != 0 || rot_dim > 256)
    return fail(Q4_ERR_UNSUPPORTED, "rot_dim=%d must be a multiple of 16 in [16, 256]", (int)rot_dim);
  if (!(theta > 0.0) || theta > 1e300) return fail(Q4_ERR_SHAPE, "theta must be positive and finite");
  if (positions == 0) return ok();
  if (!table) return fail(Q4_ERR_NULL, "table must be non-NULL");
  if (!aligned(table, 16)) return fail(Q4_ERR_ALIGN, "table needs 16-byte alignment");
  return hip_status(q4::launch_rope_table(positions, rot_dim, theta, table, static_cast<hipStream_t>(stream)),
                    "rope table launch");
}

q4_status q4_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens,
                          int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void* q_weight,
                          const void* k_weight, float eps, const int32_t* positions, const float* table,
                          int64_t table_positions, int32_t rot_dim, int32_t interleaved, void* q_out,
                          int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  q4::RopeArgs a{};
  a.q = q, a.k = k, a.q_stride = q_stride, a.k_stride = k_stride;
  a.tokens = tokens, a.q_heads = q_heads, a.kv_heads = kv_heads, a.head_dim = head_dim;
  a.q_weight = q_weight, a.k_weight = k_weight, a.eps = eps;
  a.positions = positions, a.table = table, a.table_positions = table_positions, a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.q_out = q_out, a.k_out = k_out, a.q_out_stride = q_out_stride, a.k_out_stride = k_out_stride;
  return rope_common(a, stream);
}

q4_status q4_qk_norm_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, int64_t tokens, int32_t q_heads, const void* q_weight,
                                 const void* k_weight, float eps, const int32_t* positions, const float* table,
                                 int64_t table_positions, int32_t rot_dim, int32_t interleaved, void* q_out,
                                 int64_t q_out_stride, const q4_paged_kv* cache, const int32_t* slots,
                                 void* stream) {
  q4::RopeArgs a{};
  q4_status st = check_paged(cache, &a.cache);
  if (st != Q4_OK) return st;
  a.q = q, a.k = k, a.v = v, a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.tokens = tokens, a.q_heads = q_heads, a.kv_heads = a.cache.kv_heads, a.head_dim = a.cache.head_dim;
  a.q_weight = q_weight, a.k_weight = k_weight, a.eps = eps;
  a.positions = positions, a.table = table, a.table_positions = table_positions, a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.q_out = q_out, a.q_out_stride = q_out_stride;
  a.append = true, a.slots = slots;
  return rope_common(a, stream);
}

q4_status q4_paged_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t tokens,
                             const q4_paged_kv* cache, const int32_t* slots, void* stream) {
  return q4_qk_norm_rope_append(nullptr, 0, k, k_stride, v, v_stride, tokens, 0, nullptr, nullptr, 0.0f, nullptr,
                                nullptr, 0, 0, 0, nullptr, 0, cache, slots, stream);
}

q4_status q4_paged_kv_dequant(const q4_paged_kv* cache, const int32_t* slots, int64_t tokens, void* k_out,
                              void* v_out, void* stream) {
  q4::PagedArgs c;
  q4_status st = check_paged(cache, &c);
  if (st != Q4_OK) return st;
  if (tokens < 0 || tokens >= kMaxDim) return fail(Q4_ERR_SHAPE, "tokens=%lld out of range", (long long)tokens);
  if (tokens == 0) return ok();
  if (!slots || !k_out || !v_out) return fail(Q4_ERR_NULL, "slots, k_out, v_out must be non-NULL");
  if (!aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return fail(Q4_ERR_ALIGN, "slots need 4-byte, k_out and v_out 16-byte alignment");
  return hip_status(q4::launch_paged_dequant(c, slots, tokens, k_out, v_out, static_cast<hipStream_t>(stream)),
                    "paged dequant launch");
}

size_t q4_paged_attention_workspace_bytes(int64_t seqs, int64_t tokens, int64_t max_q, int64_t max_kv,
                                          int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t group,
                                          int64_t window) {
  if (check_attn(seqs, tokens, max_q, max_kv, q_heads, kv_heads, window) != Q4_OK) return 0;
  if (check_paged_dims(1, 16, kv_heads, head_dim, group) != Q4_OK) return 0;
  q4::AttnArgs a{};
  if (pick_attn(seqs, tokens, max_q, max_kv, q_heads, kv_heads, head_dim, group, window, &a) != Q4_OK) return 0;
  return attn_workspace(a, head_dim);
}

q4_status q4_paged_attention(const void* q, int64_t q_stride, const q4_paged_kv* cache, const int32_t* block_table,
                             int64_t max_blocks, const int32_t* q_offsets, const int32_t* kv_lens, int64_t seqs,
                             int64_t tokens, int64_t max_q, int64_t max_kv, int32_t q_heads, float scale,
                             int64_t window, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  q4::AttnArgs a{};
  bool any = false;
  q4_status st = attn_args(q, q_stride, cache, block_table, max_blocks, q_offsets, kv_lens, seqs, tokens, max_q, max_kv,
                           q_heads, scale, window, out, &a, &any);
  if (st != Q4_OK) return st;
  if (!any) return ok();
  if (a.shares > 0 || a.tail > 0) {
    const size_t need = attn_workspace(a, a.cache.head_dim);
    if ((st = check_workspace(workspace, workspace_bytes, need, "q4_paged_attention_workspace_bytes")) != Q4_OK) return st;
    place_parts(&a, workspace);
  }
  return hip_status(q4::launch_attention(a, static_cast<hipStream_t>(stream)), "attention launch");
}

size_t q4_paged_attention_shared_workspace_bytes(int64_t seqs, int64_t groups, int64_t tokens, int64_t max_q,
                                                 int64_t max_kv, int64_t max_group_q, int64_t max_prefix,
                                                 int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t group) {
  if (check_attn(seqs, tokens, max_q, max_kv, q_heads, kv_heads, 0) != Q4_OK) return 0;
  if (check_prefix(groups, tokens, max_kv, max_group_q, max_prefix, q_heads, kv_heads) != Q4_OK) return 0;
  if (check_paged_dims(1, 16, kv_heads, head_dim, group) != Q4_OK) return 0;
  q4::AttnArgs a{};
  a.cache.kv_heads = kv_heads, a.cache.head_dim = head_dim, a.cache.group = group;
  a.seqs = (int)seqs, a.tokens = (int)tokens, a.max_q = (int)std::min(max_q, tokens), a.max_kv = (int)max_kv;
  a.q_heads = q_heads;
  if (pick_attn(seqs, tokens, max_q, max_kv, q_heads, kv_heads, head_dim, group, 0, &a) != Q4_OK) return 0;
  if (seqs == 0 || max_q == 0 || !has_prefix(groups, tokens, max_group_q, max_prefix)) return attn_workspace(a, head_dim);
  if (pick_shared(groups, max_group_q, max_prefix, &a) != Q4_OK) return 0;
  return shared_workspace(a);
}

q4_status q4_paged_attention_shared(const void* q, int64_t q_stride, const q4_paged_kv* cache,
                                    const int32_t* prefix_table, int64_t max_prefix_blocks,
                                    const int32_t* prefix_lens, const int32_t* group_offsets, int64_t groups,
                                    const int32_t* block_table, int64_t max_blocks, const int32_t* q_offsets,
                                    const int32_t* kv_lens, int64_t seqs, int64_t tokens, int64_t max_q,
                                    int64_t max_kv, int64_t max_group_q, int64_t max_prefix, int32_t q_heads,
                                    float scale, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  q4::AttnArgs a{};
  bool any = false;
  q4_status st = attn_args(q, q_stride, cache, block_table, max_blocks, q_offsets, kv_lens, seqs, tokens, max_q, max_kv,
                           q_heads, scale, 0, out, &a, &any);
  if (st != Q4_OK) return st;
  if ((st = check_prefix(groups, tokens, max_kv, max_group_q, max_prefix, q_heads, a.cache.kv_heads)) != Q4_OK) return st;
  if (max_prefix_blocks < 0 || max_prefix_blocks >= kMaxDim)
    return fail(Q4_ERR_SHAPE, "max_prefix_blocks=%lld out of range", (long long)max_prefix_blocks);
  if (!any) return ok();
  const bool prefix = has_prefix(groups, tokens, max_group_q, max_prefix);
  size_t need = attn_workspace(a, a.cache.head_dim);
  if (prefix) {
    if (!prefix_lens || !group_offsets || (!prefix_table && max_prefix_blocks > 0))
      return fail(Q4_ERR_NULL, "prefix_table, prefix_lens, group_offsets must be non-NULL");
    if (!aligned(prefix_table, 4) || !aligned(prefix_lens, 4) || !aligned(group_offsets, 4))
      return fail(Q4_ERR_ALIGN, "prefix_table, prefix_lens and group_offsets need 4-byte alignment");
    a.prefix_table = prefix_table, a.prefix_blocks = (int)max_prefix_blocks, a.prefix_lens = prefix_lens;
    a.group_offsets = group_offsets;
    if ((st = pick_shared(groups, max_group_q, max_prefix, &a)) != Q4_OK) return st;
    need = shared_workspace(a);
  }
  if (need > 0) {
    st = check_workspace(workspace, workspace_bytes, need, "q4_paged_attention_shared_workspace_bytes");
    if (st != Q4_OK) return st;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!prefix) {
    place_parts(&a, workspace);
    return hip_status(q4::launch_attention(a, s), "attention launch");
  }
  a.prefix_o = static_cast<float*>(workspace);
  a.prefix_ml = a.prefix_o + prefix_parts(a) * a.cache.head_dim;
  void* behind = static_cast<unsigned char*>(workspace) + prefix_bytes(a);
  if (a.own_pieces > 0) {
    a.part_o = static_cast<float*>(behind);
    a.part_ml = a.part_o + (size_t)a.own_pieces * a.tokens * a.q_heads * a.cache.head_dim;
    return hip_status(q4::launch_both_attention(a, s), "attention with shared prefixes launch");
  }
  place_parts(&a, behind);
  if (a.prefix_pieces == 0)
    return hip_status(q4::launch_line_attention(a, s), "attention with shared prefixes launch");
  q4::AttnArgs p = a;  // over the prefixes every job is cut
  p.shares = 0, p.whole = 0, p.pieces = a.prefix_pieces, p.tail = a.prefix_rows / 128 * a.cache.kv_heads * a.groups;
  hipError_t e = q4::launch_prefix_attention(p, s);
  if (e == hipSuccess) e = q4::launch_behind_attention(a, s);
  return hip_status(e, "attention with shared prefixes launch");
}

}  // extern "C"
