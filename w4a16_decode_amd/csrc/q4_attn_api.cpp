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
  q4_status st = check_paged(cache, &a.cache);
  if (st != Q4_OK) return st;
  if ((st = check_attn(seqs, tokens, max_q, max_kv, q_heads, a.cache.kv_heads, window)) != Q4_OK) return st;
  if (max_blocks < 0 || max_blocks >= kMaxDim)
    return fail(Q4_ERR_SHAPE, "max_blocks=%lld out of range", (long long)max_blocks);
  // times log2(e) it has to stay finite
  if (!(scale > -2.0e38f && scale < 2.0e38f)) return fail(Q4_ERR_SHAPE, "scale must be within +-2e38");
  if (seqs == 0 || tokens == 0 || max_q == 0) return ok();
  if ((st = check_rows("q", q, q_stride, q_heads, a.cache.head_dim)) != Q4_OK) return st;
  if (!q_offsets || !kv_lens || !out || (!block_table && max_blocks > 0 && max_kv > 0))
    return fail(Q4_ERR_NULL, "block_table, q_offsets, kv_lens, out must be non-NULL");
  if (!aligned(out, 8) || !aligned(block_table, 4) || !aligned(q_offsets, 4) || !aligned(kv_lens, 4))
    return fail(Q4_ERR_ALIGN, "out needs 8-byte, block_table, q_offsets and kv_lens 4-byte alignment");
  a.q = q, a.q_stride = q_stride, a.block_table = block_table, a.max_blocks = (int)max_blocks;
  a.q_offsets = q_offsets, a.kv_lens = kv_lens, a.seqs = (int)seqs, a.tokens = (int)tokens;
  a.max_q = (int)std::min(max_q, tokens), a.max_kv = (int)max_kv, a.q_heads = q_heads;
  a.scale = scale, a.window = (int)window, a.out = out;
  st = pick_attn(seqs, tokens, max_q, max_kv, q_heads, a.cache.kv_heads, a.cache.head_dim, a.cache.group, window, &a);
  if (st != Q4_OK) return st;
  if (a.shares > 0 || a.tail > 0) {
    const size_t parts = attn_parts(a), need = attn_workspace(a, a.cache.head_dim);
    if (!workspace || workspace_bytes < need)
      return fail(Q4_ERR_WORKSPACE, "this call needs %zu bytes of workspace (q4_paged_attention_workspace_bytes), got %zu",
                  need, workspace ? workspace_bytes : (size_t)0);
    if (!aligned(workspace, 16)) return fail(Q4_ERR_ALIGN, "workspace needs 16-byte alignment");
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = a.part_o + parts * a.cache.head_dim;
    a.cuts = reinterpret_cast<int32_t*>(a.part_ml + 2 * parts);
  }
  return hip_status(q4::launch_attention(a, static_cast<hipStream_t>(stream)), "attention launch");
}

}  // extern "C"
