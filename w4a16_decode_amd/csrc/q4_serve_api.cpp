// C ABI front end of the serving loop's calls (include/q4_serve.h): argument validation on
// the host, before any HIP call.
#include <algorithm>
#include <type_traits>

#include <hip/hip_runtime.h>

#include "../../include/q4_serve.h"
#include "q4_check.h"
#include "q4_internal.h"

using q4::aligned;
using q4::fail;
using q4::hip_status;
using q4::kMaxDim;
using q4::ok;

namespace {

constexpr int64_t kMaxSeqs = 65536, kMaxVocab = int64_t(1) << 20, kMaxRows = int64_t(1) << 22;

// Fractional bits of the weights: the sum of a row's stays below 2^63.
int weight_shift(int64_t vocab) {
  int bits = 0;
  while ((int64_t(1) << bits) < vocab) ++bits;
  return std::min(50, 62 - bits);
}

// Chunks of a row; 0: a workgroup takes the whole row, in one launch instead of four. Up to 32768 logits fit
// its registers, but from 16384 on few rows leave most of the chip idle meanwhile. In a graph, a whole
// row / chunks, us: 16000 float16 logits, 1 row: softmax 8.1 / 12.7, top-p 16.9 / 22.5; 256 rows: 9.8 / 17.5,
// 18.5 / 31.6. 32000 logits, 1 row: 12.9 / 13.0, 28.8 / 22.5; 17 rows: 13.3 / 13.7, 31.0 / 25.0; 64 rows: 13.6 / 14.9,
// 30.8 / 27.4 (with top-k too: 17.6 / 20.8); 256 rows: 14.6 / 22.3, 31.5 / 44.5.
constexpr int64_t kFewRows = 32;
int64_t sample_chunks(int64_t rows, int64_t vocab) {
  const bool whole = vocab <= 16384 || (vocab <= 32768 && rows > kFewRows);
  return whole ? 0 : (vocab + q4::kSampleChunk - 1) / q4::kSampleChunk;
}

q4_status check_sample(int64_t rows, int64_t vocab) {
  if (rows < 0 || rows >= kMaxRows || vocab <= 0 || vocab > kMaxVocab || rows * sample_chunks(rows, vocab) > q4::kMaxGroups256)
    return fail(Q4_ERR_SHAPE, "rows=%lld, vocab=%lld out of range", (long long)rows, (long long)vocab);
  return Q4_OK;
}

// The workspace's parts, from `base` on (NULL: their size alone), the widest elements first.
size_t place_sample(q4::SampleArgs* a, unsigned char* base) {
  const size_t rows = a->rows, all = rows * a->chunks;
  size_t at = 0;
  if (a->chunks == 0) return 0;
  auto part = [&](auto** p, size_t n) {
    *p = reinterpret_cast<std::remove_reference_t<decltype(*p)>>(base + at);
    at += (n * sizeof(**p) + 15) / 16 * 16;
  };
  part(&a->cuts, rows);
  part(&a->bins, rows * q4::kSampleBins);
  part(&a->sums, all);
  part(&a->cut_sums, 2 * rows);
  part(&a->tops, all);
  part(&a->counts, all);
  part(&a->list, all * q4::kSampleChunk);
  return at;
}

}  // namespace

extern "C" {

size_t q4_paged_plan_workspace_bytes(int64_t seqs, int64_t tokens) {
  if (seqs < 0 || seqs > kMaxSeqs || tokens < 0 || tokens >= kMaxDim) return 0;
  return q4::plan_one_launch(seqs, tokens) ? 0 : (size_t)(2 * seqs + 2) * 4;
}

q4_status q4_paged_plan(const int32_t* kv_lens, const int32_t* new_lens, const int32_t* reset, const int32_t* starts,
                        int64_t seqs, int64_t tokens, int32_t page_size, int64_t pages, int32_t* block_table,
                        int64_t max_blocks, int32_t* free_pages, const int32_t* free_count, int32_t* q_offsets,
                        int32_t* positions, int32_t* slots, int32_t* kv_lens_out, int32_t* free_count_out,
                        int32_t* lacking, void* workspace, size_t workspace_bytes, void* stream) {
  if (seqs < 0 || seqs > kMaxSeqs || tokens < 0 || tokens >= kMaxDim)
    return fail(Q4_ERR_SHAPE, "seqs=%lld, tokens=%lld out of range", (long long)seqs, (long long)tokens);
  if (page_size <= 0 || page_size % 16 != 0 || page_size >= kMaxDim)
    return fail(Q4_ERR_SHAPE, "page_size=%d must be a positive multiple of 16", (int)page_size);
  if (pages <= 0 || pages >= kMaxDim || pages * page_size >= (int64_t(1) << 31))
    return fail(Q4_ERR_SHAPE, "pages=%lld must be positive and pages * page_size below 2^31", (long long)pages);
  if (max_blocks < 0 || max_blocks >= kMaxDim || max_blocks * page_size > kMaxDim)
    return fail(Q4_ERR_SHAPE, "max_blocks=%lld: max_blocks * page_size must be in [0, 2^30]", (long long)max_blocks);
  if (!q_offsets || !lacking) return fail(Q4_ERR_NULL, "q_offsets and lacking must be non-NULL");
  if (seqs > 0 && (!kv_lens || !kv_lens_out || (!block_table && max_blocks > 0)))
    return fail(Q4_ERR_NULL, "kv_lens, block_table, kv_lens_out must be non-NULL");
  if (tokens > 0 && (!positions || !slots)) return fail(Q4_ERR_NULL, "positions and slots must be non-NULL");
  if (free_pages && (!free_count || !free_count_out))
    return fail(Q4_ERR_NULL, "free_count and free_count_out must be non-NULL beside free_pages");
  for (const void* p : {(const void*)kv_lens, (const void*)new_lens, (const void*)reset, (const void*)starts,
                        (const void*)block_table, (const void*)free_pages, (const void*)free_count,
                        (const void*)q_offsets, (const void*)positions, (const void*)slots, (const void*)kv_lens_out,
                        (const void*)free_count_out, (const void*)lacking})
    if (!aligned(p, 4)) return fail(Q4_ERR_ALIGN, "the arrays need 4-byte alignment");
  const size_t need = q4_paged_plan_workspace_bytes(seqs, tokens);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(Q4_ERR_WORKSPACE, "this plan needs %zu bytes of workspace (q4_paged_plan_workspace_bytes), got %zu",
                need, workspace ? workspace_bytes : (size_t)0);
  if (need > 0 && !aligned(workspace, 8)) return fail(Q4_ERR_ALIGN, "workspace needs 8-byte alignment");
  q4::PlanArgs a{};
  a.kv_lens = kv_lens, a.new_lens = new_lens, a.reset = reset, a.starts = starts;
  a.seqs = (int)seqs, a.tokens = (int)tokens, a.page_size = page_size, a.pages = (int)pages;
  a.max_blocks = (int)max_blocks, a.block_table = block_table;
  a.free_pages = free_pages, a.free_count = free_count, a.free_count_out = free_count_out;
  a.q_offsets = q_offsets, a.positions = positions, a.slots = slots, a.kv_lens_out = kv_lens_out;
  a.lacking = lacking, a.seq_info = static_cast<int32_t*>(workspace);
  return hip_status(q4::launch_plan(a, static_cast<hipStream_t>(stream)), "plan launch");
}

size_t q4_sample_workspace_bytes(int64_t rows, int64_t vocab) {
  if (check_sample(rows, vocab) != Q4_OK) return 0;
  q4::SampleArgs a{};
  // what serves a number of rows serves fewer
  const int64_t n = sample_chunks(rows, vocab) == 0 ? std::min(rows, kFewRows) : rows;
  a.rows = (int)n, a.chunks = (int)sample_chunks(n, vocab);
  return place_sample(&a, nullptr);
}

q4_status q4_sample(const void* logits, int32_t dtype, int64_t stride, int64_t rows, int64_t vocab,
                    const float* uniforms, const float* temperature, const int32_t* top_k, const float* top_p,
                    const float* min_p, int32_t* tokens, float* probs, void* workspace, size_t workspace_bytes,
                    void* stream) {
  if (dtype != Q4_F16 && dtype != Q4_BF16 && dtype != Q4_F32)
    return fail(Q4_ERR_UNSUPPORTED, "dtype=%d: logits are float16, bfloat16 or float32", (int)dtype);
  q4_status st = check_sample(rows, vocab);
  if (st != Q4_OK) return st;
  if (rows > 1 && (stride < 0 || stride >= (int64_t(1) << 40)))
    return fail(Q4_ERR_SHAPE, "stride %lld is not in [0, 2^40)", (long long)stride);
  if (rows == 0) return ok();
  if (!logits || !uniforms || !tokens) return fail(Q4_ERR_NULL, "logits, uniforms, tokens must be non-NULL");
  if (!aligned(logits, dtype == Q4_F32 ? 4 : 2) || !aligned(uniforms, 4) || !aligned(temperature, 4) ||
      !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(probs, 4))
    return fail(Q4_ERR_ALIGN, "logits and the arrays need their elements' alignment");
  q4::SampleArgs a{};
  a.logits = logits, a.dtype = dtype, a.stride = rows > 1 ? stride : vocab;
  a.rows = (int)rows, a.vocab = (int)vocab;
  a.uniforms = uniforms, a.temperature = temperature, a.top_k = top_k, a.top_p = top_p, a.min_p = min_p;
  a.tokens = tokens, a.probs = probs, a.shift = weight_shift(vocab);
  a.chunks = (int)sample_chunks(rows, vocab);
  const size_t need = place_sample(&a, static_cast<unsigned char*>(workspace));
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(Q4_ERR_WORKSPACE, "this shape needs %zu bytes of workspace (q4_sample_workspace_bytes), got %zu", need,
                workspace ? workspace_bytes : (size_t)0);
  if (need > 0 && !aligned(workspace, 16)) return fail(Q4_ERR_ALIGN, "workspace needs 16-byte alignment");
  if (!top_k && !top_p) a.bins = nullptr;
  return hip_status(q4::launch_sample(a, static_cast<hipStream_t>(stream)), "sample launch");
}

}  // extern "C"
