// C ABI front end of the product with adapters (include/q4_lora.h).
#include <algorithm>

#include <hip/hip_runtime.h>

#include "../../include/q4_lora.h"
#include "q4_check.h"
#include "q4_internal.h"

using q4::aligned;
using q4::fail;
using q4::hip_status;
using q4::kMaxDim;
using q4::ok;
using q4::round_up;

namespace {

// Float32 sums of the product, then those of A x, each from a 256-byte boundary.
size_t product_bytes(int splits, int64_t B, int64_t out) { return (size_t)round_up(splits * B * out * 4, 256); }
size_t t_bytes(int64_t B, int64_t in, int32_t rank) { return (size_t)q4::lora_splits((int)in) * B * rank * 4; }

// Workgroups of the two adapter kernels (16 rows each, 16 distinct adapters, 256 outputs).
bool grid_ok(int64_t B, int64_t out, int64_t in) {
  return (B + 15) / 16 * std::max<int64_t>(16 * q4::lora_splits((int)in), (out + 255) / 256) <= q4::kMaxGroups256;
}

bool rank_ok(int32_t rank) { return rank >= 8 && rank <= 128 && rank % 8 == 0; }

}  // namespace

extern "C" {

size_t q4_workspace_bytes_lora(int64_t B, int64_t out, int64_t in, int32_t group, int32_t rank) {
  if (B <= 0 || !rank_ok(rank)) return 0;
  int splits = 0;  // the two kinds of codes may pick different launch shapes
  for (bool asym : {false, true}) splits = std::max(splits, q4::gemm_splits(B, out, in, group, asym));
  return splits > 0 && grid_ok(B, out, in) ? product_bytes(splits, B, out) + t_bytes(B, in, rank) : 0;
}

q4_status q4_gemm_lora(const void* x, int64_t B, const void* packed, const void* scales, const void* zeros,
                       int64_t out, int64_t in, int32_t group, const void* lora_a, const void* lora_b,
                       const float* scaling, int64_t adapters, int32_t rank, const int32_t* ids, void* y,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (adapters < 0 || adapters >= kMaxDim) return fail(Q4_ERR_SHAPE, "adapters=%lld out of range", (long long)adapters);
  if (!rank_ok(rank)) return fail(Q4_ERR_UNSUPPORTED, "rank=%d must be a multiple of 8 in [8, 128]", (int)rank);
  q4::GemmArgs g{};
  q4_status st = q4::gemm_args(x, B, packed, scales, zeros, zeros != nullptr, out, in, group, y, &g);
  if (st != Q4_OK) return st;
  if (B == 0) return ok();
  if (!grid_ok(B, out, in)) return fail(Q4_ERR_SHAPE, "B=%lld: too many rows for one call", (long long)B);
  if (adapters > 0 && (!lora_a || !lora_b || !scaling || !ids))
    return fail(Q4_ERR_NULL, "lora_a, lora_b, scaling, ids must be non-NULL");
  if (adapters > 0 && (!aligned(lora_a, 16) || !aligned(lora_b, 16) || !aligned(scaling, 4) || !aligned(ids, 4)))
    return fail(Q4_ERR_ALIGN, "lora_a and lora_b need 16-byte, scaling and ids 4-byte alignment");
  const size_t need = product_bytes(g.k_splits, B, out) + t_bytes(B, in, rank);
  if (!workspace || workspace_bytes < need)
    return fail(Q4_ERR_WORKSPACE, "this shape needs %zu bytes of workspace (q4_workspace_bytes_lora), got %zu", need,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned(workspace, 16)) return fail(Q4_ERR_ALIGN, "workspace needs 16-byte alignment");
  g.workspace = workspace;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (adapters == 0) return hip_status(q4::launch_gemm(g, s), "gemm launch");
  g.partials = true;
  q4::LoraArgs a{};
  a.x = x, a.B = g.B, a.N = g.N, a.K = g.K;
  a.lora_a = lora_a, a.lora_b = lora_b, a.scaling = scaling, a.ids = ids;
  a.adapters = (int)adapters, a.rank = rank;
  a.partials = static_cast<const float*>(workspace), a.gemm_splits = g.k_splits;
  a.t = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                  product_bytes(g.k_splits, B, out));
  a.y = y;
  a.phase = 0;
  hipError_t e = q4::launch_lora(a, s);
  if (e == hipSuccess) e = q4::launch_gemm(g, s);
  a.phase = 1;
  if (e == hipSuccess) e = q4::launch_lora(a, s);
  return hip_status(e, "adapter product launch");
}

}  // extern "C"
