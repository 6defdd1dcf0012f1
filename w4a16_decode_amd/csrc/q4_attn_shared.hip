// Attention of requests that share long prefixes over the paged INT4 KV cache
// (include/q4_attn.h).
//
//   o = (sum_prefix p_t v_t + sum_own p_t v_t) / (sum_prefix p_t + sum_own p_t)
//
// The rows of all members of a group see every key of their prefix, so together they are one
// many-row product over it: the prefix is read and its codes converted once for a tile of rows
// instead of once a request. Two steps: the kernels of q4_attn_kernels.h over the prefixes, each
// job's keys cut into pieces until the chip is full, which leave (O, m + E, l) of every row and
// piece; and the same kernels over the keys behind the prefix, whose rows start from the sum of
// those as if they had seen the prefix's keys already.
#include "q4_attn_kernels.h"

namespace q4 {
namespace {

template <int D, int GC>
hipError_t prefix_t(const AttnArgs& a, hipStream_t stream) {
  const int tiles = a.prefix_rows / a.rows_group;
  const int64_t lines = (int64_t)a.cache.kv_heads * a.seqs;
  const dim3 grid((unsigned)(tiles * lines * a.prefix_pieces));
  if (a.rows_group == 128) {
    const int swizzle = lines % 8 == 0 && tiles > 1;
    hipLaunchKernelGGL((attn_rows_kernel<D, GC, true, kPrefix>), grid, dim3(256), sizeof(Shared<D, GC>), stream, a, tiles,
                       swizzle);
  } else if (a.rows_group == 32) {
    if constexpr (has_attn32(D, GC))
      hipLaunchKernelGGL((attn32_kernel<D, GC, kPrefix>), grid, dim3(256), 0, stream, a, tiles);
  } else {
    hipLaunchKernelGGL((attn16_kernel<D, GC, false, kPrefix>), grid, dim3(256), 0, stream, a, tiles);
  }
  return hipGetLastError();
}

template <int D, int GC>
int prefix_resident_t(int rows_group) {
  if (rows_group == 128)
    return resident_per_cu(reinterpret_cast<const void*>(&attn_rows_kernel<D, GC, true, kPrefix>), 256,
                           sizeof(Shared<D, GC>)) *
           device_cu_count_cached();
  if constexpr (has_attn32(D, GC)) {
    if (rows_group == 32) return resident_grid(reinterpret_cast<const void*>(&attn32_kernel<D, GC, kPrefix>), 256);
  }
  return resident_grid(reinterpret_cast<const void*>(&attn16_kernel<D, GC, false, kPrefix>), 256);
}

}  // namespace

int prefix_attention_resident(int head_dim, int group, int rows_group) {
#define Q4_CALL(D, GC) prefix_resident_t<D, GC>(rows_group)
  Q4_ATTN_DISPATCH(head_dim, group, Q4_CALL)
#undef Q4_CALL
}

hipError_t launch_prefix_attention(const AttnArgs& a, hipStream_t stream) {
#define Q4_CALL(D, GC) prefix_t<D, GC>(a, stream)
  Q4_ATTN_DISPATCH(a.cache.head_dim, a.cache.group, Q4_CALL)
#undef Q4_CALL
}

hipError_t launch_behind_attention(const AttnArgs& a, hipStream_t stream) {
#define Q4_CALL(D, GC) launch_t<D, GC, kBehind>(a, stream)
  Q4_ATTN_DISPATCH(a.cache.head_dim, a.cache.group, Q4_CALL)
#undef Q4_CALL
}

}  // namespace q4
