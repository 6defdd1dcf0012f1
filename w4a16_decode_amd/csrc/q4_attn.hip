// Attention of new tokens over the paged INT4 KV cache (include/q4_attn.h): launches of the
// kernels in q4_attn_kernels.h.
#include "q4_attn_kernels.h"

namespace q4 {

int attention_resident(int head_dim, int group, int rows_group) {
#define Q4_CALL(D, GC) resident_t<D, GC, kPlain>(rows_group)
  Q4_ATTN_DISPATCH(head_dim, group, Q4_CALL)
#undef Q4_CALL
}

hipError_t launch_attention(const AttnArgs& a, hipStream_t stream) {
#define Q4_CALL(D, GC) launch_t<D, GC, kPlain>(a, stream)
  Q4_ATTN_DISPATCH(a.cache.head_dim, a.cache.group, Q4_CALL)
#undef Q4_CALL
}

}  // namespace q4
