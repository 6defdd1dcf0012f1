// Attention of requests that share long prefixes over the paged INT4 KV cache
// (include/q4_attn.h).
//
//   o = (sum_prefix p_t v_t + sum_own p_t v_t) / (sum_prefix p_t + sum_own p_t)
//
// The rows of all members of a group see every key of their prefix, so together they are one
// many-row product over it: the prefix is read and its codes converted once for 128 rows instead
// of once a request. Three steps: the 128-row kernel over the prefixes, each job's keys cut
// into pieces until the chip is full; a join of the pieces into each row's output and the
// logarithm of its sum of weights; and the kernels of q4_attn.hip over the keys behind the
// prefix, whose rows start from that output with that logarithm as their maximum, as if the
// prefix had been one key.
#include "q4_attn_kernels.h"

namespace q4 {
namespace {

// Group whose member rows hold `token` (uniform), and its first row and number of rows.
__device__ __forceinline__ int group_of(const AttnArgs& a, int token, int* first, int* rows) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < a.seqs; base += kWave) {
    int from = 0, n = 0;
    if (base + lane < a.seqs) {
      const int begin = min(max(a.group_offsets[base + lane], 0), a.members);
      const int end = min(max(a.group_offsets[base + lane + 1], begin), a.members);
      from = min(max(a.q_offsets[begin], 0), a.tokens);
      n = min(min(max(a.q_offsets[end], from), a.tokens) - from, a.max_q);
    }
    const uint64_t in = __ballot(token >= from && token - from < n);
    if (in) {
      const int at = __builtin_ctzll(in);
      *first = uniform(__shfl(from, at, 64));
      *rows = uniform(__shfl(n, at, 64));
      return base + at;
    }
  }
  return -1;
}

// A wavefront a row: D / 4 lanes of four channels each, the 256 / D groups of lanes taking every such
// piece, added in order.
template <int D>
__global__ __launch_bounds__(256) void prefix_join_kernel(AttnArgs a, int tiles, int swizzle) {
  constexpr int LPR = D / 4, G = kWave / LPR;
  const int64_t r = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
  if (r >= (int64_t)a.tokens * a.q_heads) return;
  const int token = uniform((int)(r / a.q_heads)), head = (int)(r - (int64_t)token * a.q_heads);
  const int share = a.q_heads / a.cache.kv_heads;
  const int lane = threadIdx.x & 63;
  int first, rows;
  const int group = group_of(a, token, &first, &rows);
  if (group < 0) {
    if (lane == 0) *reinterpret_cast<float2*>(a.init_ml + 2 * r) = make_float2(kLowest, 0.0f);
    return;
  }
  // the row's place among the jobs (rows_job)
  const int kv_head = head / share, local = (token - first) * share + head - kv_head * share;
  const unsigned line = (unsigned)group * a.cache.kv_heads + kv_head, at_tile = tiles - 1 - local / 128;
  const unsigned job = swizzle ? ((line / 8) * tiles + at_tile) * 8 + line % 8 : line * tiles + at_tile;
  auto at = [&](int i) __attribute__((always_inline)) { return ((int64_t)i * a.tail + job) * 128 + local % 128; };
  const int g = lane / LPR, ch = 4 * (lane % LPR);
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  float top = kLowest, sum = 0.0f;
  float4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = g; i < a.pieces; i += G) top = fmaxf(top, ml[at(i)].x);
#pragma unroll
  for (int m = LPR; m < kWave; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
#pragma unroll 4
  for (int i = g; i < a.pieces; i += G) {
    const float2 v = ml[at(i)];
    const float f = exp2_fast(v.x - top);
    sum = __builtin_fmaf(v.y, f, sum);
    o += *reinterpret_cast<const float4_t*>(a.part_o + at(i) * D + ch) * f;
  }
#pragma unroll
  for (int m = LPR; m < kWave; m <<= 1) {
    sum += __shfl_xor(sum, m, 64);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], m, 64);
  }
  if (g == 0) *reinterpret_cast<float4_t*>(a.init_o + r * D + ch) = o * (1.0f / sum);
  if (lane == 0)
    *reinterpret_cast<float2*>(a.init_ml + 2 * r) =
        sum <= 0.0f ? make_float2(kLowest, sum) : make_float2(top + __builtin_amdgcn_logf(sum), 1.0f);
}

template <int D, int GC>
hipError_t prefix_t(const AttnArgs& a, hipStream_t stream) {
  const int64_t rows = (int64_t)a.max_q * (a.q_heads / a.cache.kv_heads);
  const int tiles = (int)((rows + 127) / 128);
  const int swizzle = (int64_t)a.cache.kv_heads * a.seqs % 8 == 0 && tiles > 1;
  hipLaunchKernelGGL((attn_rows_kernel<D, GC, true, kPrefix>), dim3((unsigned)(a.tail * a.pieces)), dim3(256),
                     sizeof(Shared<D, GC>), stream, a, tiles, swizzle);
  hipLaunchKernelGGL(prefix_join_kernel<D>, dim3((unsigned)(((int64_t)a.tokens * a.q_heads + 3) / 4)), dim3(256), 0,
                     stream, a, tiles, swizzle);
  return hipGetLastError();
}

template <int D, int GC>
int prefix_resident_t() {
  return resident_per_cu(reinterpret_cast<const void*>(&attn_rows_kernel<D, GC, true, kPrefix>), 256,
                         sizeof(Shared<D, GC>)) *
         device_cu_count_cached();
}

}  // namespace

int prefix_attention_resident(int head_dim, int group) {
#define Q4_CALL(D, GC) prefix_resident_t<D, GC>()
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
