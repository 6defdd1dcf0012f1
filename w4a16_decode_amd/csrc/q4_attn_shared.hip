// Attention of requests that share long prefixes over the paged INT4 KV cache
// (include/q4_attn.h).
//
//   o = (sum_prefix p_t v_t + sum_own p_t v_t) / (sum_prefix p_t + sum_own p_t)
//
// The rows of all members of a group see every key of their prefix, so together they are one
// many-row product over it: the prefix is read and its codes converted once for a tile of rows
// instead of once a request. Three forms (q4_attn_api.cpp picks one), all of q4_attn_kernels.h:
//   both    few rows: tiles of 16 rows over the prefixes and over the sequences' own keys in one launch, all cut
//           into pieces of about equal length that leave (O, m + E, l) a row, and their join;
//   behind  more rows: 128-row workgroups over the prefixes, cut until the chip is full, and then the
//           attention of q4_paged_attention over the own keys, whose rows start from the sum of
//           those pieces as if they had seen the prefix's keys already;
//   line    many rows of each sequence: 128-row workgroups that walk prefix and own keys as one line.
// 64 rows behind 8190 keys, 64 heads over 8 of 128 channels: 38 + 17 us, the prefix at 450 TFLOP/s; its
// 512 rows a head are 32 tiles, which fill the chip in eight pieces of 1024 keys. No unit is full meanwhile: with 14.4
// vector instructions a product the vector units issue 40 to 46 % of the time and the matrix units work 21 %. The two
// wavefronts a SIMD wait for each other's barrier and for their own chains (products, maximum, exponentials,
// products); behind the prefix vector work is 30 % and the rest latency. Nine chunks of up to 251 rows behind two
// prefixes of up to 6001 keys: 484 to 496 us, 650 TFLOP/s. 8 rows behind 1003 keys: 11 us, two launches' latency.
#include "q4_attn_kernels.h"

namespace q4 {
namespace {

// Whether eight wavefronts take a piece (HALVES): 256 channels would leave them too few registers.
constexpr bool halves(int head_dim) { return head_dim <= 128; }
template <int D, int GC>
constexpr size_t prefix_lds() {
  return (halves(D) ? 4 : 1) * sizeof(Shared<D, GC>);
}

template <int D, int GC>
hipError_t prefix_t(const AttnArgs& a, hipStream_t stream) {
  const int tiles = a.prefix_rows / 128;
  const int swizzle = (int64_t)a.cache.kv_heads * a.groups % 8 == 0 && tiles > 1;
  hipLaunchKernelGGL((attn_rows_kernel<D, GC, true, kPrefix, halves(D)>), dim3((unsigned)(a.tail * a.pieces)),
                     dim3(halves(D) ? 512 : 256), (prefix_lds<D, GC>()), stream, a, tiles, swizzle);
  return hipGetLastError();
}

template <int D, int GC>
hipError_t both_t(const AttnArgs& a, hipStream_t stream) {
  const int64_t rows = (int64_t)a.max_q * (a.q_heads / a.cache.kv_heads);
  const int tiles = (int)((rows + 15) / 16);
  const int64_t over = (int64_t)a.prefix_rows / 16 * a.cache.kv_heads * a.groups * a.prefix_pieces;
  const int64_t own = (int64_t)tiles * a.cache.kv_heads * a.seqs;
  hipLaunchKernelGGL((attn16_kernel<D, GC, false, kBoth>), dim3((unsigned)(over + own * a.own_pieces)), dim3(256), 0,
                     stream, a, tiles);
  hipLaunchKernelGGL(attn_join_both_kernel<D>, dim3((unsigned)own), dim3(kJoinBoth), 0, stream, a, tiles);
  return hipGetLastError();
}

template <int D, int GC>
hipError_t line_t(const AttnArgs& a, hipStream_t stream) {
  const int64_t rows = (int64_t)a.max_q * (a.q_heads / a.cache.kv_heads);
  const int tiles = (int)((rows + 127) / 128);
  const int swizzle = (int64_t)a.cache.kv_heads * a.seqs % 8 == 0 && tiles > 1;
  hipLaunchKernelGGL((attn_rows_kernel<D, GC, true, kLine>), dim3((unsigned)(a.whole + a.tail * a.pieces)), dim3(256),
                     sizeof(Shared<D, GC>), stream, a, tiles, swizzle);
  if (a.tail > 0)
    hipLaunchKernelGGL(attn_join_rows_kernel<D>, dim3((unsigned)(a.tail * 32)), dim3(256), 0, stream, a, tiles, swizzle);
  return hipGetLastError();
}

template <int D, int GC>
int line_resident_t() {
  return resident_per_cu(reinterpret_cast<const void*>(&attn_rows_kernel<D, GC, true, kLine>), 256,
                         sizeof(Shared<D, GC>)) *
         device_cu_count_cached();
}

template <int D, int GC>
int prefix_resident_t(int rows_group) {
  if (rows_group == 16) return resident_grid(reinterpret_cast<const void*>(&attn16_kernel<D, GC, false, kBoth>), 256);
  return resident_per_cu(reinterpret_cast<const void*>(&attn_rows_kernel<D, GC, true, kPrefix, halves(D)>),
                         halves(D) ? 512 : 256, prefix_lds<D, GC>()) *
         device_cu_count_cached();
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

int line_attention_resident(int head_dim, int group) {
#define Q4_CALL(D, GC) line_resident_t<D, GC>()
  Q4_ATTN_DISPATCH(head_dim, group, Q4_CALL)
#undef Q4_CALL
}

hipError_t launch_line_attention(const AttnArgs& a, hipStream_t stream) {
#define Q4_CALL(D, GC) line_t<D, GC>(a, stream)
  Q4_ATTN_DISPATCH(a.cache.head_dim, a.cache.group, Q4_CALL)
#undef Q4_CALL
}

hipError_t launch_both_attention(const AttnArgs& a, hipStream_t stream) {
#define Q4_CALL(D, GC) both_t<D, GC>(a, stream)
  Q4_ATTN_DISPATCH(a.cache.head_dim, a.cache.group, Q4_CALL)
#undef Q4_CALL
}

hipError_t launch_behind_attention(const AttnArgs& a, hipStream_t stream) {
#define Q4_CALL(D, GC) launch_t<D, GC, kBehind>(a, stream)
  Q4_ATTN_DISPATCH(a.cache.head_dim, a.cache.group, Q4_CALL)
#undef Q4_CALL
}

}  // namespace q4
