// Low-rank adapters of many requests beside the shared W4A16 product (include/q4_lora.h):
//
//   y[b] = x[b] W_hat^T + scaling[a] * B_a (A_a x[b]),  a = ids[b].
//
// Two thin products around the shared one. The first, t = A_a x (rank x in), reads each
// adapter's A once per 16 rows: a workgroup takes one tile of 16 rows, one of the
// distinct adapters among them and one slice of the channels, multiplies the whole
// tile by that adapter on the matrix cores and keeps the columns that asked for it
// (the others' results are discarded: the matrix work is free next to A's bytes). Slices
// of the channels go to separate workgroups, as there are few tiles in a decode
// batch. The second, B_a t (out x rank), is added to the product's float32 sums where
// they are rounded, so the product itself leaves float32 sums in the workspace.
//
// Bound: launches for few rows (4096 x 4096, rank 16, one row: 3.6 us A x, 5.8 the product, 2.6
// B t), the product for many (28672 x 8192, rank 32, 192 rows: 6 + 130 + 20 us of kernel time
// one by one, 138 together with gaps and tails overlapped; the product alone 132).
#include <algorithm>

#include "q4_device.h"
#include "q4_internal.h"

namespace q4 {
namespace {

constexpr int kShrinkWaves = 4;

// The j-th distinct adapter (in order of first appearance) among the ids of lanes 0..15,
// or -1; uniform.
__device__ __forceinline__ int distinct_id(int id, bool valid, int col, int j) {
  bool dup = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int other = __builtin_amdgcn_readlane(id, i);
    dup |= i < col && other == id;
  }
  uint32_t first = (uint32_t)__ballot(valid && !dup) & 0xFFFFu;
  for (; j > 0 && first; --j) first &= first - 1;
  if (!first) return -1;
  return __builtin_amdgcn_readlane(id, __builtin_ctz(first));
}

// t partials of one channel slice: tp[split][b][rank] (float32).
template <int RT>
__global__ __launch_bounds__(kShrinkWaves * 64) void lora_shrink_kernel(LoraArgs a, int splits, int slots,
                                                                        int blocks_per_split) {
  __shared__ float4_t part[kShrinkWaves][RT][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, c4 = lane >> 4;
  const int split = blockIdx.x % splits;
  const int j = blockIdx.x / splits % slots;
  const int64_t tile = blockIdx.x / splits / slots;
  const int64_t b = tile * 16 + col;
  const int id = b < a.B ? a.ids[b] : -1;
  const bool valid = id >= 0 && id < a.adapters;
  const int adapter = distinct_id(id, valid, col, j);
  if (adapter < 0) return;  // the whole workgroup: the same ids in every wavefront

  const uint16_t* x = static_cast<const uint16_t*>(a.x) + min(b, (int64_t)a.B - 1) * a.K + 8 * c4;
  const uint16_t* w = static_cast<const uint16_t*>(a.lora_a) + (int64_t)adapter * a.rank * a.K + 8 * c4;
  const uint16_t* row[RT];
  float4_t acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    row[t] = w + (int64_t)min(16 * t + col, a.rank - 1) * a.K;
    acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
  }
  const int blocks = (a.K + kSuperK - 1) / kSuperK;
  const int end = min((split + 1) * blocks_per_split, blocks);
  for (int s = split * blocks_per_split + wave; s < end; s += kShrinkWaves) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int k = s * kSuperK + m * kBlockK;
      if (k >= a.K) break;
      const half8_t xv = as_half8(*reinterpret_cast<const uint4*>(x + k));
#pragma unroll
      for (int t = 0; t < RT; ++t)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_half8(*reinterpret_cast<const uint4*>(row[t] + k)), xv,
                                                        acc[t], 0, 0, 0);
    }
  }
#pragma unroll
  for (int t = 0; t < RT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < RT; t += kShrinkWaves) {
    float4_t sum = part[0][t][lane];
#pragma unroll
    for (int v = 1; v < kShrinkWaves; ++v) sum += part[v][t][lane];
    const int r = 16 * t + 4 * c4;
    if (id == adapter && r < a.rank)
      *reinterpret_cast<float4_t*>(a.t + ((int64_t)split * a.B + b) * a.rank + r) = sum;
  }
}

// y = the product's split sums + scaling * B t, for `rows` (at most 16) rows and 256
// outputs a workgroup; a thread owns one output channel and keeps its B row while the
// adapter stays the same.
template <int RT>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs a, int splits, int n_blocks, int rows) {
  __shared__ float t[16][16 * RT];
  __shared__ int ids[16];
  const int nb = blockIdx.x % n_blocks;
  const int b0 = (int)(blockIdx.x / n_blocks) * rows;
  const int nrows = min(rows, a.B - b0);
  for (int e = threadIdx.x; e < nrows * 16 * RT; e += 256) {
    const int i = e / (16 * RT), r = e % (16 * RT);
    const int id = a.ids[b0 + i];
    const bool real = id >= 0 && id < a.adapters;
    if (r == 0) ids[i] = real ? id : -1;
    float sum = 0.0f;
    if (real && r < a.rank) {
      const float* src = a.t + (int64_t)(b0 + i) * a.rank + r;
      const int64_t stride = (int64_t)a.B * a.rank;
#pragma unroll 8
      for (int s = 0; s < splits; ++s) sum += src[s * stride];
      sum *= a.scaling[id];
    }
    t[i][r] = sum;
  }
  __syncthreads();
  const int n = nb * 256 + threadIdx.x;
  if (n >= a.N) return;
  uint16_t* y = static_cast<uint16_t*>(a.y);
  const int64_t split_stride = (int64_t)a.B * a.N;
  half8_t w[2 * RT];
  int held = -1;
  for (int i0 = 0; i0 < nrows; i0 += 4) {
    // four rows' sums in flight
    float sum[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float* src = a.partials + (int64_t)(b0 + min(i0 + u, nrows - 1)) * a.N + n;
      sum[u] = 0.0f;
#pragma unroll 2
      for (int k = 0; k < a.gemm_splits; ++k) sum[u] += src[k * split_stride];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u;
      if (i >= nrows) break;
      const int id = ids[i];
      if (id >= 0) {
        if (id != held) {
          const uint16_t* src = static_cast<const uint16_t*>(a.lora_b) + ((int64_t)id * a.N + n) * a.rank;
#pragma unroll
          for (int q = 0; q < 2 * RT; ++q)  // zeros behind the rank: 0 * infinity must not arise
            w[q] = as_half8(8 * q < a.rank ? *reinterpret_cast<const uint4*>(src + 8 * q) : make_uint4(0u, 0u, 0u, 0u));
          held = id;
        }
        float d = 0.0f;
#pragma unroll
        for (int q = 0; q < 2 * RT; ++q)
#pragma unroll
          for (int e = 0; e < 8; ++e) d = __builtin_fmaf((float)w[q][e], t[i][8 * q + e], d);
        sum[u] += d;
      }
      y[(int64_t)(b0 + i) * a.N + n] = __builtin_bit_cast(uint16_t, (_Float16)sum[u]);
    }
  }
}

// Workgroups' channel slices: 128-channel blocks each, at least one per wavefront.
int shrink_blocks_per_split(int K) {
  const int blocks = (K + kSuperK - 1) / kSuperK;
  return std::min(blocks, 2 * kShrinkWaves);
}

template <int RT>
void launch_t(const LoraArgs& a, hipStream_t stream) {
  const int per = shrink_blocks_per_split(a.K), splits = lora_splits(a.K);
  const int slots = (int)std::min<int64_t>(std::min<int64_t>(16, a.B), a.adapters);
  const int64_t tiles = (a.B + 15) / 16;
  const int n_blocks = (a.N + 255) / 256;
  if (a.phase == 0)
    hipLaunchKernelGGL(lora_shrink_kernel<RT>, dim3((unsigned)(tiles * slots * splits)), dim3(kShrinkWaves * 64), 0,
                       stream, a, splits, slots, per);
  else {
    // rows a workgroup takes: 16 where that still fills the chip (a B row then serves a run
    // of rows of one request), fewer in a decode batch, whose rows each bring their own
    int rows = 16;
    while (rows > 1 && (a.B + rows - 1) / rows * (int64_t)n_blocks < 2 * device_cu_count_cached()) rows /= 2;
    hipLaunchKernelGGL(lora_expand_kernel<RT>, dim3((unsigned)((a.B + rows - 1) / rows * (int64_t)n_blocks)), dim3(256),
                       0, stream, a, splits, n_blocks, rows);
  }
}

}  // namespace

int lora_splits(int K) {
  const int blocks = (K + kSuperK - 1) / kSuperK, per = shrink_blocks_per_split(K);
  return (blocks + per - 1) / per;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t stream) {
  if (a.rank <= 16) launch_t<1>(a, stream);
  else if (a.rank <= 32) launch_t<2>(a, stream);
  else if (a.rank <= 64) launch_t<4>(a, stream);
  else launch_t<8>(a, stream);
  return hipGetLastError();
}

}  // namespace q4
