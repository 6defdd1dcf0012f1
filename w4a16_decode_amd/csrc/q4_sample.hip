// The next tokens from rows of logits (include/q4_serve.h).
//
// Weights are whole numbers: w_i = rint(2^shift exp((l_i - m) / T)) in 64 bits, the row's sum
// below 2^63. Their sums are exact, so any split and any order of additions gives the same
// cuts and the same token.
//
// Ranks. key = (descending logit, ascending index) in 64 bits orders a row's tokens without
// ties. top-k and top-p each leave the tokens up to some key, found digit by digit from the
// top: sums (of ones or of weights) over the tokens that share the digits found so far, by
// their next digit.
#include "q4_device.h"
#include "q4_internal.h"

namespace q4 {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024, kWaves = kThreads / kWave;
constexpr int kDigits = 256;

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  float v;
  if constexpr (DT == 0)
    v = (float)static_cast<const _Float16*>(p)[i];
  else if constexpr (DT == 1)
    v = __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else
    v = static_cast<const float*>(p)[i];
  return v == v ? v + 0.0f : -__builtin_inff();  // no NaN, one zero
}

// Larger for larger logits.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ u64 rank_key(float v, int i) { return (u64)~ordered(v) << 32 | (uint32_t)i; }

// A row's settings.
struct Row {
  const void* logits;
  int vocab, shift;
  float top;     // largest logit
  double slope;  // log2(e) / temperature
  int k;         // tokens that top-k leaves (vocab: all)
  bool cut_p;
  double p;
  u64 w_min;  // smallest weight that min-p leaves
  double u;
};

__device__ __forceinline__ double exponent(const Row& r, float v) {
  if (v == r.top) return 0.0;
  return r.top == __builtin_inff() ? -__builtin_inf() : ((double)v - (double)r.top) * r.slope;
}
__device__ __forceinline__ u64 weight(const Row& r, float v) {
  if (v == -__builtin_inff()) return 0;
  return (u64)rint(ldexp(exp2(exponent(r, v)), r.shift));
}

struct Shared {
  u64 sums[kDigits];
  u64 wave[kWaves];
  u64 found[2];
};

__device__ __forceinline__ u64 block_sum(u64 v, Shared& s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v += __shfl_xor(v, m, 64);
  if (lane == 0) s.wave[wave] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < kWaves; ++w) v += s.wave[w];
  __syncthreads();
  return v;
}

// Smallest key up to which the tokens with keys <= last add up to `target` or more (value(i, v)
// each; 1 <= target <= their total); *upto: that sum.
template <int DT, typename Value>
__device__ u64 select_key(const Row& r, u64 last, u64 target, Shared& s, Value value) {
  u64 prefix = 0, before = 0;
  for (int bit = 56; bit >= 0; bit -= 8) {
    if (threadIdx.x < kDigits) s.sums[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < r.vocab; i += kThreads) {
      const float v = load_logit<DT>(r.logits, i);
      const u64 key = rank_key(v, i);
      if (key <= last && (bit == 56 || key >> (bit + 8) == prefix >> (bit + 8)))
        atomicAdd(&s.sums[key >> bit & 255], value(v));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      u64 sum = before;
      int d = 0;
      while (d < kDigits - 1 && sum + s.sums[d] < target) sum += s.sums[d++];
      s.found[0] = (u64)d;
      s.found[1] = sum;
    }
    __syncthreads();
    prefix |= s.found[0] << bit;
    before = s.found[1];
    __syncthreads();
  }
  return prefix;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
  __shared__ Shared s;
  __shared__ float tops[kWaves];
  const int row = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Row r;
  r.vocab = a.vocab;
  r.shift = a.shift;
  r.logits = static_cast<const char*>(a.logits) + (int64_t)row * a.stride * (DT == 2 ? 4 : 2);
  float top = -__builtin_inff();
  for (int i = threadIdx.x; i < r.vocab; i += kThreads) top = fmaxf(top, load_logit<DT>(r.logits, i));
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, tops[w]);
  r.top = top;
  if (top == -__builtin_inff()) {
    if (threadIdx.x == 0) {
      a.tokens[row] = -1;
      if (a.probs) a.probs[row] = 0.0f;
    }
    return;
  }
  const float t = a.temperature ? a.temperature[row] : 1.0f;
  r.slope = t > 0.0f ? 1.4426950408889634 / (double)t : __builtin_inf();
  r.k = a.top_k ? a.top_k[row] : 0;
  r.k = t > 0.0f ? (r.k > 0 && r.k < r.vocab ? r.k : r.vocab) : 1;
  r.p = a.top_p ? (double)a.top_p[row] : 1.0;
  r.cut_p = r.p < 1.0;
  const double pm = a.min_p ? (double)a.min_p[row] : 0.0, one = ldexp(1.0, r.shift);
  r.w_min = pm > 0.0 ? (u64)ceil((pm < 1.0 ? pm : 1.0) * one) : 0;
  r.u = (double)a.uniforms[row];

  u64 last = ~0ull;
  if (r.k < r.vocab) last = select_key<DT>(r, last, (u64)r.k, s, [](float) { return (u64)1; });
  if (r.cut_p) {
    u64 sum = 0;
    for (int i = threadIdx.x; i < r.vocab; i += kThreads) {
      const float v = load_logit<DT>(r.logits, i);
      if (rank_key(v, i) <= last) sum += weight(r, v);
    }
    sum = block_sum(sum, s);
    const double part = ceil(r.p * (double)sum);
    u64 target = part >= 1.0 ? (u64)part : 1;
    target = target < sum ? target : sum;
    last = select_key<DT>(r, last, target, s, [&](float v) { return weight(r, v); });
  }
  auto kept = [&](int i) {
    const float v = load_logit<DT>(r.logits, i);
    const u64 w = rank_key(v, i) <= last ? weight(r, v) : 0;
    return w >= r.w_min ? w : 0;
  };
  // each thread a run of tokens
  const int run = (r.vocab + kThreads - 1) / kThreads;
  const int i0 = min((int)threadIdx.x * run, r.vocab), i1 = min(i0 + run, r.vocab);
  u64 own = 0;
  for (int i = i0; i < i1; ++i) own += kept(i);
  u64 incl = own;
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    const u64 up = __shfl_up(incl, m, 64);
    if (lane >= m) incl += up;
  }
  if (lane == kWave - 1) s.wave[wave] = incl;
  __syncthreads();
  u64 total = 0, before = incl - own;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += s.wave[w];
    total += s.wave[w];
  }
  const double at = r.u > 0.0 ? floor(r.u * (double)total) : 0.0;
  u64 draw = at < 9.2e18 ? (u64)at : total;
  draw = draw < total ? draw : total - 1;
  if (draw >= before && draw < before + own) {
    int i = i0;
    for (u64 sum = before + kept(i); sum <= draw; sum += kept(i)) ++i;
    a.tokens[row] = i;
    if (a.probs)
      a.probs[row] = (float)(exp2(exponent(r, load_logit<DT>(r.logits, i))) / ((double)total / one));
  }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)a.rows), block(kThreads);
  if (a.dtype == 0)
    hipLaunchKernelGGL((sample_kernel<0>), grid, block, 0, stream, a);
  else if (a.dtype == 1)
    hipLaunchKernelGGL((sample_kernel<1>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((sample_kernel<2>), grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace q4
